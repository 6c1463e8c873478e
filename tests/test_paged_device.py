"""Calls of a PagedCache whose pool lies on another GPU than the current one enter the pool's device and leave it
again.  No GPU: the device, the library's calls and the tensors are stand-ins."""
import contextlib
import types

import pytest

torch = pytest.importorskip("torch")

from block_diffusion_speculative_target_gb300 import capi, engine  # noqa: E402

POOL = torch.device("cuda", 1)


class Tensor:
    """What the checks of the calls look at."""

    def __init__(self, *shape, dtype=torch.bfloat16, device=POOL):
        self.shape, self.dtype, self.device, self.is_cuda = shape, dtype, device, True

    def dim(self):
        return len(self.shape)

    def numel(self):
        n = 1
        for x in self.shape:
            n *= x
        return n

    def stride(self, i):
        n = 1
        for x in self.shape[i + 1:]:
            n *= x
        return n

    def is_contiguous(self):
        return True


@pytest.fixture
def cache(monkeypatch):
    at = {"device": 0, "calls": []}

    @contextlib.contextmanager
    def device(d):
        before, at["device"] = at["device"], d.index if isinstance(d, torch.device) else d
        try:
            yield
        finally:
            at["device"] = before

    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: at["device"])
    monkeypatch.setattr(torch.cuda, "current_stream",
                        lambda: types.SimpleNamespace(device_index=at["device"], cuda_stream=1000 + at["device"]))
    for name in ("dflash_paged_append", "dflash_paged_attention", "dflash_paged_attention_shared", "dflash_paged_status"):
        def call(*a, name=name, stream=None, **kw):
            if stream is None and hasattr(a[-1], "cuda_stream"):
                stream = a[-1]
            assert stream is None or stream.device_index == at["device"]  # the stream is that device's too
            at["calls"].append((name, at["device"]))
            if at.get("fail"):
                raise capi.DFlashError("refused", capi.ERR_INVALID_ARG)
            return 0
        monkeypatch.setattr(capi, name, call)
    c = engine.PagedCache.__new__(engine.PagedCache)
    c.dtype, c.tdt, c.nq, c.nkv, c.hd, c.page_size, c.max_pos = "bf16", torch.bfloat16, 4, 1, 128, 16, 64
    c.device, c.pages, c.ws = POOL, None, None
    return c, at


def i32(*shape):
    return Tensor(*shape, dtype=torch.int32)


@pytest.mark.parametrize("current", [0, 1])
def test_calls_enter_the_pools_device(cache, current):
    c, at = cache
    at["device"] = current
    q, qkv = Tensor(2, 3, 4, 128), Tensor(6, 6 * 128)
    table, lens = i32(2, 4), i32(2)

    def calls():
        c.append(0, qkv, table, lens, 3, q_out=q)
        c.attention(0, q, table, lens, Tensor(2, 3, 4, 128))
        c.attention(0, q, table, lens, Tensor(2, 3, 4, 128), shared_len=i32(1))
        c.status()

    calls()
    assert at["calls"] == [(n, 1) for n in ("dflash_paged_append", "dflash_paged_attention",
                                            "dflash_paged_attention_shared", "dflash_paged_status")]
    assert at["device"] == current
    # and leave it when a call is refused
    at["fail"] = True
    with pytest.raises(capi.DFlashError):
        c.status()
    with pytest.raises(capi.DFlashError):
        c.append(0, qkv, table, lens, 3, q_out=q)
    with pytest.raises(ValueError):  # tensors of another device stay refused
        c.attention(0, Tensor(2, 3, 4, 128, device=torch.device("cuda", 0)), table, lens, q)
    assert at["device"] == current
