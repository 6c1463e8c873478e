"""Refusals of the paged-cache entry points that need no GPU."""
import ctypes

import pytest

from block_diffusion_speculative_target_gb300 import build, capi


@pytest.fixture(scope="module")
def lib():
    build.build()
    return capi.load()


def desc(nq=4, nkv=1, hd=128, dtype=capi.BF16, theta=1e6):
    return capi.ModelDesc(1, 512, nq, nkv, hd, 256, 256, theta, 1e-6, dtype)


def create(lib, d, n_layers=1, n_pages=4, page_size=16, max_pos=64, k=1 << 20, v=1 << 21):
    h = ctypes.c_void_p()
    return lib.dflash_pages_create(ctypes.byref(d) if d is not None else None, n_layers, n_pages, page_size, max_pos, k,
                                   v, ctypes.byref(h))


def test_pages_create_refuses(lib):
    assert lib.dflash_pages_create(ctypes.byref(desc()), 1, 4, 16, 64, 1 << 20, 1 << 21, None) == capi.ERR_INVALID_ARG
    for kw in (dict(n_layers=0), dict(n_pages=0), dict(page_size=0), dict(page_size=8), dict(page_size=48),
               dict(page_size=256), dict(max_pos=0), dict(k=None), dict(v=None), dict(k=8), dict(v=(1 << 20) + 2)):
        assert create(lib, desc(), **kw) == capi.ERR_INVALID_ARG, kw
    assert create(lib, None) == capi.ERR_INVALID_ARG
    assert create(lib, desc(nq=4, nkv=3)) == capi.ERR_INVALID_ARG
    assert create(lib, desc(hd=96)) == capi.ERR_INVALID_ARG
    for theta in (0.0, -1.0, float("inf"), float("nan")):
        assert create(lib, desc(theta=theta)) == capi.ERR_INVALID_ARG
    assert create(lib, desc(nq=65)) == capi.ERR_UNSUPPORTED_SHAPE
    assert create(lib, desc(), n_pages=1 << 27) == capi.ERR_TOO_LARGE  # 2^31 pool rows


def test_workspace_refuses(lib):
    h = ctypes.c_void_p()
    d = desc()
    assert lib.dflash_paged_workspace_alloc(ctypes.byref(d), 1, 1, None) == capi.ERR_INVALID_ARG
    for batch, rows in ((0, 4), (5, 4), (1, 0)):
        assert lib.dflash_paged_workspace_alloc(ctypes.byref(d), batch, rows, ctypes.byref(h)) == capi.ERR_INVALID_ARG
    assert lib.dflash_paged_workspace_alloc(None, 1, 1, ctypes.byref(h)) == capi.ERR_INVALID_ARG
    assert lib.dflash_paged_workspace_alloc(ctypes.byref(d), 1, (1 << 20) + 1, ctypes.byref(h)) == capi.ERR_TOO_LARGE
    big = desc(nq=128)
    assert lib.dflash_paged_workspace_alloc(ctypes.byref(big), 1, 1, ctypes.byref(h)) == capi.ERR_UNSUPPORTED_SHAPE


def test_calls_refuse_missing_handles(lib):
    p = 1 << 20  # never read: the handles are checked first
    assert lib.dflash_paged_append(None, 0, 0, p, 768, 1, 1, None, p, 4, p, None, None, None) == capi.ERR_INVALID_ARG
    assert lib.dflash_paged_attention(None, 0, p, 1, 1, None, 1, 0, 0, p, 4, p, p, None, None) == capi.ERR_INVALID_ARG
    assert lib.dflash_paged_attention_shared(None, 0, p, 1, 1, None, 1, 0, 0, p, 4, p, p, p, None,
                                             None) == capi.ERR_INVALID_ARG
    assert lib.dflash_paged_status(None, None, None) == capi.ERR_INVALID_ARG
    assert lib.dflash_pages_free(None) == 0 and lib.dflash_paged_workspace_free(None) == 0
