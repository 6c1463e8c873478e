"""Refusals of the 4-bit weights' and the 8-bit pages' entry points that need no GPU, and the packed size."""
import ctypes

import pytest

from block_diffusion_speculative_target_gb300 import build, capi


@pytest.fixture(scope="module")
def lib():
    build.build()
    return capi.load()


def w4(M=256, K=256, group=128, scale=capi.BF16, zeros=0, packed=1 << 30):
    return capi.W4C(M, K, group, scale, zeros, packed)


def ref(w):
    return ctypes.byref(w) if w is not None else None


BAD = [(dict(M=0), capi.ERR_INVALID_ARG), (dict(K=0), capi.ERR_INVALID_ARG), (dict(K=-128), capi.ERR_INVALID_ARG),
       (dict(scale=2), capi.ERR_INVALID_ARG), (dict(group=16), capi.ERR_UNSUPPORTED_SHAPE),
       (dict(group=0), capi.ERR_UNSUPPORTED_SHAPE), (dict(group=256), capi.ERR_UNSUPPORTED_SHAPE),
       (dict(K=192), capi.ERR_UNSUPPORTED_SHAPE), (dict(K=48, group=32), capi.ERR_UNSUPPORTED_SHAPE),
       (dict(M=1 << 20, K=1 << 15), capi.ERR_TOO_LARGE), (dict(M=(1 << 28) + 1, K=32, group=32), capi.ERR_TOO_LARGE)]


@pytest.mark.parametrize("kw, code", BAD)
def test_shapes_refused_everywhere(lib, kw, code):
    w = w4(**kw)
    far = 1 << 40
    assert lib.dflash_w4_bytes(ref(w)) == code
    assert lib.dflash_w4_pack(ref(w), far, far, None, None) == code
    assert lib.dflash_w4_quantize(ref(w), capi.BF16, far, 1 << 28, None) == code
    assert lib.dflash_w4_unpack(ref(w), capi.BF16, far, None) == code
    assert lib.dflash_linear_w4(capi.BF16, far, 1 << 28, ref(w), None, 0, far, 1, far, None) == code


@pytest.mark.parametrize("M, K, group, scale, zeros, blocks, extra", [
    (1, 32, 32, capi.BF16, 0, 1, 4 * 128 * 2), (128, 128, 128, capi.BF16, 0, 1, 256), (129, 256, 64, capi.F32, 1, 4, 2 * 128 * 5),
    (4096, 4096, 128, capi.F32, 0, 1024, 512), (300, 160, 32, capi.BF16, 1, 6, 4 * 128 * 3)])
def test_packed_bytes(lib, M, K, group, scale, zeros, blocks, extra):
    assert lib.dflash_w4_bytes(ref(w4(M, K, group, scale, zeros, None))) == blocks * (8192 + extra)


def test_buffers_refused(lib):
    inv = capi.ERR_INVALID_ARG
    far = 1 << 40
    assert lib.dflash_w4_bytes(None) == inv
    for packed in (None, (1 << 30) + 8):
        w = w4(packed=packed)
        assert lib.dflash_w4_pack(ref(w), far, far, None, None) == inv
        assert lib.dflash_w4_unpack(ref(w), capi.BF16, far, None) == inv
        assert lib.dflash_linear_w4(capi.BF16, far, 256, ref(w), None, 0, far, 1, far, None) == inv
    w, at = w4(), 1 << 30
    assert lib.dflash_w4_pack(ref(w), None, far, None, None) == inv
    assert lib.dflash_w4_pack(ref(w), far, None, None, None) == inv
    assert lib.dflash_w4_pack(ref(w), far, far + 1, None, None) == inv       # a scale off its alignment
    assert lib.dflash_w4_pack(ref(w), far, far, far, None) == inv            # zeros that the matrix has not
    assert lib.dflash_w4_pack(ref(w4(zeros=1)), far, far, None, None) == inv  # and has
    for src in (at, at + 64, at - 64):
        assert lib.dflash_w4_pack(ref(w), src, far, None, None) == inv
        assert lib.dflash_w4_pack(ref(w), far, src, None, None) == inv
        assert lib.dflash_w4_quantize(ref(w), capi.BF16, src, 256, None) == inv
        assert lib.dflash_w4_unpack(ref(w), capi.BF16, src, None) == inv
    assert lib.dflash_w4_quantize(ref(w), 2, far, 256, None) == inv
    assert lib.dflash_w4_quantize(ref(w), capi.BF16, far, 255, None) == inv
    assert lib.dflash_w4_quantize(ref(w), capi.F32, far + 2, 256, None) == inv
    assert lib.dflash_w4_unpack(ref(w), 2, far, None) == inv
    assert lib.dflash_linear_w4(capi.BF16, far, 256, ref(w), None, 0, far, 1, None, None) == inv
    h = ctypes.c_void_p()
    assert lib.dflash_w4_workspace_alloc(0, ctypes.byref(h)) == inv
    assert lib.dflash_w4_workspace_alloc(16, None) == inv
    assert lib.dflash_w4_workspace_alloc(129, ctypes.byref(h)) == capi.ERR_TOO_LARGE
    assert lib.dflash_w4_workspace_free(None) == 0


def test_q8_pages_create_refuses(lib):
    d = capi.ModelDesc(1, 512, 4, 1, 128, 256, 256, 1e6, 1e-6, capi.BF16)
    h = ctypes.c_void_p()

    def create(k=1 << 20, v=1 << 21, ks=1 << 22, vs=1 << 23, ps=16, out=h, desc=d):
        return lib.dflash_pages_create_q8(ref(desc), 1, 4, ps, 64, k, v, ks, vs, ctypes.byref(out) if out else None)

    for kw in (dict(k=None), dict(v=None), dict(ks=None), dict(vs=None), dict(k=8), dict(v=8), dict(ks=(1 << 22) + 4),
               dict(vs=(1 << 23) + 8), dict(ps=8), dict(ps=256), dict(out=None), dict(desc=None),
               dict(desc=capi.ModelDesc(1, 512, 4, 1, 96, 256, 256, 1e6, 1e-6, capi.BF16))):
        assert create(**kw) == capi.ERR_INVALID_ARG, kw
    # parts of the pool that overlap: 4 pages of 16 rows of 128 codes, 8192 bytes, and 64 scales, 256 bytes
    for kw in (dict(v=(1 << 20) + 8176), dict(ks=(1 << 20) + 8176), dict(vs=(1 << 21) + 16), dict(vs=(1 << 22) + 240)):
        assert create(**kw) == capi.ERR_INVALID_ARG, kw


def test_read_refuses_missing_handles(lib):
    p = 1 << 20
    assert lib.dflash_paged_read(None, 0, capi.BF16, 1, 1, None, p, 4, p, p, p, None, None) == capi.ERR_INVALID_ARG
