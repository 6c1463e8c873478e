"""Weights in 4 bits on the GPU: packing, quantising and reading back, and the products, against plain arithmetic in
64 bits."""
import pytest

torch = pytest.importorskip("torch")

from block_diffusion_speculative_target_gb300 import capi  # noqa: E402
from block_diffusion_speculative_target_gb300.engine import W4Linear, W4Workspace  # noqa: E402

pytestmark = pytest.mark.gpu

TDT = {"f32": torch.float32, "bf16": torch.bfloat16}


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(4000 + seed)


class Codes:
    """A matrix as plain arrays, packed, and its values in 64 bits."""

    def __init__(self, M, K, group, scales="bf16", zeros=False, seed=0):
        g = gen(seed)
        self.M, self.K, self.group = M, K, group
        self.code = torch.randint(0, 16, (M, K), dtype=torch.uint8, device="cuda", generator=g)
        s = torch.empty(M, K // group, device="cuda").uniform_(0.5, 3.0, generator=g)
        # some scales are zero, some negative (a checkpoint may hold either)
        pick = torch.rand(M, K // group, device="cuda", generator=g)
        self.scales = torch.where(pick < 0.05, torch.zeros_like(s), torch.where(pick < 0.2, -s, s)).to(TDT[scales])
        self.zeros = torch.randint(0, 16, (M, K // group), dtype=torch.uint8, device="cuda", generator=g) if zeros else None
        self.w4 = W4Linear.from_codes(self.code[:, 0::2] | self.code[:, 1::2] << 4, self.scales, self.zeros)
        z = 8.0 if self.zeros is None else self.zeros.double().repeat_interleave(group, 1)
        self.w = (self.code.double() - z) * self.scales.double().repeat_interleave(group, 1)


SIZES = [(1, 32, 32), (2, 64, 64), (17, 96, 32), (127, 160, 32), (128, 128, 128), (129, 192, 64), (300, 384, 128),
         (1000, 1184, 32), (640, 2560, 64)]


@pytest.mark.parametrize("M, K, group", SIZES)
@pytest.mark.parametrize("scales, zeros", [("bf16", False), ("f32", True), ("bf16", True), ("f32", False)])
def test_pack_and_back(M, K, group, scales, zeros):
    c = Codes(M, K, group, scales, zeros)
    assert torch.equal(c.w4.weight(torch.float32), c.w.float())
    # (a bf16 value is the exact one rounded once: at most 12 bits of it are lost by no other step)
    assert torch.equal(c.w4.weight(torch.bfloat16), c.w.float().to(torch.bfloat16))


def test_zero_points_above_15_count_as_15():
    code = torch.zeros(4, 16, dtype=torch.uint8, device="cuda")
    z = torch.tensor([[15], [16], [200], [255]], dtype=torch.uint8, device="cuda")
    w = W4Linear.from_codes(code, torch.ones(4, 1, device="cuda"), z).weight()
    assert (w == -15).all()


@pytest.mark.parametrize("M, K, group", SIZES)
@pytest.mark.parametrize("scales, zeros", [("bf16", False), ("f32", True)])
@pytest.mark.parametrize("dtype, pad", [("bf16", 0), ("f32", 3)])
def test_quantize(M, K, group, scales, zeros, dtype, pad):
    """The codes of the stated rule, value for value (each of its steps is one float32 operation)."""
    src = torch.empty(M, K + pad, dtype=TDT[dtype], device="cuda").normal_(0, 0.02, generator=gen(1))[:, :K]
    if M > 2:
        src[1] = 0.0
        src[2] = src[2].abs() + 0.01  # a row without negative values
    got = W4Linear.from_weight(src, group, TDT[scales], zeros).weight()
    x = src.float().reshape(M, K // group, group)
    hi, lo = x.amax(-1).clamp(min=0), x.amin(-1).clamp(max=0)
    # (in torch a float32 tensor over a number is a product with the number's inverse; the quotient in 64 bits, rounded,
    # is float32's own)
    s = ((hi - lo).double() / 15 if zeros else torch.maximum(hi, -lo).double() / 7).float().to(TDT[scales]).float()
    some = s > 0
    z = torch.where(some, torch.round(-lo / s).clamp(0, 15), torch.full_like(s, 8.0)) if zeros else torch.full_like(s, 8.0)
    q = torch.where(some[..., None], (torch.round(x / s[..., None]) + z[..., None]).clamp(0, 15), z[..., None])
    want = ((q - z[..., None]) * s[..., None]).view(M, K)
    assert torch.equal(got, want)
    # and they are near: half a step, where the range is not cut (a rounded scale, zero point or the end 15 cuts it)
    off = (got.double() - src.double()).abs().view(M, K // group, group)
    room = 1.5 if zeros else 0.5 + 7 * 2.0 ** -8
    assert (off <= room * s[..., None].double() * (1 + 2.0 ** -20)).all()


def bound(x, w, add, swiglu, dtype):
    """(result, what a correct one may be off by), in 64 bits.  A sum of K products in float32, whatever its order
    and whether an addition rounds or cuts, is off by at most K 2^-23 of the sum of their magnitudes; the scale, the
    value of a weight and the addition of `add` are a rounding each."""
    x, w = x.double(), w.double()
    y, mag = x @ w.T, x.abs() @ w.abs().T
    if add is not None:
        y, mag = y + add.double(), mag + add.double().abs()
    tol = (w.shape[1] + 4) * 2.0 ** -23 * mag
    if not swiglu:
        return y, tol
    g, u, tg, tu = y[:, 0::2], y[:, 1::2], tol[:, 0::2], tol[:, 1::2]
    a = torch.nn.functional.silu(g)
    # |silu'| <= 1.1; the exponential, the quotient and the product are off by a few 2^-24 together
    t = 1.1 * tg * (u.abs() + tu) + a.abs() * tu + 2.0 ** -20 * (a * u).abs()
    return a * u, t + ((2.0 ** -8) * ((a * u).abs() + t) if dtype == "bf16" else 0)


def product(c, x, add=None, swiglu=False, ws=None):
    rows = x.shape[0]
    out = torch.full((rows, c.M // 2 if swiglu else c.M), 77.0, dtype=x.dtype if swiglu else torch.float32, device="cuda")
    c.w4.product(x, out, ws or W4Workspace(rows), add=add, swiglu=swiglu)
    return out


PRODUCTS = [
    # M, K, group, rows
    (1, 32, 32, 1), (2, 128, 128, 3), (127, 160, 32, 8), (128, 128, 64, 9), (130, 384, 128, 16), (256, 4096, 128, 1),
    (4096, 512, 64, 16), (640, 2560, 32, 17), (1000, 1184, 32, 33), (300, 192, 64, 64), (514, 1024, 128, 65),
    (1280, 640, 128, 100), (256, 2080, 32, 128), (20000, 256, 128, 5), (90, 12288, 128, 16), (2048, 320, 64, 24),
    (6144, 4096, 128, 2), (384, 8192, 64, 48),
]


@pytest.mark.parametrize("M, K, group, rows", PRODUCTS)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_product(M, K, group, rows, dtype):
    if dtype == "f32" and M * K > 1 << 22:
        M = (1 << 22) // K
    scales, zeros = [("bf16", False), ("f32", True), ("bf16", True), ("f32", False)][(M + K // 32 + rows) % 4]
    c = Codes(M, K, group, scales, zeros, seed=M)
    x = torch.empty(rows, K, dtype=TDT[dtype], device="cuda").normal_(generator=gen(2))
    got = product(c, x)
    want, tol = bound(x, c.w, None, False, dtype)
    assert ((got.double() - want).abs() <= tol).all()
    assert torch.equal(product(c, x), got)


@pytest.mark.parametrize("rows", [1, 7, 16, 40, 128])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M", [2, 126, 512, 1538])
def test_epilogues(rows, dtype, M):
    c = Codes(M, 640, 64, "bf16", True, seed=3)
    g = gen(5)
    x = torch.empty(rows, 640, dtype=TDT[dtype], device="cuda").normal_(0, 0.05, generator=g)
    add = torch.empty(rows, M, device="cuda").normal_(generator=g)
    for swiglu in (False, True):
        for a in (None, add):
            want, tol = bound(x, c.w, a, swiglu, dtype)
            assert ((product(c, x, a, swiglu).double() - want).abs() <= tol).all()
    # into the residual stream itself
    want, tol = bound(x, c.w, add, False, dtype)
    c.w4.product(x, add, W4Workspace(rows), add=add)
    assert ((add.double() - want).abs() <= tol).all()


@pytest.mark.parametrize("rows", [1, 5, 16, 70])
@pytest.mark.parametrize("pad, shift", [(8, 0), (1, 0), (0, 3), (9, 1), (2, 2)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_apart_and_off_alignment(rows, pad, shift, dtype):
    c = Codes(384, 320, 64, seed=6)
    buf = torch.full((rows * (320 + pad) + shift + 8,), float("nan"), dtype=TDT[dtype], device="cuda")
    x = buf[shift:shift + rows * (320 + pad)].view(rows, 320 + pad)[:, :320]
    x.copy_(torch.empty(rows, 320, device="cuda").normal_(generator=gen(7)))
    want, tol = bound(x, c.w, None, False, dtype)
    assert ((product(c, x).double() - want).abs() <= tol).all()


@pytest.mark.parametrize("rows, few", [(16, 1), (16, 8), (128, 1), (128, 17), (100, 16)])
def test_a_row_by_itself_and_among_others(rows, few):
    """A row's result depends on its own x and the matrix: any row, alone or in a block, has the same bits (here on both
    sides of 16 rows, as no row block of this matrix lies in runs of more than one block)."""
    c = Codes(700, 2176, 128, "f32", True, seed=8)
    x = torch.empty(rows, 2176, dtype=torch.bfloat16, device="cuda").normal_(generator=gen(9))
    whole = product(c, x)
    for at in (0, rows - few, (rows - few) // 2):
        assert torch.equal(product(c, x[at:at + few]), whole[at:at + few])


@pytest.mark.parametrize("M, K, group", [(5000, 2560, 128), (300, 12288, 64)])
@pytest.mark.parametrize("rows, few", [(16, 1), (16, 9), (128, 17), (65, 33)])
def test_a_row_of_a_large_matrix_among_others(M, K, group, rows, few):
    """Up to 16 rows, and from 17 on, the number of rows changes nothing in a row's bits, on matrices that many runs
    share as well."""
    c = Codes(M, K, group, "bf16", True, seed=15)
    x = torch.empty(rows, K, dtype=torch.bfloat16, device="cuda").normal_(generator=gen(16))
    whole = product(c, x)
    assert torch.equal(product(c, x[rows - few:]), whole[rows - few:])


@pytest.mark.parametrize("rows, pad", [(1, 0), (16, 0), (16, 1), (40, 0), (40, 1), (128, 0)])
def test_waits_that_run_out(rows, pad):
    """With a limit of 0 every wait has run out before it begins; with a few microseconds some do, while copies and
    products are in flight (rows of x on 16-byte boundaries come by other copies than rows off them).  The status says
    so, nothing but the result is written, and the next call after the status is right."""
    c = Codes(1500, 4096, 128, "bf16", True, seed=17)
    x = torch.empty(rows, 4096 + pad, dtype=torch.bfloat16, device="cuda").normal_(generator=gen(18))[:, :4096]
    ws = W4Workspace(rows)
    buf = torch.full((rows * c.M + 1024,), 77.0, device="cuda")
    out = buf[512:-512].view(rows, c.M)
    c.w4.product(x, out, ws)
    assert ws.status() == 0
    want = out.clone()
    ref, tol = bound(x, c.w, None, False, "bf16")
    assert ((want.double() - ref).abs() <= tol).all()
    try:
        for ns in (0, 0, 20000, 5000, 2000, 500):
            capi.dflash_debug_set_wait_limit(ns)
            out.fill_(77.0)
            c.w4.product(x, out, ws)
            status = ws.status()
            assert status in (0, capi.STATUS_TIMEOUT) and (ns or status)
            if not status:
                assert torch.equal(out, want)
            capi.dflash_debug_set_wait_limit(-1)
            c.w4.product(x, out, ws)
            assert ws.status() == 0 and torch.equal(out, want)
    finally:
        capi.dflash_debug_set_wait_limit(-1)
    assert (buf[:512] == 77.0).all() and (buf[-512:] == 77.0).all()


def test_values_that_are_not_finite_stay_in_their_row():
    c = Codes(300, 1152, 128, seed=10)
    for rows in (3, 16, 64):
        x = torch.empty(rows, 1152, dtype=torch.bfloat16, device="cuda").normal_(generator=gen(11))
        clean = product(c, x)
        bad = x.clone()
        bad[1, 5], bad[rows - 1, 1100] = float("nan"), float("nan")
        got = product(c, bad)
        assert torch.isnan(got[[1, rows - 1]]).all()
        keep = [i for i in range(rows) if i not in (1, rows - 1)]
        assert torch.equal(got[keep], clean[keep])


def test_one_workspace_for_many_matrices_and_a_graph():
    """Products of one stream one after another on one workspace, captured and replayed with other inputs."""
    ms = [Codes(M, K, g, seed=M) for M, K, g in ((256, 4096, 128), (6144, 256, 64), (130, 320, 32), (4096, 4096, 128))]
    ws = W4Workspace(16)
    xs = [torch.empty(16, c.K, dtype=torch.bfloat16, device="cuda").normal_(generator=gen(i)) for i, c in enumerate(ms)]
    outs = [torch.zeros(16, c.M, device="cuda") for c in ms]

    def calls():
        for c, x, o in zip(ms, xs, outs):
            c.w4.product(x, o, ws)

    calls()
    first = [o.clone() for o in outs]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        calls()
    torch.cuda.current_stream().wait_stream(s)
    for o in outs:
        o.zero_()
    graph.replay()
    assert all(torch.equal(o, f) for o, f in zip(outs, first))
    for x in xs:
        x.mul_(-2)
    graph.replay()
    graph.replay()
    assert all(torch.equal(o, -2 * f) for o, f in zip(outs, first))


def test_two_streams_with_a_workspace_each():
    c = Codes(4096, 2048, 64, seed=12)
    xs = [torch.empty(16, 2048, dtype=torch.bfloat16, device="cuda").normal_(generator=gen(20 + i)) for i in range(2)]
    want = [product(c, x) for x in xs]
    got = [torch.zeros_like(want[0]) for _ in range(2)]
    ws, st = [W4Workspace(16) for _ in range(2)], [torch.cuda.Stream() for _ in range(2)]
    for s in st:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(20):
        for i in range(2):
            with torch.cuda.stream(st[i]):
                c.w4.product(xs[i], got[i], ws[i])
    for s in st:
        torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_refusals():
    c = Codes(256, 256, 64, seed=13)
    x = torch.zeros(4, 256, dtype=torch.bfloat16, device="cuda")
    out, ws = torch.zeros(4, 256, device="cuda"), W4Workspace(4)

    def bad(kind, *a, **kw):
        with pytest.raises(kind):
            c.w4.product(*a, **kw)

    bad(ValueError, x[:, :128], out, ws)
    bad(ValueError, x.half(), out, ws)
    bad(ValueError, x.t().contiguous().t(), out, ws)
    bad(ValueError, x.cpu(), out, ws)
    bad(ValueError, x, out.bfloat16(), ws)
    bad(ValueError, x, out[:2], ws)
    bad(ValueError, x, torch.zeros(4, 128, device="cuda"), ws, swiglu=True)  # of x's type
    bad(ValueError, x, out, ws, add=torch.zeros(4, 255, device="cuda"))
    bad(ValueError, x, out, ws, add=out.bfloat16())
    bad(capi.DFlashError, torch.zeros(5, 256, dtype=torch.bfloat16, device="cuda"), torch.zeros(5, 256, device="cuda"), ws)
    bad(capi.DFlashError, x[:0], out[:0], ws)
    both = torch.zeros(5, 256, device="cuda")
    bad(capi.DFlashError, x, both[:4], ws, add=both[1:])
    odd = Codes(255, 256, 64, seed=14)
    with pytest.raises(capi.DFlashError):
        odd.w4.product(x, torch.zeros(4, 127, dtype=torch.bfloat16, device="cuda"), ws, swiglu=True)
    assert (out == 0).all()
    for kw in (dict(codes=torch.zeros(4, 64, dtype=torch.int8, device="cuda")), dict(scales=torch.zeros(3, 1, device="cuda")),
               dict(scales=torch.zeros(4, 1, dtype=torch.float16, device="cuda")),
               dict(zeros=torch.zeros(4, 2, dtype=torch.uint8, device="cuda"))):
        args = dict(codes=torch.zeros(4, 64, dtype=torch.uint8, device="cuda"), scales=torch.zeros(4, 1, device="cuda"))
        args.update(kw)
        with pytest.raises(ValueError):
            W4Linear.from_codes(**args)
    with pytest.raises(capi.DFlashError):
        W4Linear(64, 100, 32)
    with pytest.raises(ValueError):
        W4Linear(64, 128, 128, packed=torch.zeros(100, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        W4Linear.from_weight(torch.zeros(4, 128, dtype=torch.float16, device="cuda"))
