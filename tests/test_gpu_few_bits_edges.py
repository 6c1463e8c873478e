"""8-bit pages and 4-bit weights where their ranges end: value rows of zero before others, slots that hold anything,
scales far from one another, matrices whose range float32 cannot hold; against 64-bit arithmetic."""
import math

import pytest

torch = pytest.importorskip("torch")

from block_diffusion_speculative_target_gb300 import capi  # noqa: E402
from block_diffusion_speculative_target_gb300.engine import W4Linear, W4Workspace  # noqa: E402
from test_gpu_paged import CASES, HEADS, TDT, visible  # noqa: E402
from test_gpu_paged_q8 import SHARED, Batch8, attend, check, reference, untouched  # noqa: E402

pytestmark = pytest.mark.gpu

# What a weight, with its value's scale, is off by when it enters the product with the values in bf16 models.
WEIGHT = 2.0 ** -22


def near(x, q, got, causal=True, window=0, sinks=0, weight=WEIGHT):
    """Each live row against 64 bits.  A rounding of float32 is u = 2^-24.  A score is a sum of hd products, which may
    be cut instead of rounded (2 u each), times two scales: a weight is off by (2 hd + 4) u times the sum of the
    |q k|, and by 4 u of the exponential, relative, in the numerator and in the sum that divides it; the two sums
    over the keys by 2 u a key.  bf16: the weights with the values' scales are off by `weight` of themselves, or, below
    half's normal numbers, by 2^-25 under a factor that brings the row's largest to 2^7 at least: 2^-32 of the largest
    weight times value, a key; and the result is rounded once, 2^-8 of itself."""
    G, u = x.nq // x.nkv, 2.0 ** -24
    assert torch.isfinite(got).all(), "a value is not finite"
    for b, (P, r) in enumerate(zip(x.lens, x.rows)):
        r = min(max(r, 0), x.n)
        if not r:
            continue
        k, v = x.keys(b, P + r)
        for i in range(r):
            see = visible(P, r, i, causal, window, sinks, P + r)
            kk, vv = k[:, see], v[:, see]
            a = q[b, i].double().view(x.nkv, G, x.hd)
            p = torch.softmax(a @ kk.transpose(1, 2) / math.sqrt(x.hd), -1)
            want, mag = p @ vv, p @ vv.abs()
            dots = (a.abs() @ kk.abs().transpose(1, 2)).amax(-1, keepdim=True) / math.sqrt(x.hd)
            keys = kk.shape[1]
            tol = mag * u * (2 * ((2 * x.hd + 4) * dots + 4) + 4 * keys + 16)
            if x.dtype == "bf16":
                top = (p * vv.abs().amax(-1)[:, None]).amax(-1, keepdim=True)
                tol = tol + weight * mag + 2.0 ** -32 * keys * top
                tol = tol + 2.0 ** -8 * (want.abs() + tol) + 2.0 ** -134  # (bf16's least step is 2^-133)
            off = (got[b, i].double().view(x.nkv, G, x.hd) - want).abs() - tol
            assert float(off.max()) <= 0, f"row {i} of sequence {b}: {float(off.max()):.3e} more than its bound"


def lift(x, q, keys, by):
    """Raises the scores of some positions of every sequence by `by` units of log2, whatever the other entries are: the
    first entry of keys is 0 but there, and that of every query the same."""
    x.pool["k"][..., 0] = 128
    at = float(torch.tensor(by / (0.01 * 127 * 1.4426950408889634 / math.sqrt(x.hd))).to(x.dt))
    for b, P in enumerate(x.lens):
        p = torch.tensor([y for y in keys if y < P], dtype=torch.int64, device="cuda")
        page = x.table[b].long()[p // x.ps]
        x.pool["k"][0, page, :, p % x.ps, 0] = 255 if by > 0 else 1
        x.pool["k_scale"][0, page, :, p % x.ps] = 0.01
    q[..., 0] = abs(at)
    return q


def set_value_scale(x, keys, to):
    for b, P in enumerate(x.lens):
        p = torch.tensor([y for y in keys if y < P + x.n], dtype=torch.int64, device="cuda")
        x.pool["v_scale"][0, x.table[b].long()[p // x.ps], :, p % x.ps] = to


# ------------------------------------------------------------------ slots that hold anything, scales far apart


@pytest.mark.parametrize("fill", [3e38, -1e36])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("c", CASES, ids=[f"{c[0]}-p{c[1]}-n{c[3]}-{max(c[2])}-{'c' if c[5] else 'f'}-w{c[6]}-s{c[7]}"
                                          for c in CASES])
def test_slots_that_hold_no_position(c, dtype, fill):
    """Their scales are whatever the memory held: as large as float32 goes."""
    heads, ps, lens, n, rows, causal, window, sinks = c
    x = Batch8(dtype, *HEADS[heads], ps, lens, n, rows, fill=fill, extra_cols=3)
    q = x.query()
    kw = dict(causal=causal, window=window, sinks=sinks)
    out = attend(x, q, **kw)
    assert x.cache.status() == 0
    untouched(x, out)
    check(x, out, reference(x, q, **kw), "attention")


@pytest.mark.parametrize("fill", [3e38, -1e36])
@pytest.mark.parametrize("c", SHARED, ids=[f"{c[0]}-p{c[1]}-{c[2]}-n{c[4]}-w{c[7]}" for c in SHARED])
def test_slots_that_hold_no_position_behind_a_shared_prefix(c, fill):
    heads, ps, shared, behind, n, rows, causal, window, sinks = c
    x = Batch8("bf16", *HEADS[heads], ps, [shared + y for y in behind], n, rows, fill=fill, shared=shared)
    q = x.query()
    kw = dict(causal=causal, window=window, sinks=sinks)
    out = attend(x, q, shared=shared, **kw)
    assert x.cache.status() == 0
    untouched(x, out)
    check(x, out, reference(x, q, **kw), "shared")


@pytest.mark.parametrize("n", [1, 4, 8, 40])
@pytest.mark.parametrize("at", [5, 40, 299])
def test_a_large_value_with_next_to_no_weight(n, at):
    """Values of 1e-28 and one of 1e12 whose score lies 200 log2 units below the others'."""
    x = Batch8("bf16", 8, 2, 128, 32, [300, 90], n)
    x.pool["v_scale"] *= 1e-30 / 0.03
    set_value_scale(x, [at], 1e10)
    q = lift(x, x.query(), [at], -200)
    near(x, q, attend(x, q))


@pytest.mark.parametrize("n", [1, 8, 40])
def test_large_values_under_sharp_scores(n):
    """Value rows with entries up to 2^100, scores that rise and fall by tens of log2 units from key to key."""
    x = Batch8("bf16", 8, 2, 128, 32, [400, 90], n)
    x.pool["v_scale"] *= 2.0 ** 93 / 0.03
    q = x.query(scale=20.0)
    near(x, q, attend(x, q))


# ------------------------------------------------------------------ value rows of zero


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n", [1, 4, 8, 40])
@pytest.mark.parametrize("zeros, value, up, kw", [
    (16, 1e-3, 12, {}), (64, 1e-5, 12, {}), (130, 1e-6, 0, {}), (130, 0.02, 20, {}), (1, 0.02, 20, {}), (700, 1e-9, 3, {}),
    (1, 0.02, 20, dict(window=900, sinks=1)), (1, 1e-6, 0, dict(window=300, sinks=1)),
    (64, 1e-5, 6, dict(causal=False, window=500, sinks=64)), (2000, 0.02, 0, {})])
def test_values_of_zero_before_others(n, zeros, value, up, kw, dtype):
    """The first rows of a sequence hold values of zero (their scale is 0), the first key draws the most attention: the
    later weights keep their bits, whatever the scales of their values are."""
    x = Batch8(dtype, 8, 2, 128, 32, [2000, 300], n)
    x.pool["v_scale"] *= value / 0.03
    set_value_scale(x, range(zeros), 0.0)
    q = lift(x, x.query(), [0], up)
    near(x, q, attend(x, q, **kw), **kw)


@pytest.mark.parametrize("n", [1, 8, 40])
@pytest.mark.parametrize("hd", [64, 128])
def test_values_of_zero_behind_a_shared_prefix(n, hd):
    """Pieces begin anywhere: zeros at the start of the prefix, and of the sequences' own keys."""
    x = Batch8("bf16", 4, 2, hd, 16, [1000, 1300, 1001], n, shared=999)
    x.pool["v_scale"] *= 1e-6 / 0.03
    set_value_scale(x, range(200), 0.0)
    set_value_scale(x, range(960, 1050), 0.0)
    q = x.query()
    near(x, q, attend(x, q, shared=999))


@pytest.mark.parametrize("n", [1, 8, 40])
def test_scores_that_rise_after_tiny_values(n):
    """Values of 1e-28 first, then, 24 log2 units above their scores, values of zero: the sum of weights times the factor
    that brought the first ones into range is past float32."""
    x = Batch8("bf16", 8, 2, 128, 32, [80], n, fill=0.0)
    x.pool["v_scale"] *= 1e-30 / 0.03
    keys = range(64, 80 + n)
    set_value_scale(x, keys, 0.0)
    q = lift(x, x.query(), keys, 24)
    near(x, q, attend(x, q))


# ------------------------------------------------------------------ 4-bit weights


@pytest.mark.parametrize("scales", ["bf16", "f32"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("zeros", [False, True])
def test_quantize_ranges_past_float32(dtype, scales, zeros):
    """Entries of 2e38 of both signs: their range is past float32, a fifteenth of it is not.  The stated rule, value for
    value, with the range taken in 64 bits."""
    M, K, group = 130, 256, 64
    g = torch.Generator(device="cuda").manual_seed(31)
    src = ((torch.rand(M, K, dtype=torch.float64, device="cuda", generator=g) - 0.5) * 4e38).to(TDT[dtype])
    src[0, 0], src[0, 1] = 2e38, -2e38
    src[1] = src[1].abs()
    got = W4Linear.from_weight(src, group, TDT[scales], zeros).weight()
    x = src.double().view(M, K // group, group)
    hi, lo = x.amax(-1).clamp(min=0), x.amin(-1).clamp(max=0)
    s = ((hi - lo) / 15 if zeros else torch.maximum(hi, -lo) / 7).float().to(TDT[scales]).float()
    # (a quotient in 64 bits, rounded, is float32's own)
    z = torch.round((-lo / s.double()).float()).clamp(0, 15) if zeros else torch.full_like(s, 8.0)
    code = (torch.round((x / s.double()[..., None]).float()) + z[..., None]).clamp(0, 15)
    assert torch.isfinite(got).all()
    assert torch.equal(got, ((code - z[..., None]) * s[..., None]).view(M, K))


@pytest.mark.parametrize("rows", [8, 16, 17, 32, 64, 128])
def test_workspace_holds_no_more_than_calls_use(rows):
    """Partial sums: at most two pieces of 128 x rows floats a run; up to 16 rows a product takes four runs a
    multiprocessor, more rows one.  Products at that many rows, and at 16, fit it side by side with its neighbours."""
    torch.cuda.synchronize()
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    free = torch.cuda.mem_get_info()[0]
    many = [W4Workspace(rows) for _ in range(4)]
    used = (free - torch.cuda.mem_get_info()[0]) / 4
    padded = next(r for r in (8, 16, 32, 64, 128) if r >= rows)
    assert used <= sms * 2 * 128 * max(4 * min(padded, 16), padded) * 4 + (6 << 20)  # (and what an allocation rounds up to)
    g = torch.Generator(device="cuda").manual_seed(32)
    w = W4Linear.from_weight(torch.empty(20000, 1024, device="cuda").normal_(generator=g))
    dense = w.weight().double()
    for r in sorted({rows, min(rows, 16), min(rows, 9)}):
        x = torch.empty(r, 1024, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
        out = [torch.zeros(r, 20000, device="cuda") for _ in many]
        for o, ws in zip(out, many):
            w.product(x, o, ws)
        want, mag = x.double() @ dense.T, x.double().abs() @ dense.abs().T
        for o, ws in zip(out, many):
            assert ((o.double() - want).abs() <= (1024 + 4) * 2.0 ** -23 * mag).all() and ws.status() == 0


# ------------------------------------------------------------------ the bits of a weight


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("n", [1, 2, 4, 8, 40])
@pytest.mark.parametrize("shared", [None, 64])
def test_weights_keep_their_bits(n, hd, shared):
    """Queries of zero, so that all keys weigh the same, and values that cancel but for 2^-12: the even positions hold
    +127 c in every entry, the odd ones -127 c (1 + 2^-12).  A weight of one half would round the difference away."""
    x = Batch8("bf16", 8, 2, hd, 16, [59, 64] if shared is None else [64, 70], n, shared=shared or 0)
    for b, P in enumerate(x.lens):
        p = torch.arange(P + n, device="cuda")
        page = x.table[b].long()[p // 16]
        odd = (p % 2).bool()
        x.pool["v"][0, page, :, p % 16] = torch.where(odd, 1, 255).to(torch.uint8)[:, None, None]
        x.pool["v_scale"][0, page, :, p % 16] = torch.where(odd, 0.01 * (1 + 2.0 ** -12), 0.01)[:, None]
    q = torch.zeros(2, n, 8, hd, dtype=x.dt, device="cuda")
    near(x, q, attend(x, q, shared=shared))


@pytest.mark.parametrize("n", [1, 2, 4, 8, 40])
def test_an_infinite_value(n):
    """A pool that another program filled may hold a value scale of Inf: the rows that see it are infinite, others are
    what they were."""
    x = Batch8("bf16", 8, 2, 128, 32, [100, 90], n)
    q = x.query()
    want = attend(x, q)
    at = 100 + n // 2
    page, slot = int(x.table[0, at // 32]), at % 32
    x.pool["v"][0, page, :, slot] = torch.where(torch.arange(128, device="cuda") % 2 == 0, 200, 3).to(torch.uint8)
    x.pool["v_scale"][0, page, :, slot] = math.inf
    got = attend(x, q)
    assert (got[0, n // 2:, :, 0::2] == math.inf).all() and (got[0, n // 2:, :, 1::2] == -math.inf).all()
    assert torch.equal(got[0, :n // 2], want[0, :n // 2]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("rows", [1, 16, 40])
def test_products_directly_behind_packing(rows):
    """A buffer filled again and again, each time with other codes, and a product at once behind each: also captured."""
    g = torch.Generator(device="cuda").manual_seed(33)
    M, K = 3000, 1024
    codes = [torch.randint(0, 256, (M, K // 2), dtype=torch.uint8, device="cuda", generator=g) for _ in range(2)]
    dense = [torch.empty(M, K, device="cuda").normal_(generator=g) for _ in range(2)]
    scales = torch.ones(M, K // 128, device="cuda")
    x = torch.empty(rows, K, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    ws = W4Workspace(rows)
    want = []
    for w in [W4Linear.from_codes(c, scales) for c in codes] + [W4Linear.from_weight(d, scale_dtype=torch.float32) for d in dense]:
        out = torch.zeros(rows, M, device="cuda")
        w.product(x, out, ws)
        torch.cuda.synchronize()
        want.append(out)
    w = W4Linear(M, K, scale_dtype=torch.float32)
    got = [torch.zeros_like(o) for o in want]

    def calls():
        for i in (0, 2, 1, 3):
            s = torch.cuda.current_stream()
            if i < 2:
                capi.dflash_w4_pack(w._c, codes[i], scales, None, s)
            else:
                capi.dflash_w4_quantize(w._c, capi.F32, dense[i - 2], K, s)
            w.product(x, got[i], ws)

    for _ in range(5):
        calls()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        calls()
    torch.cuda.current_stream().wait_stream(side)
    for o in got:
        o.zero_()
    for _ in range(5):
        graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows", [1, 8, 16, 40])
def test_gates_far_below_zero(rows, dtype):
    """Gates down to -88.5, where e^-g is still a float32, times values of 1e30.  Gate and value are exact here; the
    exponential's argument is rounded (2^-24 of 128, twice that of the result), the rest is a few roundings, and the
    result is rounded once more."""
    code = torch.full((2, 32), 8, dtype=torch.uint8, device="cuda")
    code[0, 0] = code[1, 1] = 9
    w = W4Linear.from_codes(code[:, 0::2] | code[:, 1::2] << 4, torch.ones(2, 1, device="cuda"))
    gates = [-88.5, -88.0, -87.5, -87.0, -60.0, -1.0, 0.0, 50.0]
    x = torch.zeros(rows, 32, dtype=TDT[dtype], device="cuda")
    x[:, 0] = torch.tensor([gates[i % len(gates)] for i in range(rows)])
    x[:, 1] = torch.tensor([(-1) ** i * 1e30 for i in range(rows)])
    out = torch.zeros(rows, 1, dtype=TDT[dtype], device="cuda")
    w.product(x, out, W4Workspace(rows), swiglu=True)
    g, u = x[:, 0].double(), x[:, 1].double()
    want = g / (1 + torch.exp(-g)) * u
    tol = (2.0 ** -15 + (2.0 ** -8 if dtype == "bf16" else 0)) * want.abs()
    assert ((out[:, 0].double() - want).abs() <= tol).all()


@pytest.mark.parametrize("M, K, group", [(1, 32, 32), (130, 32, 32), (257, 64, 64), (40, 96, 32), (2, 128, 128), (300, 224, 32)])
@pytest.mark.parametrize("rows", [1, 16, 17, 33, 65, 128])
def test_matrices_narrower_than_a_block(M, K, group, rows):
    """Fewer columns than a block of 128, or than half of one."""
    g = torch.Generator(device="cuda").manual_seed(34)
    w = W4Linear.from_weight(torch.empty(M, K, device="cuda").normal_(generator=g), group, zeros=True)
    x = torch.empty(rows, K, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    out = torch.full((rows + 2, M), 77.0, device="cuda")
    ws = W4Workspace(rows)
    w.product(x, out[1:-1], ws)
    dense = w.weight().double()
    want, mag = x.double() @ dense.T, x.double().abs() @ dense.abs().T
    assert ws.status() == 0 and (out[0] == 77.0).all() and (out[-1] == 77.0).all()
    assert ((out[1:-1].double() - want).abs() <= (K + 4) * 2.0 ** -23 * mag).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n", [1, 4, 40])
@pytest.mark.parametrize("shared", [None, 64])
def test_a_batch_without_rows(n, shared, dtype):
    """No sequence has a row: nothing is written, the status stays clear, and the next call is right."""
    x = Batch8(dtype, 8, 2, 128, 32, [200, 70], n, shared=shared or 0)
    q = x.query()
    want = attend(x, q, shared=shared)
    x.n_rows = torch.zeros(2, dtype=torch.int32, device="cuda")
    assert (attend(x, q, shared=shared) == 77.0).all()
    x.n_rows.fill_(-3)
    assert (attend(x, q, shared=shared) == 77.0).all()
    x.n_rows = None
    assert torch.equal(attend(x, q, shared=shared), want) and x.cache.status() == 0
