"""8-bit pages on the GPU: the append that quantises, rows read back, and attention over codes and scales, against
64-bit implementations written here; a decoder layer of 4-bit products over such pages."""
import math
from types import SimpleNamespace

import pytest

torch = pytest.importorskip("torch")

from block_diffusion_speculative_target_gb300 import capi  # noqa: E402
from block_diffusion_speculative_target_gb300.engine import PagedCache, W4Linear, W4Workspace  # noqa: E402
from test_gpu_paged import APPENDS, CASES, HEADS, MANY, TDT, THETA, i32, rotated, shape_of, visible  # noqa: E402

pytestmark = pytest.mark.gpu


class Batch8:
    """A pool of 8-bit pages scattered over sequences, and a PagedCache over it."""

    def __init__(self, dtype, nq, nkv, hd, ps, lens, n, rows=None, seed=0, layers=1, fill=None, spare=2, extra_cols=0,
                 shared=0, max_pos=None):
        self.g = torch.Generator(device="cuda").manual_seed(2000 + seed)
        self.dtype, self.dt, self.nq, self.nkv, self.hd, self.ps, self.n = dtype, TDT[dtype], nq, nkv, hd, ps, n
        self.lens, self.rows = list(lens), [n] * len(lens) if rows is None else list(rows)
        B = len(lens)
        self.cols = max(-(-(x + n) // ps) for x in lens) + extra_cols
        common = shared // ps
        own = [-(-(x + n) // ps) - common for x in lens]
        n_pages = common + sum(own) + spare
        perm = torch.randperm(n_pages, generator=self.g, device="cuda").tolist()
        table = [[-7] * self.cols for _ in range(B)]
        at = common
        for b in range(B):
            for c in range(own[b] + common):
                table[b][c] = perm[c] if c < common else perm[at + c - common]
            at += own[b]
        self.table, self.len = i32(table), i32(self.lens)
        self.n_rows = None if rows is None else i32(rows)
        dims = (layers, n_pages, nkv, ps, hd)
        self.pool = {}
        for x in ("k", "v"):
            self.pool[x] = torch.randint(1, 256, dims, dtype=torch.uint8, device="cuda", generator=self.g)
            # scales over two orders of magnitude
            s = torch.empty(dims[:4], device="cuda").uniform_(math.log(0.001), math.log(0.03), generator=self.g).exp_()
            self.pool[x + "_scale"] = s
        if fill is not None:  # the scales of slots that hold no position
            live = torch.zeros(n_pages * ps, dtype=torch.bool, device="cuda")
            for b in range(B):
                p = torch.arange(self.lens[b] + min(max(self.rows[b], 0), n), device="cuda")
                live[self.table[b].long()[p // ps] * ps + p % ps] = True
            dead = ~live.view(1, n_pages, 1, ps).expand(dims[:4])
            for x in ("k_scale", "v_scale"):
                self.pool[x][dead] = fill
        if shared % ps:
            at, upto = shared // ps, shared % ps
            for t in self.pool.values():
                t[:, self.table[:, at].long(), :, :upto] = t[:, self.table[0, at].long()][:, None, :, :upto]
        self.cache = PagedCache(shape_of(nq, nkv, hd), dtype, n_pages, ps, max_pos or self.cols * ps, B * n, max_batch=B,
                                n_layers=layers, kv_format="q8", **self.pool)
        assert all(getattr(self.cache, x) is t for x, t in self.pool.items())

    def normal(self, *dims, scale=1.0, dtype=None):
        return torch.empty(dims, dtype=dtype or self.dt, device="cuda").normal_(0, scale, generator=self.g)

    def query(self, scale=1.5):
        return self.normal(len(self.lens), self.n, self.nq, self.hd, scale=scale)

    def values(self, x, layer, page, slot):
        """Entries of the rows at (page, slot) in 64 bits: [..., nkv, hd]."""
        return (self.pool[x][layer][page, :, slot].double() - 128) * self.pool[x + "_scale"][layer][page, :, slot].double()[..., None]

    def keys(self, b, count, layer=0):
        p = torch.arange(count, device="cuda")
        page = self.table[b].long()[p // self.ps]
        return [self.values(x, layer, page, p % self.ps).transpose(0, 1) for x in ("k", "v")]


def reference(x, q, causal=True, window=0, sinks=0, layer=0):
    """(result, attention of |values|, largest sum of |q k| scale, keys, largest |value|) in 64 bits."""
    G = x.nq // x.nkv
    out = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
    mag, dots, most, top = torch.zeros_like(out), 0.0, 1, 0.0
    for b, (P, r) in enumerate(zip(x.lens, x.rows)):
        r = min(max(r, 0), x.n)
        if not r:
            continue
        k, v = x.keys(b, P + r, layer)
        for i in range(r):
            see = visible(P, r, i, causal, window, sinks, P + r)
            kk, vv = k[:, see], v[:, see]
            a = q[b, i].double().view(x.nkv, G, x.hd)
            p = torch.softmax(a @ kk.transpose(1, 2) / math.sqrt(x.hd), -1)
            out[b, i] = (p @ vv).reshape(x.nq, x.hd)
            mag[b, i] = (p @ vv.abs()).reshape(x.nq, x.hd)
            dots = max(dots, float((a.abs() @ kk.abs().transpose(1, 2)).max()) / math.sqrt(x.hd))
            most, top = max(most, kk.shape[1]), max(top, float(vv.abs().max()))
    return out, mag, dots, most, top


def check(x, got, want, what=""):
    """As for the other pages, u = 2^-24 a rounding of float32: a score is a sum of hd products, which may be cut
    instead of rounded (2 u each), times two scales; so a weight is off by (2 hd + 4) u dots and the exponential's
    4 u, relative, the weights' and the outputs' sums over `most` keys by 2 u a key.  A bf16 result is rounded once,
    2^-8 of itself.  Before it the weights, with the values' scales, are rounded to half: 2^-11 of the attention of
    |values|, and, as weights are kept so that a row's reference is at least 2^7, below half's normal numbers
    2^-25 2^-7 of the largest value for each key."""
    ref, mag, dots, most, top = want
    u = 2.0 ** -24
    b = mag * u * (2 * ((2 * x.hd + 4) * dots + 4) + 4 * most + 16)
    if x.dtype == "bf16":
        b = b + 2.0 ** -11 * mag + 2.0 ** -31 * most * top
        b = b + 2.0 ** -8 * (ref.abs() + b)
    d = (got.double() - ref).abs() - b
    assert torch.isfinite(got).all(), f"{what}: a value is not finite"
    for i, r in enumerate(x.rows):
        r = min(max(r, 0), x.n)
        assert float(d[i, :r].max() if r else 0) <= 0, f"{what}: sequence {i} off by {float(d[i, :r].max()):.3e} more than its bound"


def attend(x, q, shared=None, **kw):
    out = torch.full_like(q, 77.0)
    x.cache.attention(0, q, x.table, x.len, out, n_rows=x.n_rows, shared_len=None if shared is None else i32([shared]), **kw)
    return out


def untouched(x, out):
    for b, r in enumerate(x.rows):
        assert (out[b, min(max(r, 0), x.n):] == 77.0).all(), f"padding rows of sequence {b} were written"


# ------------------------------------------------------------------ append


@pytest.mark.parametrize("c", APPENDS + MANY, ids=[f"{c[0]}-{c[1]}-{c[2]}x{c[3]}x{c[4]}-p{c[5]}-n{c[7]}" for c in APPENDS + MANY])
def test_append(c):
    dtype, src, nq, nkv, hd, ps, lens, n, rows, queries, pad, shift = c
    x = Batch8(dtype, nq, nkv, hd, ps, lens, n, rows, layers=2 if n < 1000 else 1)
    layer = 1 if n < 1000 else 0
    heads, B = (nq if queries else 0) + 2 * nkv, len(lens)
    width = heads * hd
    buf = x.normal(B * n * (width + pad) + shift, dtype=TDT[src])
    qkv = buf[shift:].view(B * n, width + pad)[:, :width]
    qkv[0, -hd:] = 0.0  # a row of zeros
    before = {k: t.clone() for k, t in x.pool.items()}
    q_out = torch.full((B, n, nq, hd), 77.0, dtype=x.dt, device="cuda") if queries else None
    x.cache.append(layer, qkv, x.table, x.len, n, q_out=q_out, n_rows=x.n_rows)
    assert x.cache.status() == 0
    z = qkv.double().view(B, n, heads, hd)
    j = torch.arange(n, device="cuda")
    pos = x.len[:, None].long() + j
    live = j < (torch.full((B,), n, device="cuda") if rows is None else x.n_rows)[:, None]
    turn = rotated(z[:, :, :heads - nkv], pos, hd)
    # cos and sin are off by 2^-24 of 1, each product and the sum by a rounding: 4 2^-24 of |x_lo| + |x_hi|
    size = z.abs().view(B, n, heads, 2, hd // 2).sum(3, keepdim=True).expand(B, n, heads, 2, hd // 2).reshape(B, n, heads, hd)
    tol = 4 * 2.0 ** -24 * size[:, :, :heads - nkv]
    if queries:
        half = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -24
        d = (q_out.double() - turn[:, :, :nq]).abs()
        assert (d <= tol[:, :, :nq] + half * turn[:, :, :nq].abs())[live].all()
        assert (q_out[~live] == 77.0).all()
    b, r = live.nonzero(as_tuple=True)
    page, slot = x.table[b, pos[b, r] // ps].long(), pos[b, r] % ps
    code = {k: x.pool[k][layer][page, :, slot].float() - 128 for k in ("k", "v")}
    scale = {k: x.pool[k + "_scale"][layer][page, :, slot] for k in ("k", "v")}
    # values: the rule, value for value
    v = z[b, r, heads - nkv:].float()
    s = (v.abs().amax(-1).double() / 127).float()  # (float32's quotient)
    assert torch.equal(scale["v"], s)
    assert torch.equal(code["v"], torch.where(s[..., None] > 0, torch.round(v / s[..., None]), torch.zeros_like(v)))
    # keys: the scale within the rotation's error and two roundings, an entry within half a step of the rotated row
    k, t = turn[b, r, heads - 2 * nkv:], tol[b, r, heads - 2 * nkv:]
    s = k.abs().amax(-1)
    assert ((scale["k"].double() * 127 - s).abs() <= t.amax(-1) + 2.0 ** -23 * s).all()
    off = (code["k"].double() * scale["k"].double()[..., None] - k).abs()
    assert (off <= t + (0.5 + 2.0 ** -15) * scale["k"].double()[..., None]).all()
    assert (code["k"].abs() <= 127).all()
    # nothing else is written
    rest = torch.ones(x.pool["k"].shape[1], ps, dtype=torch.bool, device="cuda")
    rest[page, slot] = False
    for name, now in x.pool.items():
        assert torch.equal(now[layer].transpose(1, 2)[rest], before[name][layer].transpose(1, 2)[rest]), name
        if layer:
            assert torch.equal(now[0], before[name][0]), name


@pytest.mark.parametrize("hd", [64, 128])
def test_append_of_rows_that_are_not_finite(hd):
    """Such a row reads back as NaN; its neighbours are as they would be without it."""
    x = Batch8("bf16", 4, 2, hd, 16, [5], 8)
    qkv = x.normal(8, 8 * hd, dtype=torch.float32)
    clean = qkv.clone()
    for row, at in ((1, 6 * hd + 3), (2, 7 * hd - 1), (3, 4 * hd), (5, 8 * hd - 1)):
        qkv[row, at] = [float("nan"), float("inf"), -float("inf"), float("nan")][row % 4]
    got = []
    for rows in (clean, qkv):
        x.cache.append(0, rows, x.table, x.len, 8, q_out=torch.zeros(1, 8, 4, hd, dtype=x.dt, device="cuda"))
        k, v = (torch.zeros(1, 2, 8, hd, device="cuda") for _ in range(2))
        x.cache.read(0, x.table, x.len, k, v)
        got.append(torch.cat([k, v], 1))
    assert x.cache.status() == 0 and torch.isfinite(got[0]).all()
    bad = torch.zeros(4, 8, dtype=torch.bool, device="cuda")  # heads k0 k1 v0 v1
    bad[2, 1] = bad[2, 2] = bad[0, 3] = bad[3, 5] = True
    assert torch.isnan(got[1][0][bad]).all()
    assert torch.equal(got[1][0][~bad], got[0][0][~bad])


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_append_rounds_ties_to_even(hd, dtype):
    """Quotients at a tie and a step of float32 to its sides, at scales of powers of two and others, down to those below
    the normal numbers: the codes of the stated rule, value for value (values are not rotated, scales are seen)."""
    tops = [127.0, 127.0 * 2.0 ** -100, 127.0 * 2.0 ** 100, 127.0 * 2.0 ** -135, 2.0 ** -140, 3.7, 1e-20, 1e20, 0.0]
    n = 3 * len(tops)
    x = Batch8(dtype, 1, 1, hd, 32, [0], n)
    half = torch.arange(hd, device="cuda") * 2 - (hd - 1)  # odd numbers
    half = half.clamp(-253, 253).double() / 2  # ties: j + 1 / 2
    rows = []
    for top in tops:
        s = float(torch.tensor(top, dtype=torch.float32).double().div(127).float())
        v = (half * s).float()
        up, down = torch.full_like(v, math.inf), torch.full_like(v, -math.inf)
        for y in (v, torch.nextafter(v, up), torch.nextafter(v, down)):
            y = y.clamp(-top, top)
            y[0] = top
            rows.append(y)
    v = torch.stack(rows)
    qkv = torch.zeros(n, 3 * hd, device="cuda")
    qkv[:, 2 * hd:] = v
    x.cache.append(0, qkv, x.table, x.len, n, q_out=torch.zeros(1, n, 1, hd, dtype=x.dt, device="cuda"))
    assert x.cache.status() == 0
    p = torch.arange(n, device="cuda")
    page = x.table[0].long()[p // 32]
    got, gs = x.pool["v"][0][page, 0, p % 32], x.pool["v_scale"][0][page, 0, p % 32]
    s = (v.abs().amax(1).double() / 127).float()
    assert torch.equal(gs, s)
    # (the quotient in 64 bits, rounded, is float32's own; a row of zeros holds 128)
    q = (v.double() / torch.where(s > 0, s, torch.ones_like(s)).double()[:, None]).float()
    assert torch.equal(got.double(), torch.round(q).clamp(-127, 127).double() + 128)


def test_append_reports_capacity_and_bad_pages():
    x = Batch8("bf16", 4, 1, 128, 16, [30, 5], 4)
    qkv = x.normal(8, 6 * 128)
    before = {k: t.clone() for k, t in x.pool.items()}
    q = torch.zeros(2, 4, 4, 128, dtype=x.dt, device="cuda")
    x.cache.append(0, qkv, x.table, i32([x.cols * 16 - 1, 5]), 4, q_out=q)
    assert x.cache.status() == capi.STATUS_CAPACITY
    assert (q[0, 1:] == 0).all() and (q[1].abs().sum(-1) > 0).all()
    for k, t in x.pool.items():
        t.copy_(before[k])
    t = x.table.clone()
    t[0, 1], t[1, 0] = 10 ** 6, -1
    x.cache.append(0, qkv, t, x.len, 4, q_out=q)  # sequence 0: positions 30, 31 in page 1 (bad), 32, 33 in page 2
    assert x.cache.status() == capi.STATUS_BOUNDS
    for k in ("v", "v_scale"):
        assert (x.pool[k] != before[k]).flatten(2).any(2).sum() == 1, k


# ------------------------------------------------------------------ read


READS = [
    # dtype, nq, nkv, hd, ps, start, n, rows
    ("bf16", 4, 1, 128, 16, [0], 1, None), ("bf16", 32, 8, 128, 64, [0, 63, 1000], 130, [130, 0, 65]),
    ("bf16", 12, 4, 64, 32, [17, 5], 63, None), ("f32", 4, 4, 64, 128, [200, 0, 1], 64, [64, -3, 9]),
    ("f32", 8, 2, 128, 16, [33], 4000, None),
]


@pytest.mark.parametrize("fmt", ["q8", "model"])
@pytest.mark.parametrize("out", ["f32", "model"])
@pytest.mark.parametrize("c", READS, ids=[f"{c[0]}-{c[2]}x{c[3]}-p{c[4]}-n{c[6]}" for c in READS])
def test_read(c, out, fmt):
    dtype, nq, nkv, hd, ps, start, n, rows = c
    x = Batch8(dtype, nq, nkv, hd, ps, start, n, rows, layers=2, fill=float("nan"))
    cache = x.cache
    if fmt == "model":
        dims = x.pool["k"].shape
        pools = [x.normal(*dims) for _ in range(2)]
        cache = PagedCache(shape_of(nq, nkv, hd), dtype, dims[1], ps, x.cols * ps, len(start), n_layers=2, k=pools[0],
                           v=pools[1])
    odt = x.dt if out == "model" else torch.float32
    B = len(start)
    got = [torch.full((B, nkv, n, hd), 77.0, dtype=odt, device="cuda") for _ in range(2)]
    cache.read(1, x.table, x.len, *got, n_rows=x.n_rows)
    assert cache.status() == 0
    for b in range(B):
        r = min(max(x.rows[b], 0), n)
        p = start[b] + torch.arange(r, device="cuda")
        page = x.table[b].long()[p // ps]
        for i, name in enumerate(("k", "v")):
            want = x.values(name, 1, page, p % ps).float() if fmt == "q8" else pools[i][1][page, :, p % ps]
            assert torch.equal(got[i][b, :, :r], want.to(odt).transpose(0, 1))
            assert (got[i][b, :, r:] == 77.0).all()
    one = torch.full_like(got[0], 77.0)
    cache.read(1, x.table, x.len, v_out=one, n_rows=x.n_rows)
    assert torch.equal(one, got[1])
    cache.read(1, x.table, x.len, k_out=one, n_rows=x.n_rows)
    assert torch.equal(one, got[0])


def test_read_reports_capacity_and_bad_pages():
    x = Batch8("bf16", 4, 1, 128, 16, [30, 5], 4, max_pos=40)
    out = [torch.full((2, 1, 4, 128), 77.0, dtype=x.dt, device="cuda") for _ in range(2)]
    x.cache.read(0, x.table, i32([38, -1]), *out)  # positions 40, 41; -1
    assert x.cache.status() == capi.STATUS_CAPACITY
    assert (out[0][0, 0, 2:] == 77.0).all() and (out[0][1, 0, 0] == 77.0).all()
    assert (out[0][0, 0, :2] != 77.0).all() and (out[0][1, 0, 1:] != 77.0).all()
    t = x.table.clone()
    t[0, 1] = x.pool["k"].shape[1]
    x.cache.read(0, t, x.len, *out)
    assert x.cache.status() == capi.STATUS_BOUNDS


# ------------------------------------------------------------------ attention


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("c", CASES, ids=[f"{c[0]}-p{c[1]}-n{c[3]}-{max(c[2])}-{'c' if c[5] else 'f'}-w{c[6]}-s{c[7]}"
                                          for c in CASES])
def test_attention(c, dtype):
    """Every row within the bound that its arithmetic allows; padding rows stay as they were; the scales of slots
    that hold no position are NaN, and so are the padding rows' queries."""
    heads, ps, lens, n, rows, causal, window, sinks = c
    x = Batch8(dtype, *HEADS[heads], ps, lens, n, rows, fill=float("nan"), extra_cols=3)
    q = x.query()
    for b, r in enumerate(x.rows):
        q[b, r:] = float("nan")
    kw = dict(causal=causal, window=window, sinks=sinks)
    out = attend(x, q, **kw)
    assert x.cache.status() == 0
    untouched(x, out)
    check(x, out.masked_fill(torch.isnan(q), 0.0) if rows else out, reference(x, q, **kw), "attention")
    assert torch.equal(attend(x, q, **kw).nan_to_num(), out.nan_to_num())


SHARED = [
    # heads, ps, shared, lens behind it, n, rows, causal, window, sinks
    ("gqa4", 16, 300, [1, 0, 40], 1, None, True, 0, 0), ("wide", 64, 1024, [5, 100], 16, None, True, 0, 0),
    ("gqa5", 32, 130, [7, 0, 64, 200], 15, [15, 0, 3, 1], True, 0, 0), ("mha64", 128, 500, [1, 2, 3], 5, None, False, 0, 0),
    ("gqa3", 16, 999, [50, 9], 40, None, True, 0, 0), ("gqa4", 16, 2000, [30, 700], 4, None, True, 600, 20),
    ("one", 64, 64, [0, 0], 1, None, True, 0, 0), ("mqa", 32, 31, [5, 1], 3, None, True, 0, 0),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("c", SHARED, ids=[f"{c[0]}-p{c[1]}-{c[2]}-n{c[4]}-w{c[7]}" for c in SHARED])
def test_shared_prefix(c, dtype):
    heads, ps, shared, behind, n, rows, causal, window, sinks = c
    x = Batch8(dtype, *HEADS[heads], ps, [shared + y for y in behind], n, rows, fill=float("nan"), shared=shared)
    q = x.query()
    kw = dict(causal=causal, window=window, sinks=sinks)
    out = attend(x, q, shared=shared, **kw)
    assert x.cache.status() == 0
    untouched(x, out)
    check(x, out, reference(x, q, **kw), "shared")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n", [1, 9, 40])
@pytest.mark.parametrize("key, value", [(1e-6, 1e-6), (1.0, 1e4), (1e-3, 1e30), (1e-25, 1e-30), (1.0, 1.0)])
def test_scales_of_any_size(key, value, n, dtype):
    """Keys, values and queries far from one: scales of 1e-30 and 1e30, and queries that make up for the keys'."""
    x = Batch8(dtype, 8, 2, 128, 32, [300, 45], n)
    x.pool["k_scale"] *= key / 0.03
    x.pool["v_scale"] *= value / 0.03
    x.pool["v_scale"][:, :, :, ::3] *= 1e-4  # and far from one another
    # (float32 queries hold 1e25 / 127; bf16 ones too)
    q = (x.query().float() * (0.03 / key)).to(x.dt)
    check(x, attend(x, q), reference(x, q), "scales")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n", [1, 16, 64])
def test_rows_that_read_as_nan_reach_only_those_that_see_them(n, dtype):
    """A key and a value with scale NaN behind the first row of a block, a value in a window's blind part: rows that
    see them are NaN, others are not touched."""
    x = Batch8(dtype, 4, 1, 128, 16, [200], n)
    q = x.query()
    kw = dict(causal=True, window=100, sinks=4)
    want = attend(x, q, **kw)

    def spoil(name, p):
        x.pool[name][0, int(x.table[0, p // 16]), 0, p % 16] = float("nan")

    spoil("k_scale", 50)
    spoil("v_scale", 60)  # seen by no row: 200 - 99 = 101 is the first row's window
    assert torch.equal(attend(x, q, **kw), want)
    at = 200 + n // 2  # seen from row n / 2 on
    for name in ("v_scale", "k_scale"):
        keep = {k: t.clone() for k, t in x.pool.items()}
        spoil(name, at)
        got = attend(x, q, **kw)
        assert torch.isnan(got[0, n // 2:]).all()
        assert torch.equal(got[0, :n // 2], want[0, :n // 2])
        for k, t in x.pool.items():
            t.copy_(keep[k])


FAR = [  # heads, lens, n, kwargs: more sequences than a CTA has threads, lengths of every kind, items of every height
    ("gqa4", [(7 * b) % 90 for b in range(300)], 1, {}), ("gqa4", [(13 * b) % 70 for b in range(150)], 16, {}),
    ("mha64", [(5 * b) % 40 for b in range(260)], 3, dict(window=20, sinks=2)), ("mqa", [64 * b for b in range(9)], 3, {}),
]


@pytest.mark.parametrize("c", FAR, ids=[f"{c[0]}-{len(c[1])}-n{c[2]}" for c in FAR])
def test_attention_of_many_sequences(c):
    heads, lens, n, kw = c
    x = Batch8("bf16", *HEADS[heads], 16, lens, n, fill=float("nan"))
    q = x.query()
    out = attend(x, q, **kw)
    assert x.cache.status() == 0
    check(x, out, reference(x, q, **kw), "many sequences")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n", [1, 8, 33])
def test_attention_reports_bad_pages(n, dtype):
    """A page outside the pool: the status says so, and the other sequences' rows are what they were."""
    x = Batch8(dtype, 4, 1, 128, 32, [500, 300, 200], n)
    q = x.query()
    want = attend(x, q)
    for bad in (-1, x.pool["k"].shape[1], 2 ** 31 - 1, -2 ** 31):
        good = int(x.table[1, 3])
        x.table[1, 3] = bad
        got = attend(x, q)
        assert x.cache.status() == capi.STATUS_BOUNDS
        x.table[1, 3] = good
        assert torch.equal(got[[0, 2]], want[[0, 2]])
        assert torch.equal(attend(x, q), want) and x.cache.status() == 0


@pytest.mark.parametrize("n, shared", [(1, None), (16, None), (100, None), (40, 1920)])
def test_attention_whose_waits_run_out(n, shared):
    """With a limit of 0 every wait for copies and products has run out before it begins (calls of few rows have none).
    The status says so, nothing but the result is written, and the next call after the status is right."""
    x = Batch8("bf16", 8, 2, 128, 32, [2000, 2000, 2100], n, shared=shared or 0)
    q = x.query()
    buf = torch.full((q.numel() + 1024,), 77.0, dtype=x.dt, device="cuda")
    out = buf[512:-512].view(q.shape)

    def call():
        x.cache.attention(0, q, x.table, x.len, out, shared_len=None if shared is None else i32([shared]))

    call()
    assert x.cache.status() == 0
    want = out.clone()
    check(x, want, reference(x, q), "before")
    pool = {k: t.clone() for k, t in x.pool.items()}
    try:
        for ns in (0, 0, 20000, 2000, 300):
            capi.dflash_debug_set_wait_limit(ns)
            out.fill_(77.0)
            call()
            status = x.cache.status()
            assert status in (0, capi.STATUS_TIMEOUT) and (ns or n == 1 or status)
            if not status:
                assert torch.equal(out, want)
            capi.dflash_debug_set_wait_limit(-1)
            call()
            assert x.cache.status() == 0 and torch.equal(out, want)
    finally:
        capi.dflash_debug_set_wait_limit(-1)
    assert all(torch.equal(t, pool[k]) for k, t in x.pool.items())
    assert (buf[:512] == 77.0).all() and (buf[-512:] == 77.0).all()


@pytest.mark.parametrize("n", [1, 9, 64])
def test_value_scales_below_zero(n):
    """A pool that another program filled may hold them; the entries are (u - 128) s all the same."""
    x = Batch8("bf16", 4, 1, 128, 16, [300, 60], n)
    x.pool["v_scale"].neg_().mul_(1e6)
    x.pool["v_scale"][..., ::3] *= -1e-3
    q = x.query()
    check(x, attend(x, q), reference(x, q), "negative scales")


@pytest.mark.parametrize("n", [1, 8, 40])
def test_on_another_stream_and_replayed(n):
    """Append, attention and reading back on a stream of their own and in a graph: the results of the plain calls."""
    x = Batch8("bf16", 8, 2, 128, 64, [200, 63, 900], n)
    q, out = x.query(), torch.zeros(3, n, 8, 128, dtype=x.dt, device="cuda")
    qkv = x.normal(3, n, 12 * 128)
    rows = torch.zeros(3, 2, n, 128, dtype=x.dt, device="cuda")
    qr = torch.zeros_like(q)

    def calls():
        x.cache.append(0, qkv.view(3 * n, -1), x.table, x.len, n, q_out=qr)
        x.cache.attention(0, qr, x.table, x.len, out)
        x.cache.read(0, x.table, x.len, rows)

    calls()
    want = [t.clone() for t in (out, rows, qr)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        for t in (out, rows, qr):
            t.zero_()
        calls()
    torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(a, b) for a, b in zip((out, rows, qr), want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls()
    for t in (out, rows, qr):
        t.zero_()
    graph.replay()
    graph.replay()
    assert all(torch.equal(a, b) for a, b in zip((out, rows, qr), want))
    assert x.cache.status() == 0


@pytest.mark.parametrize("n", [1, 8, 40])
def test_queries_that_are_not_finite_stay_in_their_row(n):
    """A query row that holds an infinity or a NaN gives NaN in its head, and every other row what it gave before."""
    x = Batch8("bf16", 8, 2, 128, 32, [300, 90, 700], n)
    q = x.query()
    want = attend(x, q)
    bad = q.clone()
    bad[0, 0, 3, 5], bad[1, n - 1, 6, 0], bad[2, n // 2, 1, 127] = math.inf, math.nan, -math.inf
    got = attend(x, bad)
    assert x.cache.status() == 0
    for b, i, h in ((0, 0, 3), (1, n - 1, 6), (2, n // 2, 1)):
        assert torch.isnan(got[b, i, h]).all()
        got[b, i, h] = want[b, i, h]
    assert torch.equal(got, want)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_pools_past_32_bits(dtype):
    """Codes of more than 2^32 bytes: every call reaches the last pages."""
    x = Batch8(dtype, 8, 8, 128, 128, [300, 50, 1000], 40, spare=36000)
    assert x.pool["k"].numel() > 2 ** 32
    x.table[0, :3] = torch.arange(3, device="cuda", dtype=torch.int32) + x.pool["k"].shape[1] - 3
    for n in (1, 4, 40):
        q = x.query()[:, :n].contiguous()
        y = SimpleNamespace(**vars(x))
        y.n, y.rows, y.keys = n, [n] * 3, x.keys
        out = torch.zeros_like(q)
        x.cache.attention(0, q, x.table, x.len, out)
        check(y, out, reference(y, q), f"{n} rows")
    back = torch.zeros(3, 8, 300, 128, device="cuda")
    start = torch.zeros_like(x.len)
    x.cache.read(0, x.table, start, back, n_rows=i32([300, 50, 300]))
    assert torch.equal(back[0], x.keys(0, 300)[0].float())
    qkv = x.normal(3, 24 * 128)
    x.cache.append(0, qkv, x.table, x.len, 1, q_out=torch.zeros(3, 1, 8, 128, dtype=x.dt, device="cuda"))
    page = int(x.table[0, 300 // 128])
    v = qkv[0, 16 * 128:].view(8, 128).float()
    s = (v.abs().amax(1).double() / 127).float()
    assert torch.equal(x.pool["v_scale"][0, page, :, 300 % 128], s)
    want = torch.round((v.double() / s.double()[:, None]).float()).double() + 128
    assert torch.equal(x.pool["v"][0, page, :, 300 % 128].double(), want)
    assert x.cache.status() == 0


def test_refusals():
    x = Batch8("bf16", 4, 1, 128, 16, [30, 5], 4)
    c, q = x.cache, x.query()
    out = torch.zeros(2, 1, 4, 128, dtype=x.dt, device="cuda")
    for a in ((None, None), (out[:1], None), (out.half(), None), (out, out.float()), (out.transpose(2, 3), None),
              (out[:, :, :3], None), (out.cpu(), None)):
        with pytest.raises(ValueError):
            c.read(0, x.table, x.len, *a)
    for layer in (-1, 1):
        with pytest.raises(capi.DFlashError):
            c.read(layer, x.table, x.len, out)
    with pytest.raises(capi.DFlashError):  # over one another
        c.read(0, x.table, x.len, out, out)
    # results over the codes or the scales
    big = x.pool["k"].view(torch.bfloat16).flatten()[:out.numel()].view(out.shape)
    with pytest.raises(capi.DFlashError):
        c.read(0, x.table, x.len, big)
    scales = x.pool["v_scale"].view(torch.bfloat16).flatten()
    over = scales[:128].view(1, 1, 1, 128)
    with pytest.raises(capi.DFlashError):
        c.read(0, x.table[:1], x.len[:1], over)
    rows = torch.zeros(1, 4 * 128, dtype=x.dt, device="cuda").view(1, 1, 4, 128)
    if scales.numel() >= 4 * 128:
        with pytest.raises(capi.DFlashError):
            c.attention(0, rows, x.table[:1], x.len[:1], scales[:4 * 128].view(1, 1, 4, 128))
    good = {k: t.clone() for k, t in x.pool.items()}
    shape = shape_of(4, 1, 128)
    dims = x.pool["k"].shape

    def make(**kw):
        return PagedCache(shape, "bf16", dims[1], 16, 64, 8, kv_format="q8", **{**good, **kw})

    for kw in (dict(k=None), dict(k_scale=None), dict(k=good["k"].to(torch.int8)), dict(v_scale=good["v_scale"].double()),
               dict(v_scale=good["v_scale"][:, :-1]), dict(k=good["k"].cpu())):
        with pytest.raises(ValueError):
            make(**kw)
    with pytest.raises(ValueError):
        PagedCache(shape, "bf16", dims[1], 16, 64, 8, kv_format="q4")
    with pytest.raises(ValueError):
        PagedCache(shape, "bf16", dims[1], 16, 64, 8, k_scale=good["k_scale"], v_scale=good["v_scale"])
    made = PagedCache(shape, "bf16", 3, 16, 48, 8, kv_format="q8")
    assert (made.k == 128).all() and (made.v_scale == 0).all() and made.k.shape == (1, 3, 1, 16, 128)
    assert q is not None


# ------------------------------------------------------------------ together


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n", [1, 16])
def test_a_decoder_layer(n, dtype):
    """A pre-norm decoder layer with 4-bit weights over 8-bit pages, call by call, captured and replayed: each step
    against 64 bits from the step before, as the layer hands it on."""
    H, nq, nkv, hd, F, B = 512, 4, 1, 128, 1024, 3
    if dtype == "f32":
        H, nq, nkv, hd, F = 256, 4, 4, 64, 768
    lens = [40, 0, 133]
    x = Batch8(dtype, nq, nkv, hd, 16, lens, n)
    rows, dt = B * n, x.dt
    mats = {k: W4Linear.from_weight(x.normal(*s, scale=0.05, dtype=torch.float32), 64, zeros=k == "down")
            for k, s in dict(qkv=((nq + 2 * nkv) * hd, H), o=(H, nq * hd), gate_up=(2 * F, H), down=(H, F)).items()}
    ws = W4Workspace(rows)
    gains = [x.normal(H) for _ in range(2)]
    resid0 = x.normal(rows, H, dtype=torch.float32)
    resid = resid0.clone()
    a, a2 = (torch.zeros(rows, H, dtype=dt, device="cuda") for _ in range(2))
    qkv = torch.zeros(rows, (nq + 2 * nkv) * hd, device="cuda")
    q, o = (torch.zeros(B, n, nq, hd, dtype=dt, device="cuda") for _ in range(2))
    mid, act = torch.zeros(rows, H, device="cuda"), torch.zeros(rows, F, dtype=dt, device="cuda")
    code = capi.BF16 if dtype == "bf16" else capi.F32

    def layer():
        capi.dflash_rmsnorm(code, resid, gains[0], a, rows, H, 1e-6)
        mats["qkv"].product(a, qkv, ws)
        x.cache.append(0, qkv, x.table, x.len, n, q_out=q)
        x.cache.attention(0, q, x.table, x.len, o)
        mats["o"].product(o.view(rows, nq * hd), mid, ws, add=resid)
        capi.dflash_rmsnorm(code, mid, gains[1], a2, rows, H, 1e-6)
        mats["gate_up"].product(a2, act, ws, swiglu=True)
        mats["down"].product(act, resid, ws, add=mid)

    layer()
    assert x.cache.status() == 0
    eager = [t.clone() for t in (a, qkv, q, o, mid, a2, act, resid)]
    w = {k: m.weight(torch.float32).double() for k, m in mats.items()}

    def near(got, want, mag):
        """A sum of at most 2048 products: 2^-11 of their magnitudes (2048 2^-23 and more than as much again)."""
        assert ((got.double() - want).abs() <= 2.0 ** -11 * mag + (2.0 ** -8 if got.dtype == torch.bfloat16 else 0) * want.abs()).all()

    def times(m, v):
        return v.double() @ w[m].T, v.double().abs() @ w[m].abs().T

    for got, src, gain in ((a, resid0, gains[0]), (a2, mid, gains[1])):
        want = src.double() / (src.double().square().mean(1, keepdim=True) + 1e-6).sqrt() * gain.double()
        near(got, want, want.abs())
    near(qkv, *times("qkv", a))
    want = rotated(qkv.double().view(B, n, -1, hd)[:, :, :nq], x.len[:, None] + torch.arange(n, device="cuda"), hd)
    near(q, want, qkv.abs().max())
    check(x, o, reference(x, q), "layer")
    y, m = times("o", o.view(rows, -1))
    near(mid, y + resid0.double(), m + resid0.double().abs())
    y, m = times("gate_up", a2)
    want = torch.nn.functional.silu(y[:, 0::2]) * y[:, 1::2]
    near(act, want, 1.1 * m[:, 0::2] * (y[:, 1::2].abs() + 1) + m[:, 1::2] * y[:, 0::2].abs())
    y, m = times("down", act)
    near(resid, y + mid.double(), m + mid.double().abs())
    # captured: the same bits
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        layer()
    torch.cuda.current_stream().wait_stream(s)
    for _ in range(2):
        resid.copy_(resid0)
        for t in (a, qkv, q, o, mid, a2, act):
            t.zero_()
        graph.replay()
        for t, e in zip((a, qkv, q, o, mid, a2, act, resid), eager):
            assert torch.equal(t, e)
    assert x.cache.status() == 0


def test_pages_to_a_cache_and_back():
    """A sequence read out of 8-bit pages, written into other ones: the codes are the same where the row's largest
    entry has code 1 or 255 (its scale is then kept)."""
    x = Batch8("f32", 4, 4, 64, 16, [0], 50)
    x.pool["k"][..., 0] = 255
    x.pool["v"][..., 5] = 1
    k, v = (torch.zeros(1, 4, 50, 64, device="cuda") for _ in range(2))
    x.cache.read(0, x.table, x.len, k, v)
    rows = torch.cat([k, v], 1).transpose(1, 2).reshape(50, 8 * 64).contiguous()
    y = Batch8("f32", 4, 4, 64, 32, [0], 50, seed=1)
    # position 0 of a one-row call is not rotated: rows are appended at position 0 of 50 sequences of one page each
    one = PagedCache(SimpleNamespace(**{**vars(shape_of(4, 4, 64)), "rope_theta": THETA}), "f32", 50, 16, 16, 50,
                     kv_format="q8")
    one.append(0, rows, torch.arange(50, dtype=torch.int32, device="cuda")[:, None].contiguous(),
               torch.zeros(50, dtype=torch.int32, device="cuda"), 1)
    page = x.table[0].long()[torch.arange(50, device="cuda") // 16]
    slot = torch.arange(50, device="cuda") % 16
    for name in ("k", "v"):
        was = x.pool[name][0][page, :, slot]
        assert torch.equal(getattr(one, name)[0, :, :, 0], was)
        s = x.pool[name + "_scale"][0][page, :, slot]
        assert ((getattr(one, name + "_scale")[0, :, :, 0] - s).abs() <= 2.0 ** -22 * s).all()
    assert y is not None
