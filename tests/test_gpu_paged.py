"""The paged cache on the GPU: the append with the rotation on the way,
attention over pages (sliding window, sinks, ragged rows) and attention of a
batch that shares a prefix, against 64-bit implementations written here."""
import math
from types import SimpleNamespace

import pytest

torch = pytest.importorskip("torch")

from block_diffusion_speculative_target_gb300 import capi  # noqa: E402
from block_diffusion_speculative_target_gb300.engine import PagedCache  # noqa: E402

pytestmark = pytest.mark.gpu

TDT = {"f32": torch.float32, "bf16": torch.bfloat16}
THETA = 1.0e6


def shape_of(nq, nkv, hd):
    return SimpleNamespace(n_layers=1, hidden=nq * hd, n_q=nq, n_kv=nkv, head_dim=hd, ffn=256, vocab=256,
                           rope_theta=THETA, eps=1e-6)


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Batch:
    """A pool with scattered pages, their tables, lengths and a PagedCache over them."""

    def __init__(self, dtype, nq, nkv, hd, ps, lens, n, rows=None, seed=0, layers=1, fill=None, spare=2, extra_cols=0,
                 shared=0):
        self.g = torch.Generator(device="cuda").manual_seed(1000 + seed)
        self.dtype, self.dt, self.nq, self.nkv, self.hd, self.ps, self.n = dtype, TDT[dtype], nq, nkv, hd, ps, n
        self.lens, self.rows = list(lens), [n] * len(lens) if rows is None else list(rows)
        B = len(lens)
        self.cols = max(-(-(x + n) // ps) for x in lens) + extra_cols
        common = shared // ps
        own = [-(-(x + n) // ps) - common for x in lens]
        n_pages = common + sum(own) + spare
        perm = torch.randperm(n_pages, generator=self.g, device="cuda").tolist()
        table = [[-7] * self.cols for _ in range(B)]  # entries that no call may use are no pages
        at = common
        for b in range(B):
            for c in range(own[b] + common):
                table[b][c] = perm[c] if c < common else perm[at + c - common]
            at += own[b]
        self.table = i32(table)
        self.len, self.n_rows = i32(self.lens), None if rows is None else i32(rows)
        dims = (layers, n_pages, nkv, ps, hd)
        self.k, self.v = self.normal(*dims), self.normal(*dims)
        if fill is not None:  # what lies in slots that hold no position
            for b in range(B):
                live = torch.zeros(n_pages * ps, dtype=torch.bool, device="cuda")
            for b in range(B):
                p = torch.arange(self.lens[b] + min(max(self.rows[b], 0), n), device="cuda")
                live[self.table[b].long()[p // ps] * ps + p % ps] = True
            dead = ~live.view(1, n_pages, 1, ps, 1).expand(dims)
            self.k[dead] = fill
            self.v[dead] = fill
        if shared % ps:
            at = shared // ps
            for pool in (self.k, self.v):
                pool[:, self.table[:, at].long(), :, :shared % ps] = pool[:, self.table[0, at].long()][:, None, :, :shared % ps]
        self.cache = PagedCache(shape_of(nq, nkv, hd), dtype, n_pages, ps, self.cols * ps, B * n, max_batch=B,
                                n_layers=layers, k=self.k, v=self.v)

    def normal(self, *dims, scale=1.0, dtype=None):
        return torch.empty(dims, dtype=dtype or self.dt, device="cuda").normal_(0, scale, generator=self.g)

    def query(self, scale=1.5):
        return self.normal(len(self.lens), self.n, self.nq, self.hd, scale=scale)

    def keys(self, b, count, layer=0):
        """The first `count` keys and values of sequence b: [nkv][count][hd] in 64 bits."""
        pages = self.table[b].long()[:-(-count // self.ps)]
        take = lambda t: t[layer][pages].permute(1, 0, 2, 3).reshape(self.nkv, -1, self.hd)[:, :count].double()  # noqa: E731
        return take(self.k), take(self.v)


def visible(P, rows, i, causal, window, sinks, count):
    """Which of `count` keys row i of a sequence with P held positions sees."""
    j = torch.arange(count, device="cuda")
    see = j <= P + i if causal else j < P + rows
    if window:
        see &= (j > P + i - window if causal else j >= P - window) | (j < sinks)
    return see


def reference(x, q, causal=True, window=0, sinks=0, layer=0):
    """(result, attention of |values|, largest sum of |q k| scale, keys) in 64 bits; rows that are padding hold 0."""
    G = x.nq // x.nkv
    out = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
    mag, dots, most = torch.zeros_like(out), 0.0, 1
    for b, (P, r) in enumerate(zip(x.lens, x.rows)):
        r = min(max(r, 0), x.n)
        if not r:
            continue
        k, v = x.keys(b, P + r, layer)
        for i in range(r):
            see = visible(P, r, i, causal, window, sinks, P + r)
            kk, vv = k[:, see], v[:, see]
            a = q[b, i].double().view(x.nkv, G, x.hd)
            z = a @ kk.transpose(1, 2) / math.sqrt(x.hd)
            p = torch.softmax(z, -1)
            out[b, i] = (p @ vv).reshape(x.nq, x.hd)
            mag[b, i] = (p @ vv.abs()).reshape(x.nq, x.hd)
            dots = max(dots, float((a.abs() @ kk.abs().transpose(1, 2)).max()) / math.sqrt(x.hd))
            most = max(most, kk.shape[1])
    return out, mag, dots, most


def bound(x, ref, mag, dots, most):
    """What a correct result may be off by.  u = 2^-24 (half a step of float32).
    A score is a sum of hd products: off by (hd + 2) u dots with the scaling, so a weight is off by that
    and the exponential's 4 u, relative; the weights' sum and the output's sum over `most` keys by `most` u
    each, and merging pieces by a few u more.  All of these scale with the attention of |values|.  A bf16
    result is rounded once (2^-8 of itself), and the weights once before the product with the values
    (2^-8 of the attention of |values|)."""
    u = 2.0 ** -24
    b = mag * u * (2 * ((x.hd + 2) * dots + 4) + 2 * most + 16)
    return b if x.dtype == "f32" else b + 2.0 ** -8 * (ref.abs() + b) + 2.0 ** -8 * mag


def check(x, got, want, what=""):
    ref, mag, dots, most = want
    d = (got.double() - ref).abs() - bound(x, ref, mag, dots, most)
    assert torch.isfinite(got).all(), f"{what}: a value is not finite"
    for b, r in enumerate(x.rows):
        r = min(max(r, 0), x.n)
        assert float(d[b, :r].max() if r else 0) <= 0, f"{what}: sequence {b} off by {float(d[b, :r].max()):.3e} more than its bound"


def attend(x, q, shared=None, **kw):
    out = torch.full_like(q, 77.0)
    x.cache.attention(0, q, x.table, x.len, out, n_rows=x.n_rows, shared_len=None if shared is None else i32([shared]), **kw)
    return out


def untouched(x, out):
    for b, r in enumerate(x.rows):
        assert (out[b, min(max(r, 0), x.n):] == 77.0).all(), f"padding rows of sequence {b} were written"


# ------------------------------------------------------------------ append


def rotated(x, pos, hd):
    """Rows x [..., heads, hd] in 64 bits rotated at pos [...]."""
    half = hd // 2
    a = pos.double()[..., None, None] * THETA ** (-torch.arange(half, device="cuda", dtype=torch.float64) / half)
    lo, hi = x[..., :half], x[..., half:]
    return torch.cat([lo * a.cos() - hi * a.sin(), hi * a.cos() + lo * a.sin()], -1)


APPENDS = [
    # dtype, in, nq, nkv, hd, ps, lens, n, rows, queries, pad (elements between rows), shift (elements off alignment)
    ("bf16", "f32", 32, 8, 128, 16, [4096], 1, None, True, 0, 0),
    ("bf16", "bf16", 5, 1, 128, 64, [0, 63, 64, 130], 16, [16, 3, 0, 9], True, 0, 0),
    ("bf16", "f32", 4, 1, 128, 32, [15, 31, 33], 7, [9, -2, 7], True, 24, 0),
    ("bf16", "bf16", 12, 4, 64, 128, [1000, 5], 33, None, True, 8, 0),
    ("bf16", "bf16", 4, 4, 64, 16, [17, 3], 5, None, True, 3, 1),
    ("f32", "f32", 4, 4, 64, 16, [0, 100], 16, None, True, 0, 0),
    ("f32", "f32", 8, 2, 128, 64, [61, 200, 1], 5, [5, 1, 2], True, 5, 3),
    ("bf16", "bf16", 8, 2, 128, 32, [7, 40], 16, [16, 2], False, 0, 0),
    ("bf16", "f32", 40, 8, 128, 128, [98300 - 128], 200, None, True, 0, 0),
]


@pytest.mark.parametrize("c", APPENDS, ids=[f"{c[0]}-{c[1]}-{c[2]}x{c[3]}x{c[4]}-p{c[5]}-n{c[7]}" for c in APPENDS])
def test_append(c):
    dtype, src, nq, nkv, hd, ps, lens, n, rows, queries, pad, shift = c
    x = Batch(dtype, nq, nkv, hd, ps, lens, n, rows, layers=2)
    heads = (nq if queries else 0) + 2 * nkv
    B, width = len(lens), heads * hd
    buf = x.normal(B * n * (width + pad) + shift, dtype=TDT[src])
    qkv = buf[shift:].view(B * n, width + pad)[:, :width]
    k0, v0 = x.k.clone(), x.v.clone()
    q_out = torch.full((B, n, nq, hd), 77.0, dtype=x.dt, device="cuda") if queries else None
    x.cache.append(1, qkv, x.table, x.len, n, q_out=q_out, n_rows=x.n_rows)
    assert x.cache.status() == 0
    z = qkv.double().view(B, n, heads, hd)
    pos = x.len[:, None] + torch.arange(n, device="cuda")
    turn = rotated(z[:, :, :heads - nkv], pos, hd)
    # cos and sin are off by 2^-24 of 1 and each of the two products and the sum once more: 4 * 2^-24 of
    # |x_lo| + |x_hi|; a bf16 result is rounded once more
    size = z.abs().view(B, n, heads, 2, hd // 2).sum(3, keepdim=True).expand(B, n, heads, 2, hd // 2).reshape(B, n, heads, hd)
    tol = 4 * 2.0 ** -24 * size[:, :, :heads - nkv]
    half = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -24
    wk, wv = k0.clone().double(), v0.clone()
    tk = torch.zeros_like(wk)
    for b in range(B):
        r = min(max(x.rows[b], 0), n)
        for j in range(r):
            p = lens[b] + j
            page = int(x.table[b, p // ps])
            wk[1, page, :, p % ps] = turn[b, j, -nkv:]
            tk[1, page, :, p % ps] = tol[b, j, -nkv:] + half * turn[b, j, -nkv:].abs()
            wv[1, page, :, p % ps] = z[b, j, -nkv:].to(x.dt)
        if queries:
            d = (q_out[b, :r].double() - turn[b, :r, :nq]).abs()
            assert (d <= tol[b, :r, :nq] + half * turn[b, :r, :nq].abs()).all()
            assert (q_out[b, r:] == 77.0).all()
    assert torch.equal(x.v, wv)
    assert ((x.k.double() - wk).abs() <= tk).all()


MANY = [
    # dtype, in, nq, nkv, hd, ps, lens, n, rows, queries, pad, shift
    ("bf16", "bf16", 40, 8, 128, 128, [0, 5, 300], 1000, [1000, 0, 999], True, 0, 0),
    ("bf16", "f32", 5, 1, 128, 16, [17, 4000], 11500, None, True, 0, 0),  # 7 heads: a group of one short
    ("bf16", "bf16", 12, 3, 64, 32, [1, 70], 9000, [9000, 8191], True, 5, 3),  # rows read entry by entry
    ("f32", "f32", 8, 2, 64, 64, [33], 26500, None, True, 0, 0),
    ("bf16", "bf16", 9, 3, 128, 16, [9, 3], 13100, None, False, 0, 0),
]


@pytest.mark.parametrize("c", MANY, ids=[f"{c[0]}-{c[1]}-{c[2]}x{c[3]}x{c[4]}-p{c[5]}-n{c[7]}" for c in MANY])
def test_append_many_rows(c):
    """Enough rows that a thread takes several heads; one page of the first sequence is none."""
    dtype, src, nq, nkv, hd, ps, lens, n, rows, queries, pad, shift = c
    x = Batch(dtype, nq, nkv, hd, ps, lens, n, rows)
    heads, B = (nq if queries else 0) + 2 * nkv, len(lens)
    width = heads * hd
    buf = x.normal(B * n * (width + pad) + shift, dtype=TDT[src])
    qkv = buf[shift:].view(B * n, width + pad)[:, :width]
    k0, v0 = x.k.clone(), x.v.clone()
    q_out = torch.full((B, n, nq, hd), 77.0, dtype=x.dt, device="cuda") if queries else None
    hole = (lens[0] + n // 2) // ps  # a column of the table
    was = int(x.table[0, hole])
    x.table[0, hole] = x.k.shape[1]
    x.cache.append(0, qkv, x.table, x.len, n, q_out=q_out, n_rows=x.n_rows)
    assert x.cache.status() == capi.STATUS_BOUNDS
    x.table[0, hole] = was
    z = qkv.double().view(B, n, heads, hd)
    j = torch.arange(n, device="cuda")
    pos = x.len[:, None].long() + j
    live = j < (torch.full((B,), n, device="cuda") if rows is None else x.n_rows)[:, None]
    turn = rotated(z[:, :, :heads - nkv], pos, hd)
    # as above: four roundings of |x_lo| + |x_hi|, and the result's own
    size = z.abs().view(B, n, heads, 2, hd // 2).sum(3, keepdim=True).expand(B, n, heads, 2, hd // 2).reshape(B, n, heads, hd)
    tol = 4 * 2.0 ** -24 * size[:, :, :heads - nkv] + (2.0 ** -8 if dtype == "bf16" else 2.0 ** -24) * turn.abs()
    if queries:
        assert ((q_out.double() - turn[:, :, :nq]).abs() <= tol[:, :, :nq])[live].all()
        assert (q_out[~live] == 77.0).all()
    kept = live.clone()
    kept[0] &= pos[0] // ps != hole
    b, r = kept.nonzero(as_tuple=True)
    page, slot = x.table[b, pos[b, r] // ps].long(), pos[b, r] % ps
    got_k, got_v = x.k[0].permute(0, 2, 1, 3)[page, slot], x.v[0].permute(0, 2, 1, 3)[page, slot]
    assert ((got_k.double() - turn[b, r, -nkv:]).abs() <= tol[b, r, -nkv:]).all()
    assert torch.equal(got_v, z[b, r, -nkv:].to(x.dt))
    rest = torch.ones(x.k.shape[1], ps, dtype=torch.bool, device="cuda")
    rest[page, slot] = False
    for now, then in ((x.k, k0), (x.v, v0)):
        assert torch.equal(now[0].permute(0, 2, 1, 3)[rest], then[0].permute(0, 2, 1, 3)[rest])


def test_append_reports_capacity_and_bad_pages():
    """A position past the table, past the rotation table and in a page outside the pool: the row is
    skipped, the bit is set, everything else is written."""
    x = Batch("bf16", 4, 1, 128, 16, [30, 5], 4)
    qkv = x.normal(8, 6 * 128)
    v0 = x.v.clone()
    q = torch.zeros(2, 4, 4, 128, dtype=x.dt, device="cuda")
    x.cache.append(0, qkv, x.table, i32([x.cols * 16 - 1, 5]), 4, q_out=q)  # rows 1..3 of sequence 0 are past the end
    assert x.cache.status() == capi.STATUS_CAPACITY
    assert (q[0, 1:] == 0).all() and (q[1].abs().sum(-1) > 0).all()
    x.v.copy_(v0)
    t = x.table.clone()
    t[0, 1], t[1, 0] = 10 ** 6, -1
    x.cache.append(0, qkv, t, x.len, 4, q_out=q)  # sequence 0: positions 30, 31 in page 1 (bad), 32, 33 in page 2
    assert x.cache.status() == capi.STATUS_BOUNDS
    assert (x.v != v0).flatten(2).any(2).sum() == 1  # one page changed
    small = PagedCache(shape_of(4, 1, 128), "bf16", x.k.shape[1], 16, 32, 8, k=x.k, v=x.v)
    small.append(0, qkv, x.table, i32([31, 0]), 4, q_out=q)
    assert small.status() == capi.STATUS_CAPACITY


# ------------------------------------------------------------------ attention

HEADS = {"gqa4": (4, 1, 128), "gqa5": (5, 1, 128), "mha64": (4, 4, 64), "gqa3": (6, 2, 64), "wide": (32, 8, 128),
         "mqa": (16, 1, 128), "mqa64": (64, 1, 64), "one": (1, 1, 128)}

CASES = [
    # heads, ps, lens, n, rows, causal, window, sinks
    ("gqa4", 16, [0], 1, None, True, 0, 0),
    ("gqa4", 16, [0, 1, 15, 16, 127, 128, 129], 1, None, True, 0, 0),
    ("wide", 64, [4095], 1, None, True, 0, 0),
    ("gqa5", 32, [700, 0, 255, 31], 16, None, True, 0, 0),
    ("gqa5", 32, [700, 0, 255, 31], 15, [15, 0, 1, 7], True, 0, 0),
    ("gqa5", 128, [700, 64], 16, None, False, 0, 0),
    ("mha64", 16, [300, 17, 1], 5, None, False, 0, 0),
    ("gqa3", 128, [1000, 3, 500], 40, [40, 2, 33], True, 0, 0),
    ("mqa", 16, [513, 90], 17, None, True, 0, 0),
    ("mqa64", 64, [200, 11], 9, None, True, 0, 0),
    ("one", 16, [1], 128, None, True, 0, 0),
    ("wide", 128, [0, 300], 128, None, True, 0, 0),
    ("gqa4", 16, [5000], 16, None, True, 100, 0),
    ("gqa4", 64, [5000, 90, 0], 16, None, True, 100, 4),
    ("gqa4", 16, [900, 130], 16, [3, 16], True, 1, 0),
    ("gqa4", 16, [900, 130], 7, None, True, 1, 1),
    ("gqa5", 32, [2500, 600], 15, None, False, 512, 64),
    ("gqa5", 32, [300], 15, None, False, 1, 200),
    ("mha64", 16, [777, 30], 3, None, True, 200, 130),
    ("wide", 32, [9000, 2500], 1, None, True, 128, 300),
    ("gqa3", 64, [400], 1, None, True, 100000, 5),
    ("wide", 16, [30000, 100, 7, 12000], 1, None, True, 0, 0),
    ("gqa4", 128, [2000], 100, None, False, 300, 10),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("c", CASES, ids=[f"{c[0]}-p{c[1]}-n{c[3]}-{max(c[2])}-{'c' if c[5] else 'f'}-w{c[6]}-s{c[7]}"
                                          for c in CASES])
def test_attention(c, dtype):
    """Every row within the bound that its arithmetic allows; padding rows stay as they were; slots that
    hold no position are full of NaN, and so are the padding rows' queries."""
    heads, ps, lens, n, rows, causal, window, sinks = c
    x = Batch(dtype, *HEADS[heads], ps, lens, n, rows, fill=float("nan"), extra_cols=3)
    q = x.query()
    for b, r in enumerate(x.rows):
        q[b, r:] = float("nan")
    kw = dict(causal=causal, window=window, sinks=sinks)
    out = attend(x, q, **kw)
    assert x.cache.status() == 0
    untouched(x, out)
    want = reference(x, q, **kw)
    check(x, out.masked_fill(torch.isnan(q), 0.0) if rows else out, want, "attention")
    # any shared length that all sequences reach is the same, when they hold the same keys there
    if len(lens) == 1:
        for sh in (1, ps, 128, lens[0], lens[0] + 9):
            check(x, attend(x, q, shared=sh, **kw), want, f"shared {sh}")
        assert x.cache.status() == 0


SHARED = [
    # heads, ps, shared, own lens, n, rows, causal, window, sinks
    ("wide", 16, 1024, [0, 1, 130, 17, 300], 1, None, True, 0, 0),
    ("gqa4", 64, 500, [0, 40, 1], 16, None, True, 0, 0),
    ("gqa5", 32, 700, [64, 3, 0, 90], 15, [0, 15, 2, 7], True, 0, 0),
    ("gqa5", 32, 700, [64, 3], 15, None, False, 0, 0),
    ("mha64", 128, 300, [10, 0], 3, None, True, 0, 0),
    ("gqa3", 16, 127, [10, 0], 3, None, True, 0, 0),
    ("wide", 16, 640, [5, 200], 16, None, True, 300, 20),
    ("gqa4", 128, 2000, [5, 600, 0], 8, [8, 0, 3], True, 64, 130),
    ("gqa4", 128, 900, [5, 600], 8, None, False, 700, 0),
    ("mqa", 16, 5000, list(range(0, 400, 10)), 1, None, True, 0, 0),
    ("gqa5", 64, 2000, [0, 7, 30, 0, 64, 128, 200, 1], 16, None, True, 0, 0),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("c", SHARED, ids=[f"{c[0]}-p{c[1]}-s{c[2]}-b{len(c[3])}-n{c[4]}-w{c[7]}" for c in SHARED])
def test_shared_prefix(c, dtype):
    heads, ps, shared, own, n, rows, causal, window, sinks = c
    x = Batch(dtype, *HEADS[heads], ps, [shared + y for y in own], n, rows, fill=float("nan"), shared=shared)
    q = x.query()
    for b, r in enumerate(x.rows):
        if not r:
            x.table[b] = -1  # a sequence without rows names no pages
    kw = dict(causal=causal, window=window, sinks=sinks)
    want = reference(x, q, **kw)
    for sh in (shared, shared + 5, 10 ** 9, 0, -3) if shared % ps == 0 and 0 in [o for o, r in zip(own, x.rows) if r] else (shared, 0):
        out = attend(x, q, shared=sh, **kw)
        assert x.cache.status() == 0
        untouched(x, out)
        check(x, out, want, f"shared {sh}")


def test_shared_prefix_is_read_from_one_table():
    """The common keys come from the first live sequence's pages: another's entries there are not read."""
    x = Batch("bf16", 4, 1, 128, 16, [512, 600, 530], 2, rows=[0, 2, 2], shared=512)
    q = x.query()
    want = reference(x, q)
    t = x.table.clone()
    t[0] = -1
    t[2, :32] = 10 ** 6
    out = torch.full_like(q, 77.0)
    x.cache.attention(0, q, t, x.len, out, n_rows=x.n_rows, shared_len=i32([512]))
    assert x.cache.status() == 0
    check(x, out, want)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_values_behind_a_mask_stay_there(dtype, bad):
    """Keys and values that a row does not see are NaN or infinite while other rows of the same block see
    them: only those that see them are touched."""
    x = Batch(dtype, 4, 1, 128, 16, [300, 40], 8)
    q = x.query()
    # the last two rows' own keys and values, and position 290 (outside the window of rows from 5 on)
    for b, p in ((0, 306), (0, 307), (1, 46), (0, 290)):
        page, slot = int(x.table[b, p // 16]), p % 16
        x.k[0, page, 0, slot] = bad
        x.v[0, page, 0, slot, 5:] = bad
    out = attend(x, q, window=14, sinks=2)
    ref, mag, dots, most = reference(x, q, window=14, sinks=2)
    sees = {0: [i for i in range(8) if 300 + i - 14 < 290 or i >= 6], 1: [6, 7]}
    for b in (0, 1):
        for i in range(8):
            if i in sees[b]:
                # the key's score may be +-inf: the row is NaN where the value is, as the definition has it
                assert torch.equal(torch.isfinite(out[b, i]), torch.isfinite(ref[b, i])), (b, i)
    clean = [(b, i) for b in (0, 1) for i in range(8) if i not in sees[b]]
    assert clean
    y = Batch(dtype, 4, 1, 128, 16, [300, 40], 8)
    want = reference(y, q, window=14, sinks=2)
    lim = bound(y, *want)
    for b, i in clean:
        assert ((out[b, i].double() - want[0][b, i]).abs() <= lim[b, i]).all(), (b, i)


def test_infinite_value_is_weighed_by_the_rows_that_see_it():
    """A value of +inf behind a finite key: +inf for the rows that see it, finite for those that do not."""
    x = Batch("bf16", 4, 1, 128, 16, [200], 6)
    q = x.query()
    x.v[0, int(x.table[0, 203 // 16]), 0, 203 % 16, 7] = float("inf")
    out = attend(x, q)
    ref = reference(x, q)[0]
    assert torch.equal(torch.isinf(out), torch.isinf(ref))
    assert torch.isinf(out[0, 3:, :, 7]).all() and torch.isfinite(out[0, :3]).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_large_scores(dtype):
    """Scores far apart (one key far above the rest, all far below zero, growing along the sequence)."""
    for kind in range(3):
        x = Batch(dtype, 4, 1, 128, 64, [1500], 4, seed=kind)
        q = x.query()
        pos = torch.arange(x.cols * 64, device="cuda")
        gain = [torch.where(pos == 700, 40.0, 0.2), torch.full_like(pos, -1.0, dtype=torch.float32), pos / 100.0][kind]
        d = q[0].float().mean((0, 1)).sign()
        pages = x.table[0].long()[:x.cols]
        x.k[0, pages] = (x.k[0, pages].float() * 0.3 + (gain.view(x.cols, 1, 64, 1) * d)).to(x.dt)
        out = attend(x, q)
        check(x, out, reference(x, q), f"kind {kind}")


def test_zero_rows_everywhere():
    x = Batch("bf16", 4, 1, 128, 16, [100, 20], 4, rows=[0, 0])
    q = x.query()
    for sh in (None, 64):
        out = attend(x, q, shared=sh)
        assert (out == 77.0).all() and x.cache.status() == 0


def test_bad_page_is_reported_and_stays_in_its_sequence():
    x = Batch("bf16", 4, 1, 128, 16, [300, 200], 2)
    q = x.query()
    want = reference(x, q)
    for page in (-1, x.k.shape[1], 2 ** 31 - 1, -2 ** 31):
        t = x.table.clone()
        t[0, 3] = page
        out = torch.zeros_like(q)
        x.cache.attention(0, q, t, x.len, out)
        assert x.cache.status() == capi.STATUS_BOUNDS
        d = (out[1].double() - want[0][1]).abs() - bound(x, *want)[1]
        assert d.max() <= 0
    x.cache.attention(0, q, x.table, i32([x.cols * 16 - 1, 200]), out)
    assert x.cache.status() == capi.STATUS_CAPACITY


def test_offsets_past_32_bits():
    """Pages whose elements lie beyond 2^31 (and bytes beyond 2^32) of the pool."""
    n_pages, ps, nkv, hd = 17000, 128, 8, 128
    x = Batch("bf16", 32, nkv, hd, ps, [1000, 129], 3)
    pool_k, pool_v = (torch.empty(n_pages, nkv, ps, hd, dtype=x.dt, device="cuda") for _ in range(2))
    far = n_pages - x.k.shape[1]
    pool_k[far:], pool_v[far:] = x.k[0], x.v[0]
    cache = PagedCache(shape_of(32, nkv, hd), "bf16", n_pages, ps, 2048, 6, k=pool_k, v=pool_v)
    t = torch.where(x.table >= 0, x.table + far, x.table)
    qkv = x.normal(6, 48 * 128)
    q, q2 = (torch.zeros(2, 3, 32, 128, dtype=x.dt, device="cuda") for _ in range(2))
    x.cache.append(0, qkv, x.table, x.len, 3, q_out=q)
    cache.append(0, qkv, t, x.len, 3, q_out=q2)
    assert torch.equal(q, q2) and torch.equal(pool_k[far:], x.k[0]) and torch.equal(pool_v[far:], x.v[0])
    out = torch.zeros_like(q)
    cache.attention(0, q, t, x.len, out)
    assert cache.status() == 0
    check(x, out, reference(x, q))


# ------------------------------------------------------------------ used together


def test_decoding_steps_together():
    """Three sequences that share a prompt, prefilled in chunks and decoded step by step in blocks whose
    accepted part varies: append, attention, attention with the shared prefix, lengths moved by the caller,
    on another stream and from captured graphs; two layers.  Every step against the plain computation over
    the contiguous history."""
    nq, nkv, hd, ps, n, shared, B = 8, 2, 128, 16, 8, 160, 3
    x = Batch("bf16", nq, nkv, hd, ps, [shared + 150] * B, n, layers=2, shared=shared)
    x.len.fill_(0)
    x.k.fill_(float("nan"))
    x.v.fill_(float("nan"))
    gen = torch.Generator(device="cuda").manual_seed(3)
    hist = [[[], []] for _ in range(B)]  # rotated keys, values of each sequence, as appended, per layer
    width = (nq + 2 * nkv) * hd

    def rows(count):
        return [torch.empty(count, width, device="cuda").normal_(generator=gen) for _ in range(2)]

    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        # the prompt once, through the first sequence's table
        for at in range(0, shared, 80):
            qkv = rows(80)
            one, chunk = i32([at]), torch.zeros(1, 80, nq, hd, dtype=x.dt, device="cuda")
            big = PagedCache(shape_of(nq, nkv, hd), "bf16", x.k.shape[1], ps, x.cols * ps, 80, n_layers=2, k=x.k, v=x.v)
            for layer in range(2):
                big.append(layer, qkv[layer], x.table[:1], one, 80, q_out=chunk)
                out = torch.zeros_like(chunk)
                big.attention(layer, chunk, x.table[:1], one, out)
                y = SimpleNamespace(**{**x.__dict__, "lens": [at], "rows": [80], "n": 80, "keys": x.keys})
                check(y, out, reference(y, chunk, layer=layer), f"prompt {at} layer {layer}")
            assert big.status() == 0
        x.len.fill_(shared)
        q = torch.zeros(2, B, n, nq, hd, dtype=x.dt, device="cuda")
        o1, o2, live, sh = torch.zeros_like(q), torch.zeros_like(q), i32([n] * B), i32([shared])
        qkv = [torch.zeros(B * n, width, device="cuda") for _ in range(2)]

        def step():
            for layer in range(2):
                x.cache.append(layer, qkv[layer], x.table, x.len, n, q_out=q[layer], n_rows=live)
                x.cache.attention(layer, q[layer], x.table, x.len, o1[layer], window=120, sinks=4, n_rows=live)
                x.cache.attention(layer, q[layer], x.table, x.len, o2[layer], n_rows=live, shared_len=sh)

        step()  # before the capture: modules load
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            step()
        lens = [shared] * B
        for s in range(6):
            counts = [(n, 1, 3), (1, 1, 1), (0, 8, 2)][s % 3]
            live.copy_(i32(counts))
            for layer, r in enumerate(rows(B * n)):
                qkv[layer].copy_(r)
            graph.replay() if s % 2 else step()
            x.lens, x.rows = lens, list(counts)
            for layer in range(2):
                check(x, o1[layer], reference(x, q[layer], window=120, sinks=4, layer=layer), f"step {s} window")
                check(x, o2[layer], reference(x, q[layer], layer=layer), f"step {s} shared")
            keep = [max(0, c - 1) for c in counts]  # the caller keeps part of the block
            lens = [a + b for a, b in zip(lens, keep)]
            x.len.copy_(i32(lens))
        assert x.cache.status() == 0
    torch.cuda.current_stream().wait_stream(stream)


def test_equal_calls_give_equal_bits():
    x = Batch("bf16", 40, 8, 128, 32, [3000, 10, 700, 4096, 1], 15, rows=[15, 3, 0, 9, 1], shared=0)
    q = x.query()
    first = attend(x, q)
    for _ in range(5):
        assert torch.equal(first, attend(x, q))


# stacked rows (n x query heads of a KV head) on both sides of every size at which the work is laid out anew
STACKED = [(1, 15), (1, 16), (1, 17), (2, 16), (11, 3), (16, 4), (13, 5), (64, 1), (65, 1), (32, 4), (43, 3), (128, 2), (257, 1)]


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("n,G", STACKED, ids=[f"{n * G}" for n, G in STACKED])
def test_stacked_rows(n, G, hd):
    """Few long sequences (pieces to join) and short ones, all and one of them padded, with and without the
    window, causal or not, on their own and behind a shared prefix; the same call gives the same bits."""
    x = Batch("bf16", 2 * G, 2, hd, 32, [6000, 640, 1000], n, rows=[n, max(n - 3, 0), 1], fill=float("nan"), seed=n * G, shared=640)
    q = x.query()
    for kw in (dict(), dict(window=700, sinks=5), dict(causal=False)):
        want = reference(x, q, **kw)
        for sh in (None, 640):
            out = attend(x, q, shared=sh, **kw)
            untouched(x, out)
            check(x, out, want, f"{kw} shared {sh}")
            assert torch.equal(out, attend(x, q, shared=sh, **kw))
    assert x.cache.status() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,n", [(33, 1), (64, 3), (128, 1), (129, 2), (300, 1), (700, 1)])
def test_many_sequences(B, n, dtype):
    """More sequences than lanes, than a warp plans, than threads and CTAs; one is long, some have no rows."""
    own = [(37 * b) % 200 for b in range(B)]
    own[B // 2] = 2000
    rows = [0 if b % 7 == 3 else 1 + b % n for b in range(B)]
    x = Batch(dtype, 8, 2, 64, 16, [160 + o for o in own], n, rows=rows, fill=float("nan"), seed=B, shared=160)
    q = x.query()
    for kw in (dict(), dict(window=90, sinks=2)):
        want = reference(x, q, **kw)
        for sh in (None, 160):
            out = attend(x, q, shared=sh, **kw)
            untouched(x, out)
            check(x, out, want, f"{kw} shared {sh}")
            assert torch.equal(out, attend(x, q, shared=sh, **kw))
    assert x.cache.status() == 0


def test_calls_at_the_same_time():
    """Two workspaces over one pool, on two streams, eager and from graphs: neither disturbs the other."""
    xs = [Batch("bf16", 8, 2, 128, 16, lens, n, seed=n) for lens, n in (([5000, 700, 3], 1), ([900, 4000], 16))]
    qs = [x.query() for x in xs]
    wants = [reference(x, q) for x, q in zip(xs, qs)]
    streams = [torch.cuda.Stream() for _ in xs]
    outs = [[torch.full_like(q, 77.0) for _ in range(8)] for q in qs]
    torch.cuda.synchronize()
    graphs = []
    for x, q, s, o in zip(xs, qs, streams, outs):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1], stream=s):
            for y in o[4:]:
                x.cache.attention(0, q, x.table, x.len, y)
    for k in range(4):
        for x, q, s, o in zip(xs, qs, streams, outs):
            with torch.cuda.stream(s):
                x.cache.attention(0, q, x.table, x.len, o[k])
    for s, g in zip(streams, graphs):
        with torch.cuda.stream(s):
            g.replay()
    torch.cuda.synchronize()
    for x, o, want in zip(xs, outs, wants):
        check(x, o[0], want)
        assert all(torch.equal(o[0], y) for y in o[1:])
        assert x.cache.status() == 0


def test_results_at_sixteen_bytes():
    """Queries and results that start 16 bytes past any larger boundary."""
    x = Batch("bf16", 8, 2, 128, 16, [900, 40], 5)
    q = x.query()
    first = attend(x, q)
    qb, ob = (torch.full((q.numel() + 16,), 77.0, dtype=x.dt, device="cuda") for _ in range(2))
    q2, o2 = qb[8:-8].view(q.shape), ob[8:-8].view(q.shape)
    q2.copy_(q)
    x.cache.attention(0, q2, x.table, x.len, o2)
    assert torch.equal(first, o2) and (ob[:8] == 77.0).all() and (ob[-8:] == 77.0).all()
    check(x, first, reference(x, q))


def test_status_in_stream_order():
    """Reading the status on another stream than the default one clears it before the next call's bits, not after."""
    x = Batch("bf16", 4, 1, 128, 16, [300, 200], 2)
    q = x.query()
    out = torch.zeros_like(q)
    bad = x.table.clone()
    bad[0, 3] = -1
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        for _ in range(50):
            x.cache.attention(0, q, bad, x.len, out)
            assert x.cache.status() == capi.STATUS_BOUNDS
        assert x.cache.status() == 0


# ------------------------------------------------------------------ refusals


def test_overlapping_memory_is_refused():
    x = Batch("bf16", 4, 1, 128, 16, [40, 5], 4)
    buf = torch.zeros(2, *x.query().shape, dtype=x.dt, device="cuda")
    flat = buf.view(-1)
    size = buf[0].numel()
    for at in (0, 8, size - 8):
        with pytest.raises(capi.DFlashError) as e:
            x.cache.attention(0, flat[:size].view(buf[0].shape), x.table, x.len, flat[at:at + size].view(buf[0].shape))
        assert e.value.code == capi.ERR_INVALID_ARG
    x.cache.attention(0, buf[0], x.table, x.len, buf[1])
    rows = torch.zeros(8 * 6 * 128 + size, dtype=x.dt, device="cuda")
    qkv, width = rows[:8 * 6 * 128].view(8, 6 * 128), 8 * 6 * 128
    for at in (0, 8, width - 8):
        with pytest.raises(capi.DFlashError) as e:
            x.cache.append(0, qkv, x.table, x.len, 4, q_out=rows[at:at + size].view(buf[0].shape))
        assert e.value.code == capi.ERR_INVALID_ARG
    x.cache.append(0, qkv, x.table, x.len, 4, q_out=rows[width:].view(buf[0].shape))
    assert x.cache.status() == 0


def test_refusals():
    x = Batch("bf16", 4, 1, 128, 16, [40, 5], 4)
    q, out, sh = x.query(), torch.zeros(2, 4, 4, 128, dtype=x.dt, device="cuda"), i32([0])
    c, L = x.cache, capi.load()

    def attention(**kw):
        a = dict(pages=c.pages, layer=0, q=q.data_ptr(), batch=2, n=4, n_rows=None, causal=1, window=0, sinks=0,
                 table=x.table.data_ptr(), stride=x.cols, len=x.len.data_ptr(), out=out.data_ptr(), ws=c.ws)
        a.update(kw)
        v = list(a.values())
        rc = L.dflash_paged_attention(*v, None)
        assert L.dflash_paged_attention_shared(*v[:12], sh.data_ptr(), *v[12:], None) == rc
        return rc

    for kw in (dict(pages=None), dict(layer=1), dict(layer=-1), dict(q=None), dict(q=q.data_ptr() + 2), dict(batch=0),
               dict(batch=3), dict(n=0), dict(n=5), dict(window=-1), dict(sinks=-1), dict(table=None), dict(stride=0),
               dict(len=None), dict(out=None), dict(out=out.data_ptr() + 8), dict(ws=None)):
        assert attention(**kw) == capi.ERR_INVALID_ARG, kw
    assert attention(stride=1 << 27) == capi.ERR_TOO_LARGE
    assert L.dflash_paged_attention_shared(c.pages, 0, q.data_ptr(), 2, 4, None, 1, 0, 0, x.table.data_ptr(), x.cols,
                                           x.len.data_ptr(), None, out.data_ptr(), c.ws, None) == capi.ERR_INVALID_ARG
    other = PagedCache(shape_of(8, 1, 128), "bf16", 4, 16, 64, 8)
    assert attention(ws=other.ws) == capi.ERR_INVALID_ARG
    qkv = x.normal(8, 6 * 128, dtype=torch.float32)

    def append(**kw):
        a = dict(pages=c.pages, layer=0, dtype=capi.F32, qkv=qkv.data_ptr(), ld=6 * 128, batch=2, n=4, n_rows=None,
                 table=x.table.data_ptr(), stride=x.cols, len=x.len.data_ptr(), q_out=q.data_ptr(), ws=c.ws)
        a.update(kw)
        return L.dflash_paged_append(*a.values(), None)

    for kw in (dict(pages=None), dict(layer=1), dict(dtype=7), dict(qkv=None), dict(qkv=qkv.data_ptr() + 2),
               dict(ld=6 * 128 - 1), dict(batch=0), dict(n=0), dict(table=None), dict(stride=0), dict(len=None),
               dict(q_out=q.data_ptr() + 2), dict(ws=None)):
        assert append(**kw) == capi.ERR_INVALID_ARG, kw
    f = PagedCache(shape_of(4, 1, 128), "f32", 4, 16, 64, 8)
    assert append(pages=f.pages, dtype=capi.BF16, ws=f.ws) == capi.ERR_INVALID_ARG  # bf16 rows into float32 pages
    assert c.status() == 0
    k = x.k
    for bad in (dict(n_pages=0), dict(page_size=24), dict(page_size=256), dict(max_pos=0)):
        a = dict(n_pages=k.shape[1], page_size=16, max_pos=64)
        a.update(bad)
        with pytest.raises((capi.DFlashError, ValueError)):
            PagedCache(shape_of(4, 1, 128), "bf16", a["n_pages"], a["page_size"], a["max_pos"], 8)
    with pytest.raises(capi.DFlashError) as e:
        PagedCache(shape_of(65, 1, 64), "bf16", 4, 16, 64, 8)
    assert e.value.code == capi.ERR_UNSUPPORTED_SHAPE
    with pytest.raises(ValueError):
        c.attention(0, q.float(), x.table, x.len, out)
    with pytest.raises(ValueError):
        c.attention(0, q, x.table.long(), x.len, out)
    with pytest.raises(ValueError):
        c.attention(0, q, x.table, x.len, out[:1])
    with pytest.raises(ValueError):
        c.attention(0, q, x.table[:, ::2], x.len, out)
    with pytest.raises(ValueError):
        c.append(0, qkv[:, :-1], x.table, x.len, 4, q_out=q)
    assert torch.equal(out, torch.zeros_like(out))
