"""The paged cache at the edges of what its calls allow, on the GPU."""
import pytest

torch = pytest.importorskip("torch")

from block_diffusion_speculative_target_gb300 import capi  # noqa: E402
from block_diffusion_speculative_target_gb300.engine import PagedCache  # noqa: E402
from test_gpu_paged import HEADS, Batch, attend, bound, check, i32, reference, shape_of, untouched, visible  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("heads,B,n", [("gqa4", 3, 1), ("gqa5", 5, 16), ("gqa4", 40, 1), ("mqa", 2, 20)])
def test_lengths_moved_by_the_kernel_before(heads, B, n, dtype):
    """Lengths, rows and the shared length are written by the kernels that run directly before the attention
    (and before an append and the attention), in a graph that is replayed many times: every call goes by
    what they wrote, so each result is the one of the same call made alone, bit for bit."""
    nq, nkv, hd = HEADS[heads]
    steps, shared = 6, 128
    top = [shared + 700 + 90 * (b % 9) for b in range(B)]
    x = Batch(dtype, nq, nkv, hd, 16, top, n, rows=[n] * B, seed=B, shared=shared)
    q, live, sh = x.query(), x.n_rows, i32([0])
    first = i32([shared + 11 * (b % 7) for b in range(B)])
    rows0 = i32([n - (b % 2) * (n - 1) for b in range(B)])
    qkv = x.normal(B * n, (nq + 2 * nkv) * hd)
    scratch = torch.zeros_like(q)
    outs = [torch.full_like(q, 77.0) for _ in range(steps)]

    def move(k):
        x.len.add_(97 + k)
        live.copy_(rows0 if k % 2 else torch.full_like(rows0, n))
        sh.fill_(0 if k % 3 == 0 else shared)

    def call(k, out):
        # (the append writes rows that its own attention sees; the pool is put back before every pass)
        if k % 2:
            x.cache.append(0, qkv, x.table, x.len, n, q_out=scratch, n_rows=live)
        x.cache.attention(0, q, x.table, x.len, out, n_rows=live, shared_len=sh if k % 3 else None)

    k0, v0 = x.k.clone(), x.v.clone()

    def reset():
        x.len.copy_(first)
        x.k.copy_(k0)
        x.v.copy_(v0)
        for o in outs:
            o.fill_(77.0)

    want = []
    reset()
    for k in range(steps):
        move(k)
        torch.cuda.synchronize()
        out = torch.full_like(q, 77.0)
        call(k, out)
        torch.cuda.synchronize()
        want.append(out)
    reset()
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        for k in range(steps):
            move(k)
            call(k, outs[k])
    with torch.cuda.stream(stream):
        for rep in range(30):
            reset()
            if rep % 3 == 2:
                for k in range(steps):
                    move(k)
                    call(k, outs[k])
            else:
                graph.replay()
            for k in range(steps):
                assert torch.equal(outs[k], want[k]), (rep, k)
    assert x.cache.status() == 0


def hide(x, causal, window, sinks, shared, bad):
    """The table with every entry whose positions no row sees replaced by `bad`."""
    t = x.table.clone()
    seen = []
    for P, r in zip(x.lens, x.rows):
        s = torch.zeros(x.cols * x.ps, dtype=torch.bool, device="cuda")
        for i in range(r):
            see = visible(P, r, i, causal, window, sinks, P + r)
            s[:P + r] |= see
        seen.append(s)
    common = torch.stack(seen).any(0)
    common[shared:] = False  # what some row sees of the shared positions is read from one table
    for b, s in enumerate(seen):
        keep = (s | common).view(x.cols, x.ps).any(1)
        t[b, ~keep] = bad
    return t


HIDDEN = [
    # heads, ps, lens, n, rows, causal, window, sinks
    ("gqa4", 16, [1000, 333, 90], 1, None, True, 100, 4),
    ("gqa4", 16, [1000, 333, 90], 1, None, True, 37, 0),
    ("gqa4", 16, [1000, 333, 90], 4, [4, 0, 2], True, 100, 130),
    ("gqa5", 32, [5000, 700], 6, None, True, 200, 40),
    ("gqa5", 16, [777, 200], 16, None, True, 64, 17),
    ("gqa4", 64, [3000, 450], 16, [16, 9], True, 150, 64),
    ("gqa4", 16, [2100, 640], 16, None, False, 250, 5),
    ("mha64", 16, [900, 301], 40, None, True, 90, 20),
    ("gqa4", 32, [1500], 40, None, True, 33, 3),
    ("wide", 16, [900], 100, None, False, 333, 50),
    ("gqa4", 16, [600, 700, 800], 2, None, True, 1, 1),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("c", HIDDEN, ids=[f"{c[0]}-p{c[1]}-n{c[3]}-{'c' if c[5] else 'f'}-w{c[6]}-s{c[7]}" for c in HIDDEN])
def test_entries_of_pages_that_no_row_sees_are_not_read(c, dtype):
    """Pages behind the window, and between the first tokens and the window, may have been given away: their
    entries are no pages, or another sequence's."""
    heads, ps, lens, n, rows, causal, window, sinks = c
    for shared in (0, 300):
        if shared > min(lens):
            continue
        x = Batch(dtype, *HEADS[heads], ps, lens, n, rows, fill=float("nan"), shared=shared)
        q = x.query()
        kw = dict(causal=causal, window=window, sinks=sinks)
        want = reference(x, q, **kw)
        for bad in (-1, 10 ** 6):
            t = hide(x, causal, window, sinks, shared, bad)
            assert (t == bad).any()
            out = torch.full_like(q, 77.0)
            x.cache.attention(0, q, t, x.len, out, n_rows=x.n_rows, shared_len=i32([shared]) if shared else None, **kw)
            assert x.cache.status() == 0, (shared, bad)
            untouched(x, out)
            check(x, out, want, f"shared {shared} bad {bad}")


# stacked rows 4, 16, 20, 24, 32, 64, 128, 256, 260 of 4 or 5 query heads a KV head
LAYOUTS = [(1, 4), (4, 4), (4, 5), (6, 4), (8, 4), (16, 4), (32, 4), (64, 4), (52, 5)]


@pytest.mark.parametrize("dtype,hd", [("bf16", 128), ("bf16", 64), ("f32", 128)])
@pytest.mark.parametrize("n,G", LAYOUTS, ids=[f"{n * G}" for n, G in LAYOUTS])
@pytest.mark.parametrize("window", [0, 300])
def test_values_that_are_not_finite(n, G, dtype, hd, window):
    """Infinite and NaN values in tiles that every row sees and in tiles that rows see in part: a row that sees
    one has the definition's infinity or NaN in that dimension, and nothing else of any row is touched."""
    for shared in (0, 384):
        x = Batch(dtype, G, 1, hd, 32, [3000, 900, 517], n, rows=[n, max(n - 2, 1), 1], seed=n * G, shared=shared)
        q = x.query()
        inf, nan = float("inf"), float("nan")

        def put(b, p, d, value):
            for s in range(3) if p < shared else (b,):
                x.v[0, int(x.table[s, p // 32]), 0, p % 32, d] = value

        for b, P in enumerate(x.lens):
            for base in (P - 150, P - 450, P + x.rows[b] - 1, P - 280, 200):  # (200: in the prefix of all)
                put(b, base, 3, inf)
                put(b, base, 8, -inf)
                put(b, base, 21, nan)
                put(b, base, 30, inf)
            put(b, P - 170, 30, -inf)  # both infinities
            put(b, P + x.rows[b] - 1, 40, inf)  # the last row's own position
        kw = dict(window=window, sinks=0 if n % 2 else 210)
        ref, mag, dots, most = reference(x, q, **kw)
        out = attend(x, q, shared=shared or None, **kw)
        untouched(x, out)
        lim = bound(x, ref, mag, dots, most)
        for b, r in enumerate(x.rows):
            got, want = out[b, :r].double(), ref[b, :r]
            for kind in (torch.isnan, torch.isposinf, torch.isneginf):
                assert torch.equal(kind(got), kind(want)), (kind.__name__, shared, b)
            ok = want.isfinite()
            assert ((got - want).abs() <= lim[b, :r])[ok].all(), (shared, b)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_many_rows_behind_a_wide_table(dtype):
    """16384 rows of 32 / 8 heads whose tables could name 131072 positions: what the lengths come to counts,
    and the result is that of narrow tables, bit for bit."""
    B, n, ps = 8, 2048, 64
    hd = 128 if dtype == "bf16" else 64
    x = Batch(dtype, 32, 8, hd, ps, [40 * b for b in range(B)], n, rows=[n - 100 * b for b in range(B)], shared=0)
    q = x.query()
    narrow = attend(x, q)
    cache = PagedCache(shape_of(32, 8, hd), dtype, x.k.shape[1], ps, 131072, B * n, max_batch=B, k=x.k, v=x.v)
    wide = torch.full((B, 131072 // ps), -1, dtype=torch.int32, device="cuda")
    wide[:, :x.cols] = x.table
    for shared in (None, 0):
        out = torch.full_like(q, 77.0)
        cache.attention(0, q, wide, x.len, out, n_rows=x.n_rows, shared_len=None if shared is None else i32([shared]))
        assert torch.equal(out, narrow)
    assert cache.status() == 0
    for b in (0, 5, 7):
        for i in (0, 1, 1000, x.rows[b] - 1):
            k, v = x.keys(b, x.lens[b] + i + 1)
            a = q[b, i].double().view(8, 4, hd)
            p = torch.softmax(a @ k.transpose(1, 2) / hd ** 0.5, -1)
            ref, mag = (p @ v).view(32, hd), (p @ v.abs()).view(32, hd)
            dots = float((a.abs() @ k.abs().transpose(1, 2)).max()) / hd ** 0.5
            assert ((narrow[b, i].double() - ref).abs() <= bound(x, ref, mag, dots, k.shape[1])).all(), (b, i)


def test_work_beyond_the_plan_is_refused():
    """65536 float32 rows of 64 heads, 2^10 groups a head, behind a table and a handle of 2^20 positions: 2^31
    tiles could lie on the line.  (Every array is as large as the call says.)"""
    n, heads, hd, ps = 1 << 16, 64, 64, 128
    cache = PagedCache(shape_of(heads, heads, hd), "f32", 1, ps, 1 << 20, n, max_batch=1)
    q = torch.zeros(1, n, heads, hd, device="cuda")
    out = torch.full_like(q, 77.0)
    table, length = torch.zeros(1, (1 << 20) // ps, dtype=torch.int32, device="cuda"), i32([0])
    with pytest.raises(capi.DFlashError) as e:
        cache.attention(0, q, table, length, out)
    assert e.value.code == capi.ERR_TOO_LARGE and (out == 77.0).all()
    # what lies past max_pos does not count
    small = PagedCache(shape_of(heads, heads, hd), "f32", 1, ps, 64, 64, max_batch=1)
    some = q[:, :64].contiguous()
    small.attention(0, some, table, length, out[:, :64].contiguous())
    assert small.status() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B", [3, 140])
def test_attention_reports_positions_that_the_handle_does_not_hold(dtype, B):
    """A length below zero, and rows past max_pos inside the table, set the status as the append does; other
    sequences are not touched."""
    x = Batch(dtype, 4, 1, 128, 16, [60] * B, 4, extra_cols=2)
    cache = PagedCache(shape_of(4, 1, 128), dtype, x.k.shape[1], 16, 64, 4 * B, max_batch=B, k=x.k, v=x.v)
    q = x.query()
    out = torch.full_like(q, 77.0)
    cache.attention(0, q, x.table, x.len, out)  # rows at 60..63: the last ones
    assert cache.status() == 0
    want = reference(x, q)
    check(x, out, want)
    lim = bound(x, *want)
    for bad in (61, -1, -2 ** 31, 2 ** 31 - 1):
        lens = x.len.clone()
        lens[1] = bad
        for sh in (None, 16):
            out = torch.full_like(q, 77.0)
            cache.attention(0, q, x.table, lens, out, shared_len=None if sh is None else i32([0]))
            assert cache.status() == capi.STATUS_CAPACITY, bad
            for b in (0, 2, B - 1):
                assert ((out[b].double() - want[0][b]).abs() <= lim[b]).all(), (bad, b)
    # a sequence without rows in the call names no position
    lens = x.len.clone()
    lens[1] = 61
    rows = i32([4, 0] + [4] * (B - 2))
    cache.attention(0, q, x.table, lens, out, n_rows=rows)
    assert cache.status() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_results_over_the_pool_are_refused(dtype):
    """A result inside a pool, rows to append that lie in one, and an append to pools that share memory would
    race with the call's own reads and writes."""
    x = Batch(dtype, 4, 1, 128, 16, [40, 5], 4)
    q, pools = x.query(), torch.zeros(3, *x.k.shape, dtype=x.dt, device="cuda")
    size, each = q.numel(), x.k.numel()
    flat = pools.view(-1)
    cache = PagedCache(shape_of(4, 1, 128), dtype, x.k.shape[1], 16, 64, 8, k=pools[0], v=pools[1])
    qkv = x.normal(8, 6 * 128)

    def refused(call):
        with pytest.raises(capi.DFlashError) as e:
            call()
        assert e.value.code == capi.ERR_INVALID_ARG

    for at in (0, each - 8, each + 16, 2 * each - 8):
        inside = flat[at:at + size].view(q.shape)
        refused(lambda: cache.attention(0, q, x.table, x.len, inside))
        refused(lambda: cache.attention(0, q, x.table, x.len, inside, shared_len=i32([0])))
        refused(lambda: cache.append(0, qkv, x.table, x.len, 4, q_out=inside))
    rows = flat[each - 8 * 6 * 128 + 8:][:8 * 6 * 128].view(8, 6 * 128)
    refused(lambda: cache.append(0, rows, x.table, x.len, 4, q_out=q))
    same = PagedCache(shape_of(4, 1, 128), dtype, x.k.shape[1], 16, 64, 8, k=pools[0], v=pools[0])
    refused(lambda: same.append(0, qkv, x.table, x.len, 4, q_out=q))
    assert (pools == 0).all() and cache.status() == 0
    # right behind the pools, and reading one that serves as keys and values, is fine
    out = flat[2 * each:2 * each + size].view(q.shape)
    cache.append(0, qkv, x.table, x.len, 4, q_out=q)
    cache.attention(0, q, x.table, x.len, out)
    same.attention(0, q, x.table, x.len, out)
    assert cache.status() == 0 and same.status() == 0 and torch.isfinite(out).all()


# one token's and up to 32 stacked rows; more
STACKS = [(1, 4, 128), (4, 4, 128), (5, 4, 128), (8, 4, 128), (6, 5, 64), (32, 1, 64), (16, 4, 128), (13, 5, 64), (40, 4, 128)]


@pytest.mark.parametrize("n,G,hd", STACKS, ids=[f"{n * G}x{hd}" for n, G, hd in STACKS])
def test_a_row_in_a_block_and_as_a_token(n, G, hd):
    """Row i of a block against the definition and against the same row as a single token of the position.
    u = 2^-24.  Up to 32 stacked rows a weight enters the product as hi + lo of bf16: lo is the rest of the
    first rounding (2^-8 of the weight at most) rounded once more, so the pair is off by 2^-16 of the weight
    and the sum by 2^-16 of the attention of |values|; beyond, by 2^-8 of it.  The result is rounded once
    (2^-8 of itself); float32 sums as in `bound`."""
    x = Batch("bf16", 2 * G, 2, hd, 32, [3000, 700], n, seed=n + G)
    q = x.query()
    token = PagedCache(shape_of(2 * G, 2, hd), "bf16", x.k.shape[1], 32, x.cols * 32, 2, k=x.k, v=x.v)
    for kw in (dict(), dict(window=500, sinks=70)):
        ref, mag, dots, most = reference(x, q, **kw)
        sums = mag * 2.0 ** -24 * (2 * ((hd + 2) * dots + 4) + 2 * most + 16)
        pair = sums + 2.0 ** -16 * mag
        pair = pair + 2.0 ** -8 * (ref.abs() + pair)
        lim = pair if n * G <= 32 else pair + 2.0 ** -8 * (1 + 2.0 ** -8) * mag
        out = attend(x, q, **kw)
        assert ((out.double() - ref).abs() <= lim).all(), kw
        for i in range(0, n, max(1, n // 4)):
            one = torch.full_like(q[:, i:i + 1].contiguous(), 77.0)
            token.attention(0, q[:, i:i + 1].contiguous(), x.table, x.len + i, one, **kw)
            assert ((one[:, 0].double() - ref[:, i]).abs() <= pair[:, i]).all(), (i, kw)
            assert ((one[:, 0].double() - out[:, i].double()).abs() <= pair[:, i] + lim[:, i]).all(), (i, kw)
    assert x.cache.status() == 0 and token.status() == 0


TIMEOUTS = [  # heads, lens, n, shared, kwargs: every layout, pieces joined by CTAs, by a kernel and with a prefix's
    ("gqa4", [4000, 3000, 10], 1, None, {}),
    ("gqa4", [4000, 3000, 10], 7, None, dict(window=900, sinks=9)),
    ("gqa4", [4000, 3000, 10], 16, None, {}),
    ("gqa5", [4000, 300], 40, None, {}),
    ("wide", [2000, 2000, 2100], 100, 1920, {}),
    ("gqa4", [2000, 2000, 2100], 1, 1920, {}),
]


@pytest.mark.parametrize("c", TIMEOUTS, ids=[f"{c[0]}-n{c[2]}-{c[3]}" for c in TIMEOUTS])
def test_a_wait_that_runs_out(c):
    """With a limit of 0 every wait for work has run out before it begins; with a few microseconds some do, while
    copies and products are in flight.  The status says so, nothing but the result is written, and the next call
    after the status is right."""
    heads, lens, n, shared, kw = c
    x = Batch("bf16", *HEADS[heads], 32, lens, n, shared=shared or 0)
    q = x.query()
    sh = None if shared is None else i32([shared])
    buf = torch.full((q.numel() + 1024,), 77.0, dtype=x.dt, device="cuda")
    out = buf[512:-512].view(q.shape)

    def call():
        x.cache.attention(0, q, x.table, x.len, out, shared_len=sh, **kw)

    call()
    assert x.cache.status() == 0
    want = out.clone()
    check(x, want, reference(x, q, **kw))
    k0, v0 = x.k.clone(), x.v.clone()
    try:
        for ns in (0, 0, 20000, 5000, 2000, 1000, 300):
            capi.dflash_debug_set_wait_limit(ns)
            out.fill_(77.0)
            call()
            status = x.cache.status()
            assert status in (0, capi.STATUS_TIMEOUT) and (ns or status)
            if not status:
                assert torch.equal(out, want)
            capi.dflash_debug_set_wait_limit(-1)
            call()
            assert x.cache.status() == 0 and torch.equal(out, want)
    finally:
        capi.dflash_debug_set_wait_limit(-1)
    assert torch.equal(x.k, k0) and torch.equal(x.v, v0)
    assert (buf[:512] == 77.0).all() and (buf[-512:] == 77.0).all()


SHORT = [  # heads, hd, G, B, shared, window, sinks: runs of items of one tile, with one and two query tiles
    (8, 64, 2, 130, 130, 100, 128),
    (8, 128, 2, 130, 128, 0, 0),
    (2, 128, 4, 300, 0, 0, 0),
    (8, 64, 13, 21, 256, 90, 5),
    (4, 128, 33, 12, 130, 0, 0),
]


@pytest.mark.parametrize("c", SHORT, ids=[f"{c[0]}x{c[2]}x{c[1]}-b{c[3]}" for c in SHORT])
def test_short_items_one_after_another(c):
    """Many items of one key tile in a CTA's run: its warps may be whole items apart."""
    nkv, hd, G, B, shared, window, sinks = c
    own = [(29 * b) % 100 for b in range(B)]
    x = Batch("bf16", nkv * G, nkv, hd, 64, [shared + o for o in own], 1, shared=shared, fill=float("nan"))
    q, kw = x.query(), dict(window=window, sinks=sinks)
    want = reference(x, q, **kw)
    for sh in (shared, None) if shared else (None,):
        first = attend(x, q, shared=sh, **kw)
        assert x.cache.status() == 0
        check(x, first, want, f"shared {sh}")
        outs = [torch.full_like(q, 77.0) for _ in range(40)]
        one = None if sh is None else i32([sh])
        for out in outs:
            x.cache.attention(0, q, x.table, x.len, out, shared_len=one, **kw)
        assert x.cache.status() == 0
        assert all(torch.equal(out, first) for out in outs)
