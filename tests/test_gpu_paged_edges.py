"""The paged cache at the edges of what its calls allow, on the GPU."""
import pytest

torch = pytest.importorskip("torch")

from test_gpu_paged import HEADS, Batch, i32  # noqa: E402

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
