"""Cases that measure the paged-cache operators: the append of rotated keys and
values into pages, attention over pages with a sliding window and sinks, and
attention of a batch that shares a prefix.

``run`` computes an operator in plain torch where ``own`` is false, and makes
the library's call where it is true.  Shapes are those of the repository's
workloads: 32 query and 8 KV heads of 128, 40 and 8, the small layouts with one
KV head, and the fp32 layout of 4 heads of 64.
"""
import json
import math
import random
from types import SimpleNamespace

import torch

own = False

THETA = 1.0e6
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def _case(name, op, **kw):
    c = {"name": name, "op": op, "dtype": "bf16", "in_dtype": "bf16", "nq": 32, "nkv": 8, "hd": 128, "page": 64,
         "batch": 1, "n": 1, "ragged": False, "lo": 0, "hi": 0, "causal": True, "window": 0, "sinks": 0, "shared": 0}
    c.update(kw)
    return c


def listed():
    return [
        # one decoded token's keys and values: the smallest call, all latency
        _case("append-token", "append", in_dtype="f32", lo=4096, hi=4096),
        # the blocks of a ragged batch of 8 speculative sequences, from the QKV product's float32 rows
        _case("append-blocks", "append", in_dtype="f32", batch=8, n=16, ragged=True, lo=2048, hi=6144, page=16),
        # a prefill of 8 prompts, appended at once
        _case("append-prefill", "append", nq=40, batch=8, n=2048, lo=0, hi=4096, page=128),
        # one sequence, one token, 4K context: latency
        _case("decode-4k", "attend", lo=4095, hi=4095, page=16),
        # verification of 16-row blocks for 8 ragged sequences
        _case("verify-batch8", "attend", batch=8, n=16, lo=2048, hi=6144),
        # a served batch of single tokens with contexts up to 36K, 5 query heads per KV head
        _case("decode-batch32", "attend", nq=40, batch=32, lo=512, hi=36864, page=32),
        # 15-row blocks far into 98K contexts, seen through a window of 4096 with 64 sinks; a padded batch
        _case("window-98k", "attend", batch=16, n=15, ragged=True, lo=49152, hi=98304, window=4096, sinks=64, page=16),
        # a prefill chunk of 128 rows behind 36K keys: products, not bytes
        _case("chunk-36k", "attend", nq=40, n=128, lo=36864, hi=36864, page=128),
        # the first chunks of 8 prompts: many rows over few keys
        _case("chunk-first", "attend", batch=8, n=128, lo=0, hi=256, page=32),
        # the fp32 layout: 4 heads of 64, a drafter's non-causal blocks
        _case("draft-f32", "attend", dtype="f32", nq=4, nkv=4, hd=64, batch=4, n=16, lo=128, hi=1024, causal=False,
              page=16),
        # 64 sequences one token each behind a common 12K prompt
        _case("shared-decode", "shared", batch=64, lo=1, hi=512, shared=12288, page=16),
        # 8 speculative blocks behind a common 36K document
        _case("shared-verify", "shared", nq=40, batch=8, n=16, lo=16, hi=2048, shared=36864),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["append", "attend", "attend", "shared"])
    f32 = rng.random() < 0.2
    nq, nkv, hd = rng.choice([(4, 4, 64), (8, 2, 64), (4, 1, 128), (32, 8, 128)]) if f32 else rng.choice(
        [(32, 8, 128), (40, 8, 128), (4, 1, 128), (5, 1, 128), (8, 8, 128), (12, 4, 64), (16, 2, 128)])
    c = {"op": op, "dtype": "f32" if f32 else "bf16", "nq": nq, "nkv": nkv, "hd": hd,
         "page": rng.choice([16, 32, 64, 128]), "ragged": rng.random() < 0.3, "lo": 0, "causal": True, "window": 0,
         "sinks": 0, "shared": 0}
    c["in_dtype"] = "f32" if f32 or rng.random() < 0.5 else "bf16"
    if op == "append":
        rows = _log(rng, 1, 16384)
        c["batch"] = _log(rng, 1, min(rows, 256))
        c["n"] = max(1, rows // c["batch"])
        c["hi"] = _log(rng, 1, 8192)
        return c
    c["n"] = rng.choice([1, 1, _log(rng, 2, 16), _log(rng, 17, 128)])
    # row-keys budgets keep a drawn case below the largest listed one, for the plain form too
    c["batch"] = _log(rng, 2 if op == "shared" else 1, 4 if c["n"] > 16 else 48)
    budget = (1 << 18) if f32 else (1 << 19)
    most = min(98304, budget // c["batch"], (1 << 27) // (c["batch"] * c["n"] * nq))
    ctx = _log(rng, 1, max(1, most))
    if op == "shared":
        c["hi"] = _log(rng, 1, max(1, min(2048, ctx)))
        c["shared"] = max(1, ctx - c["hi"])
    else:
        c["hi"] = ctx
        c["causal"] = rng.random() < 0.75
    c["lo"] = int(c["hi"] * rng.choice([0, 0.25, 1]))
    if rng.random() < 0.4:
        c["window"] = _log(rng, 1, max(2, ctx))
        c["sinks"] = rng.choice([0, 1, 4, 64, 130])
    return c


def lengths(case):
    """Keys held by each sequence before the call, and its rows of this call: of the case alone."""
    r = random.Random(json.dumps({k: v for k, v in sorted(case.items()) if k != "name"}))
    lens = [case["shared"] + r.randint(case["lo"], case["hi"]) for _ in range(case["batch"])]
    rows = [r.randint(0 if b else 1, case["n"]) if case["ragged"] else case["n"] for b in range(case["batch"])]
    return lens, rows


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    c = SimpleNamespace(**case)
    dt = DTYPES[c.dtype]

    def normal(*shape, dtype=dt, scale=1.0):
        return torch.empty(shape, dtype=dtype, device="cuda").normal_(0.0, scale, generator=g)

    lens, rows = lengths(case)
    cols = max(-(-(x + c.n) // c.page) for x in lens)
    # every sequence's pages, scattered over the pool; the pages of a shared prefix come once
    common = c.shared // c.page
    need = torch.tensor([-(-(x + c.n) // c.page) - common for x in lens], device="cuda")
    own_pages = sum(-(-(x + c.n) // c.page) - common for x in lens)
    n_pages = common + own_pages + 3
    perm = torch.randperm(n_pages, generator=g, device="cuda", dtype=torch.int32)
    first = common + torch.cumsum(need, 0) - need
    col = torch.arange(cols, device="cuda")
    idx = torch.where(col[None] < common, col[None], first[:, None] + col[None] - common)
    held = col[None] < (need + common)[:, None]
    table = torch.where(held, perm[idx.clamp(max=n_pages - 1)], torch.zeros((), dtype=torch.int32, device="cuda"))
    k, v = normal(n_pages, c.nkv, c.page, c.hd), normal(n_pages, c.nkv, c.page, c.hd)
    s = {"case": c, "table": table.contiguous(), "k": k, "v": v, "cap": cols * c.page,
         "len": torch.tensor(lens, dtype=torch.int32, device="cuda"),
         "rows": torch.tensor(rows, dtype=torch.int32, device="cuda") if c.ragged else None,
         "shared": torch.tensor([c.shared], dtype=torch.int32, device="cuda")}
    if c.shared % c.page:
        # the page where the prefix ends is each sequence's own: a copy of the first one's
        at = c.shared // c.page
        for pool in (k, v):
            pool[table[:, at].long(), :, :c.shared % c.page] = pool[table[0, at].long(), :, :c.shared % c.page]
    if c.op == "append":
        s["qkv"] = normal(c.batch * c.n, (c.nq + 2 * c.nkv) * c.hd, dtype=DTYPES[c.in_dtype])
        s["q"] = torch.zeros(c.batch, c.n, c.nq, c.hd, dtype=dt, device="cuda")
    else:
        s["q"] = normal(c.batch, c.n, c.nq, c.hd, scale=1.5)
        s["out"] = torch.zeros(c.batch, c.n, c.nq, c.hd, dtype=dt, device="cuda")
    if own:
        from block_diffusion_speculative_target_gb300.engine import PagedCache

        shape = SimpleNamespace(n_layers=1, hidden=c.nq * c.hd, n_q=c.nq, n_kv=c.nkv, head_dim=c.hd, ffn=256, vocab=256,
                                rope_theta=THETA, eps=1e-6)
        s["cache"] = PagedCache(shape, c.dtype, n_pages=n_pages, page_size=c.page, max_pos=s["cap"],
                                max_rows=c.batch * c.n, max_batch=c.batch, k=k, v=v)
    return s


def run(state):
    c = state["case"]
    if own:
        cache = state["cache"]
        if c.op == "append":
            cache.append(0, state["qkv"], state["table"], state["len"], c.n, q_out=state["q"], n_rows=state["rows"])
            return {"q": state["q"], "k": state["k"], "v": state["v"]}
        cache.attention(0, state["q"], state["table"], state["len"], state["out"], causal=c.causal, window=c.window,
                        sinks=c.sinks, n_rows=state["rows"], shared_len=state["shared"] if c.op == "shared" else None)
        return state["out"]
    return _append(state, c) if c.op == "append" else _attend(state, c)


def _append(s, c):
    half = c.hd // 2
    j = torch.arange(c.n, device="cuda")
    pos = s["len"][:, None].long() + j                                      # [batch, n]
    x = s["qkv"].float().view(c.batch, c.n, c.nq + 2 * c.nkv, c.hd)
    # angles of far positions in 64 bits
    inv = THETA ** (-2.0 * torch.arange(half, device="cuda", dtype=torch.float64) / c.hd)
    a = pos[..., None].double() * inv
    cos, sin = a.cos().float()[:, :, None], a.sin().float()[:, :, None]
    lo, hi = x[:, :, :c.nq + c.nkv, :half], x[:, :, :c.nq + c.nkv, half:]
    rot = torch.cat([lo * cos - hi * sin, hi * cos + lo * sin], -1).to(s["q"].dtype)
    val = x[:, :, c.nq + c.nkv:].to(s["q"].dtype)
    live = torch.ones_like(pos, dtype=torch.bool) if s["rows"] is None else j[None] < s["rows"][:, None]
    live = live[..., None, None]
    s["q"].copy_(torch.where(live, rot[:, :, :c.nq], s["q"]))
    page, slot = s["table"].long().gather(1, pos // c.page), pos % c.page
    for pool, new in ((s["k"], rot[:, :, c.nq:]), (s["v"], val)):
        # a padding row's slot is its sequence's own too, and keeps what it held
        tgt = pool[page, :, slot]
        pool.index_put_((page[..., None], torch.arange(c.nkv, device="cuda"), slot[..., None]),
                        torch.where(live, new, tgt))
    return {"q": s["q"], "k": s["k"], "v": s["v"]}


def _attend(s, c):
    G = c.nq // c.nkv
    keys = torch.arange(s["cap"], device="cuda")
    page, slot = s["table"].long()[:, keys // c.page], keys % c.page
    k = s["k"][page, :, slot].float().permute(0, 2, 1, 3)                     # [batch, nkv, keys, hd]
    v = s["v"][page, :, slot].float().permute(0, 2, 1, 3)
    q = s["q"].float().view(c.batch, c.n, c.nkv, G, c.hd).permute(0, 2, 3, 1, 4).reshape(c.batch, c.nkv, G * c.n, c.hd)
    i = torch.arange(c.n, device="cuda")
    rows = s["rows"][:, None] if s["rows"] is not None else torch.full_like(s["len"], c.n)[:, None]
    length = s["len"][:, None]
    pos = length + i                                                         # [batch, n]
    last = pos if c.causal else (length + rows - 1).expand(c.batch, c.n)
    seen = keys <= last[..., None]                                          # [batch, n, keys]
    if c.window:
        first = pos - c.window + 1 if c.causal else (length - c.window).expand(c.batch, c.n)
        seen = seen & ((keys >= first[..., None]) | (keys < c.sinks))
    z = (q @ k.transpose(2, 3) / math.sqrt(c.hd)).view(c.batch, c.nkv, G, c.n, s["cap"])
    z = z.masked_fill(~seen[:, None, None], float("-inf"))
    p = torch.exp(z - z.amax(-1, keepdim=True))
    o = (p.view(c.batch, c.nkv, G * c.n, s["cap"]) @ v).view(c.batch, c.nkv, G, c.n, c.hd) / p.sum(-1, keepdim=True)
    o = o.permute(0, 3, 1, 2, 4).reshape(c.batch, c.n, c.nq, c.hd).to(s["out"].dtype)
    s["out"].copy_(torch.where((i < rows)[..., None, None], o, s["out"]))
    return s["out"]


def _spans(case):
    """Per live row of each sequence: the visible key ranges [0, a) and [b, e), disjoint."""
    lens, rows = lengths(case)
    for P, r in zip(lens, rows):
        got = []
        for i in range(r):
            e = P + i + 1 if case["causal"] else P + r
            b = 0
            if case["window"]:
                b = max(0, P + i - case["window"] + 1 if case["causal"] else P - case["window"])
            got.append((min(case["sinks"], b, e) if case["window"] else 0, b, e))
        yield P, r, got


def work(case):
    size = 2 if case["dtype"] == "bf16" else 4
    nq, nkv, hd = case["nq"], case["nkv"], case["hd"]
    lens, rows = lengths(case)
    if case["op"] == "append":
        in_size = 2 if case["in_dtype"] == "bf16" else 4
        n = sum(rows) * (nq + 2 * nkv) * hd
        return {"bytes": n * (in_size + size), "flops": 6 * sum(rows) * (nq + nkv) * hd // 2}
    held, seen, prefix = 0, 0, set()
    for P, r, got in _spans(case):
        seen += sum(a + e - b for a, b, e in got)
        if not got:
            continue
        a, b, e = max(x[0] for x in got), min(x[1] for x in got), max(x[2] for x in got)
        a = min(a, b)
        s = case["shared"]
        prefix |= {(min(a, s), min(b, s))}
        held += max(0, a - s) + max(0, e - max(b, s))                       # keys of its own that some row sees
    if case["shared"]:
        # of the common keys, those that some row sees: once for all
        a, b = max(x[0] for x in prefix), min(x[1] for x in prefix)
        held += a + case["shared"] - max(a, b) if a < b else case["shared"]
    return {"bytes": 2 * held * nkv * hd * size + 2 * sum(rows) * nq * hd * size, "flops": 4 * seen * nq * hd}


def exact(case, seed):
    """The operators' definitions in 64 bits, a sequence and a head at a time."""
    c = SimpleNamespace(**case)
    lens, rows = lengths(case)
    s = prepare(case, seed)
    out = torch.zeros(c.batch, c.n, c.nq, c.hd, dtype=torch.float64, device="cuda")
    if c.op == "append":
        k, v = s["k"].double(), s["v"].double()
        x = s["qkv"].double().view(c.batch, c.n, -1, c.hd)
        i = torch.arange(c.hd // 2, device="cuda", dtype=torch.float64)
        freq = torch.exp(-math.log(THETA) * 2 * i / c.hd)
        for b in range(c.batch):
            r = rows[b]
            if not r:
                continue
            at = torch.arange(lens[b], lens[b] + r, device="cuda")
            turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"), at[:, None].double() * freq)
            z = torch.complex(x[b, :r, :c.nq + c.nkv, :c.hd // 2], x[b, :r, :c.nq + c.nkv, c.hd // 2:]) * turn[:, None]
            z = torch.cat([z.real, z.imag], -1)
            out[b, :r] = z[:, :c.nq]
            pg = s["table"][b].long()[at // c.page]
            k[pg, :, at % c.page] = z[:, c.nq:]
            v[pg, :, at % c.page] = x[b, :r, c.nq + c.nkv:]
        return {"q": out, "k": k, "v": v}
    G = c.nq // c.nkv
    for b, (P, r, got) in enumerate(_spans(case)):
        if not r:
            continue
        e = max(x[2] for x in got)
        pages = s["table"][b].long()[:-(-e // c.page)]
        at = torch.arange(e, device="cuda")
        hide = torch.stack([(at >= y) | ((at >= a) & (at < f)) for a, f, y in got])
        for h in range(c.nkv):
            kk = s["k"][pages, h].reshape(-1, c.hd)[:e].double()
            vv = s["v"][pages, h].reshape(-1, c.hd)[:e].double()
            for u in range(h * G, (h + 1) * G):
                z = s["q"][b, :r, u].double() @ kk.T * c.hd ** -0.5
                z[hide] = -math.inf
                out[b, :r, u] = torch.softmax(z, 1) @ vv
    return out
