"""Cases that measure a decoder layer's operators on few bits: products with 4-bit
weights and group scales, keys and values quantised to 8 bits as they are
written into pages and read back, and attention over such pages.

``run`` computes an operator in plain torch where ``own`` is false, and makes
the library's calls where it is true.  Shapes are those of the repository's
workloads: hidden 4096 with 32 query and 8 KV heads of 128, hidden 5120 with 40
and 8, the small layouts with one KV head, and the fp32 layout of 4 heads of 64.
"""
import json
import math
import random
from types import SimpleNamespace

import torch

own = False

THETA = 1.0e6
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def _linear(name, rows, m, k, **kw):
    c = {"name": name, "op": "linear", "dtype": "bf16", "rows": rows, "m": m, "k": k, "group": 128, "scales": "bf16",
         "zeros": False, "add": False, "swiglu": False}
    c.update(kw)
    return c


def _pages(name, op, **kw):
    c = {"name": name, "op": op, "dtype": "bf16", "in_dtype": "f32", "nq": 32, "nkv": 8, "hd": 128, "page": 64, "batch": 1,
         "n": 1, "ragged": False, "lo": 0, "hi": 0, "causal": True, "window": 0, "sinks": 0, "shared": 0}
    c.update(kw)
    return c


def listed():
    return [
        # one token through an attention output projection, added to the residual stream: latency
        _linear("w4-token", 1, 4096, 4096, add=True),
        # a verified block's q|k|v rows; zero points, groups of 32, float32 scales
        _linear("w4-block-qkv", 16, 6144, 4096, group=32, scales="f32", zeros=True),
        # a verified block's gate and up rows with the activation
        _linear("w4-block-swiglu", 16, 24576, 4096, group=64, swiglu=True),
        # a block's scores against the whole vocabulary: the most bytes
        _linear("w4-block-head", 15, 151936, 5120),
        # 8 sequences' blocks, or a prefill chunk, through the down projection
        _linear("w4-rows128", 128, 4096, 12288, group=64, zeros=True, add=True),
        # one token's keys and values, quantised on the way into their page, and read back: all latency
        _pages("store8-token", "store", lo=4096, hi=4096),
        # a prefill of 8 prompts, stored and read back
        _pages("store8-prefill", "store", nq=40, in_dtype="bf16", batch=8, n=2048, lo=0, hi=4096, page=128),
        # a 36K context read back, as for moving a sequence out of its pages
        _pages("read8-36k", "read", batch=2, n=36864, ragged=True, page=16),
        # a served batch of single tokens with contexts up to 36K, 5 query heads per KV head
        _pages("attend8-decode32", "attend", nq=40, batch=32, lo=512, hi=36864, page=32),
        # verification of 16-row blocks for 8 ragged sequences
        _pages("attend8-verify8", "attend", batch=8, n=16, lo=2048, hi=6144),
        # a prefill chunk of 128 rows behind 36K keys: products, not bytes
        _pages("attend8-chunk", "attend", nq=40, n=128, lo=36864, hi=36864, page=128),
        # a drafter's non-causal blocks of 8 sequences in a window of 4096 behind 64 first keys; a padded batch
        _pages("attend8-window", "attend", batch=8, n=15, ragged=True, lo=16384, hi=49152, causal=False, window=4096,
               sinks=64, page=16),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    if rng.random() < 0.5:
        f32 = rng.random() < 0.15
        group = rng.choice([32, 64, 128])
        k = group * _log(rng, 1, (1024 if f32 else 25600) // group)
        m = 2 * _log(rng, 1, min(76000, (1 << 20 if f32 else 1 << 28) // k // 2))
        return {"op": "linear", "dtype": "f32" if f32 else "bf16",
                "rows": rng.choice([1, 16, _log(rng, 1, 16), _log(rng, 17, 128)]), "m": m, "k": k, "group": group,
                "scales": rng.choice(["bf16", "f32"]), "zeros": rng.random() < 0.5, "add": rng.random() < 0.4,
                "swiglu": rng.random() < 0.3}
    op = rng.choice(["store", "read", "attend", "attend", "attend"])
    f32 = rng.random() < 0.15
    nq, nkv, hd = rng.choice([(4, 4, 64), (8, 2, 64), (4, 1, 128)]) if f32 else rng.choice(
        [(32, 8, 128), (40, 8, 128), (4, 1, 128), (5, 1, 128), (8, 8, 128), (12, 4, 64), (16, 2, 128)])
    c = {"op": op, "dtype": "f32" if f32 else "bf16", "nq": nq, "nkv": nkv, "hd": hd,
         "page": rng.choice([16, 32, 64, 128]), "ragged": rng.random() < 0.3, "lo": 0, "causal": True, "window": 0,
         "sinks": 0, "shared": 0}
    c["in_dtype"] = "f32" if f32 or rng.random() < 0.5 else "bf16"
    if op in ("store", "read"):
        rows = _log(rng, 1, 16384 if op == "store" else 65536)
        c["batch"] = _log(rng, 1, min(rows, 256))
        c["n"] = max(1, rows // c["batch"])
        c["hi"] = _log(rng, 1, 8192) if op == "store" else 0
        return c
    c["n"] = rng.choice([1, 1, _log(rng, 2, 16), _log(rng, 17, 128)])
    # row-keys budgets keep a drawn case below the largest listed one, for the plain form too
    c["batch"] = _log(rng, 1, 4 if c["n"] > 16 else 48)
    budget = (1 << 17) if f32 else (1 << 19)
    most = min(98304, budget // c["batch"], (1 << 27) // (c["batch"] * c["n"] * nq))
    ctx = _log(rng, 1, max(1, most))
    if c["batch"] > 1 and rng.random() < 0.25:
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
    return _prepare_linear(c, g) if c.op == "linear" else _prepare_pages(case, c, g)


def _normal(g, shape, dtype, scale=1.0):
    return torch.empty(shape, dtype=dtype, device="cuda").normal_(0.0, scale, generator=g)


def _prepare_linear(c, g):
    dt, groups = DTYPES[c.dtype], c.k // c.group
    # two codes a byte, the even column's in the low half
    codes = torch.randint(0, 256, (c.m, c.k // 2), dtype=torch.uint8, device="cuda", generator=g)
    # scales of weights of about 0.02, spread by a factor of three
    scales = torch.empty((c.m, groups), dtype=torch.float32, device="cuda").uniform_(0.002, 0.006, generator=g)
    scales = scales.to(DTYPES[c.scales])
    zeros = torch.randint(5, 11, (c.m, groups), dtype=torch.uint8, device="cuda", generator=g) if c.zeros else None
    out_cols = c.m // 2 if c.swiglu else c.m
    s = {"case": c, "codes": codes, "scales": scales, "zeros": zeros, "x": _normal(g, (c.rows, c.k), dt),
         "add": _normal(g, (c.rows, c.m), torch.float32) if c.add else None,
         "out": torch.zeros((c.rows, out_cols), dtype=dt if c.swiglu else torch.float32, device="cuda")}
    if own:
        from block_diffusion_speculative_target_gb300.engine import W4Linear, W4Workspace

        s["w4"] = W4Linear.from_codes(codes, scales, zeros)
        s["ws"] = W4Workspace(max_rows=c.rows)
    return s


def _prepare_pages(case, c, g):
    dt = DTYPES[c.dtype]
    lens, rows = lengths(case)
    # every sequence's pages, scattered over the pool; the pages of a shared prefix come once
    cols = max(-(-(x + c.n) // c.page) for x in lens)
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
    # rows of normal entries hold codes of a standard deviation near 127 / 2.7 and scales near 2.7 / 127
    dims = (n_pages, c.nkv, c.page, c.hd)
    pool = {}
    for name in ("k", "v"):
        x = _normal(g, dims, torch.bfloat16, 47.0).round_().clamp_(-127, 127)
        pool[name] = x.add_(128).to(torch.uint8)
        pool[name + "_scale"] = torch.empty(dims[:3], dtype=torch.float32, device="cuda").uniform_(0.017, 0.026, generator=g)
    s = {"case": c, "table": table.contiguous(), "cap": cols * c.page, **pool,
         "len": torch.tensor(lens, dtype=torch.int32, device="cuda"),
         "rows": torch.tensor(rows, dtype=torch.int32, device="cuda") if c.ragged else None,
         "shared": torch.tensor([c.shared], dtype=torch.int32, device="cuda")}
    if c.shared % c.page:
        # the page where the prefix ends is each sequence's own: a copy of the first one's
        at, upto = c.shared // c.page, c.shared % c.page
        for p in pool.values():
            p[table[:, at].long(), :, :upto] = p[table[0, at].long(), :, :upto]
    if c.op == "attend":
        s["q"] = _normal(g, (c.batch, c.n, c.nq, c.hd), dt, 1.5)
        s["out"] = torch.zeros((c.batch, c.n, c.nq, c.hd), dtype=dt, device="cuda")
    else:
        s["k_out"], s["v_out"] = (torch.zeros((c.batch, c.nkv, c.n, c.hd), dtype=dt, device="cuda") for _ in range(2))
    if c.op == "store":
        s["qkv"] = _normal(g, (c.batch * c.n, (c.nq + 2 * c.nkv) * c.hd), DTYPES[c.in_dtype])
        s["q"] = torch.zeros((c.batch, c.n, c.nq, c.hd), dtype=dt, device="cuda")
    if own:
        from block_diffusion_speculative_target_gb300.engine import PagedCache

        shape = SimpleNamespace(n_layers=1, hidden=c.nq * c.hd, n_q=c.nq, n_kv=c.nkv, head_dim=c.hd, ffn=256, vocab=256,
                                rope_theta=THETA, eps=1e-6)
        s["cache"] = PagedCache(shape, c.dtype, n_pages=n_pages, page_size=c.page, max_pos=s["cap"],
                                max_rows=c.batch * (c.n if c.op == "attend" else 1), max_batch=c.batch, kv_format="q8",
                                **pool)
    return s


def run(state):
    c = state["case"]
    if own:
        if c.op == "linear":
            state["w4"].product(state["x"], state["out"], state["ws"], add=state["add"], swiglu=c.swiglu)
            return state["out"]
        cache = state["cache"]
        if c.op == "attend":
            cache.attention(0, state["q"], state["table"], state["len"], state["out"], causal=c.causal, window=c.window,
                            sinks=c.sinks, n_rows=state["rows"], shared_len=state["shared"] if c.shared else None)
            return state["out"]
        if c.op == "store":
            cache.append(0, state["qkv"], state["table"], state["len"], c.n, q_out=state["q"], n_rows=state["rows"])
        cache.read(0, state["table"], state["len"], state["k_out"], state["v_out"], n_rows=state["rows"])
        return _held(state, c)
    if c.op == "linear":
        return _product(state, c)
    if c.op == "attend":
        return _attend(state, c)
    if c.op == "store":
        _append(state, c)
    return _read(state, c)


def _held(s, c):
    """What a store or a read returns: the entries as the values that their codes stand for, and the scales."""
    out = {"k": s["k_out"], "v": s["v_out"]}
    return {**out, "q": s["q"], "k_scale": s["k_scale"], "v_scale": s["v_scale"]} if c.op == "store" else out


def _product(s, c):
    code = torch.stack([s["codes"] & 15, s["codes"] >> 4], -1).view(c.m, c.k // c.group, c.group).float()
    code -= 8.0 if s["zeros"] is None else s["zeros"][..., None].float()
    w = (code * s["scales"].float()[..., None]).view(c.m, c.k)
    y = s["x"].float() @ w.T
    if c.add:
        y = y + s["add"]
    if c.swiglu:
        gate, up = y[:, 0::2], y[:, 1::2]
        y = gate / (1.0 + torch.exp(-gate)) * up
    return s["out"].copy_(y)


def _live(s, c):
    j = torch.arange(c.n, device="cuda")
    return torch.ones((c.batch, c.n), dtype=torch.bool, device="cuda") if s["rows"] is None else j < s["rows"][:, None]


def _append(s, c):
    half = c.hd // 2
    pos = s["len"][:, None].long() + torch.arange(c.n, device="cuda")         # [batch, n]
    x = s["qkv"].float().view(c.batch, c.n, c.nq + 2 * c.nkv, c.hd)
    # angles of far positions in 64 bits
    inv = THETA ** (-2.0 * torch.arange(half, device="cuda", dtype=torch.float64) / c.hd)
    a = pos[..., None].double() * inv
    cos, sin = a.cos().float()[:, :, None], a.sin().float()[:, :, None]
    lo, hi = x[:, :, :c.nq + c.nkv, :half], x[:, :, :c.nq + c.nkv, half:]
    rot = torch.cat([lo * cos - hi * sin, hi * cos + lo * sin], -1)
    live = _live(s, c)[..., None, None]
    s["q"].copy_(torch.where(live, rot[:, :, :c.nq].to(s["q"].dtype), s["q"]))
    page, slot = s["table"].long().gather(1, pos // c.page), pos % c.page
    at = (page[..., None], torch.arange(c.nkv, device="cuda"), slot[..., None])
    steps = torch.full((), 127.0, device="cuda")  # (a division by a Python number is a product with its inverse)
    for name, new in (("k", rot[:, :, c.nq:]), ("v", x[:, :, c.nq + c.nkv:])):
        scale = new.abs().amax(-1, keepdim=True) / steps
        code = (torch.round(new / scale).clamp(-127, 127) + 128.0).to(torch.uint8)
        # a padding row's slot is its sequence's own too, and keeps what it held
        s[name].index_put_(at, torch.where(live, code, s[name][at]))
        s[name + "_scale"].index_put_(at, torch.where(live[..., 0], scale[..., 0], s[name + "_scale"][at]))


def _rows_of(s, pos, c):
    """Keys and values of positions [batch, n] in float32: [batch, nkv, n, hd]."""
    page, slot = s["table"].long().gather(1, pos // c.page), pos % c.page
    return [(s[x][page, :, slot].float().sub_(128.0) * s[x + "_scale"][page, :, slot][..., None]).transpose(1, 2)
            for x in ("k", "v")]


def _read(s, c):
    pos = s["len"][:, None].long() + torch.arange(c.n, device="cuda")
    live = _live(s, c)[:, None, :, None]
    for out, new in zip((s["k_out"], s["v_out"]), _rows_of(s, pos, c)):
        out.copy_(torch.where(live, new.to(out.dtype), out))
    return _held(s, c)


def _attend(s, c):
    G = c.nq // c.nkv
    keys = torch.arange(s["cap"], device="cuda")
    k, v = _rows_of(s, keys.expand(c.batch, -1), c)                           # [batch, nkv, keys, hd]
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
    return s["out"].copy_(torch.where((i < rows)[..., None, None], o, s["out"]))


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
    if case["op"] == "linear":
        m, k, rows, groups = case["m"], case["k"], case["rows"], case["k"] // case["group"]
        weights = m * k // 2 + m * groups * ((2 if case["scales"] == "bf16" else 4) + case["zeros"])
        out = rows * m // 2 * size if case["swiglu"] else rows * m * 4
        return {"bytes": weights + rows * k * size + out + rows * m * 4 * case["add"], "flops": 2 * rows * m * k}
    nq, nkv, hd = case["nq"], case["nkv"], case["hd"]
    lens, rows = lengths(case)
    entry = 2 * nkv * (hd + 4)                                                # a position's codes and scales
    if case["op"] == "read":
        return {"bytes": sum(rows) * (entry + 2 * nkv * hd * size), "flops": sum(rows) * 2 * nkv * hd}
    if case["op"] == "store":
        in_size = 2 if case["in_dtype"] == "bf16" else 4
        return {"bytes": sum(rows) * ((nq + 2 * nkv) * hd * in_size + nq * hd * size + entry + 2 * nkv * hd * size),
                "flops": sum(rows) * hd * (3 * (nq + nkv) + 8 * nkv)}
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
    return {"bytes": held * entry + 2 * sum(rows) * nq * hd * size, "flops": 4 * seen * nq * hd}


def exact(case, seed):
    """The operators' definitions in 64 bits: a slice of weight rows at a time, a sequence and a head at a time."""
    c = SimpleNamespace(**case)
    s = prepare(case, seed)
    if c.op == "linear":
        return _exact_product(s, c)
    lens, rows = lengths(case)
    if c.op == "attend":
        return _exact_attend(s, c, case)
    k, v = (torch.zeros((c.batch, c.nkv, c.n, c.hd), dtype=torch.float64, device="cuda") for _ in range(2))
    q = torch.zeros((c.batch, c.n, c.nq, c.hd), dtype=torch.float64, device="cuda")
    ks, vs = s["k_scale"].double(), s["v_scale"].double()
    i = torch.arange(c.hd // 2, device="cuda", dtype=torch.float64)
    freq = torch.exp(-math.log(THETA) * 2 * i / c.hd)
    for b in range(c.batch):
        r = rows[b]
        if not r:
            continue
        at = torch.arange(lens[b], lens[b] + r, device="cuda")
        pg = s["table"][b].long()[at // c.page]
        if c.op == "read":
            for out, x in ((k, "k"), (v, "v")):
                held = s[x][pg, :, at % c.page].double() - 128
                out[b, :, :r] = (held * s[x + "_scale"][pg, :, at % c.page].double()[..., None]).transpose(0, 1)
            continue
        x = s["qkv"].double().view(c.batch, c.n, -1, c.hd)[b, :r]
        turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"), at[:, None].double() * freq)
        z = torch.complex(x[:, :c.nq + c.nkv, :c.hd // 2], x[:, :c.nq + c.nkv, c.hd // 2:]) * turn[:, None]
        z = torch.cat([z.real, z.imag], -1)
        q[b, :r] = z[:, :c.nq]
        for out, scales, new in ((k, ks, z[:, c.nq:]), (v, vs, x[:, c.nq + c.nkv:])):
            step = new.abs().amax(-1) / 127
            scales[pg, :, at % c.page] = step
            out[b, :, :r] = (torch.round(new / step[..., None]) * step[..., None]).transpose(0, 1)
    return {"k": k, "v": v, "q": q, "k_scale": ks, "v_scale": vs} if c.op == "store" else {"k": k, "v": v}


def _exact_product(s, c):
    y = torch.empty((c.rows, c.m), dtype=torch.float64, device="cuda")
    x = s["x"].double()
    per = max(1, (1 << 27) // c.k)
    for m in range(0, c.m, per):
        byte = s["codes"][m:m + per].to(torch.int16)
        w = torch.empty((byte.shape[0], c.k), dtype=torch.float64, device="cuda")
        w[:, 0::2], w[:, 1::2] = byte % 16, byte // 16
        zero = 8 if s["zeros"] is None else s["zeros"][m:m + per].double().repeat_interleave(c.group, 1)
        w = (w - zero) * s["scales"][m:m + per].double().repeat_interleave(c.group, 1)
        y[:, m:m + per] = x @ w.T
    if c.add:
        y += s["add"].double()
    if not c.swiglu:
        return y
    return torch.nn.functional.silu(y[:, 0::2]) * y[:, 1::2]


def _exact_attend(s, c, case):
    out = torch.zeros((c.batch, c.n, c.nq, c.hd), dtype=torch.float64, device="cuda")
    G = c.nq // c.nkv
    for b, (P, r, got) in enumerate(_spans(case)):
        if not r:
            continue
        e = max(x[2] for x in got)
        pages = s["table"][b].long()[:-(-e // c.page)]
        at = torch.arange(e, device="cuda")
        hide = torch.stack([(at >= y) | ((at >= a) & (at < f)) for a, f, y in got])
        for h in range(c.nkv):
            kk, vv = (((s[x][pages, h].double() - 128) * s[x + "_scale"][pages, h].double()[..., None]
                       ).reshape(-1, c.hd)[:e] for x in ("k", "v"))
            for u in range(h * G, (h + 1) * G):
                z = s["q"][b, :r, u].double() @ kk.T * c.hd ** -0.5
                z[hide] = -math.inf
                out[b, :r, u] = torch.softmax(z, 1) @ vv
    return out
