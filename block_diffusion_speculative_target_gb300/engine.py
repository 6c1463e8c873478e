"""Device-resident DFlash models and decoding sessions over the C ABI.

``Model`` owns the target's and the drafter's weights in the library's packed
layouts (q|k|v rows in one matrix, gate/up rows interleaved, the drafter's
k|v rows of every layer gathered for one injection product) and exposes each
canonical matrix as a view for loading.  ``Session`` owns the KV caches, the
workspace and the per-sequence device state, and sequences the stages:

    prefill (chunks of <= 128 rows): target_verify(commit) -> fuse -> inject
    step: fuse -> inject -> draft -> [teacher force] -> verify -> accept/rollback

Every stage is one call into libdflash.so; nothing here computes.
"""
from __future__ import annotations

import ctypes

import numpy as np
import torch

from . import capi

_DT = {"f32": (capi.F32, torch.float32), "bf16": (capi.BF16, torch.bfloat16)}
LAYER_PARTS = ("attn_norm", "wq", "wk", "wv", "wo", "ffn_norm", "w_gate", "w_up", "w_down")


def desc_of(shape, dtype: str, n_layers=None) -> capi.ModelDesc:
    return capi.ModelDesc(n_layers if n_layers is not None else shape.n_layers, shape.hidden, shape.n_q, shape.n_kv,
                          shape.head_dim, shape.ffn, shape.vocab, shape.rope_theta, shape.eps, _DT[dtype][0])


def _raw_stream(index):
    """The current stream of a device as the handle that the C ABI takes (torch.cuda.current_stream() makes a Stream
    object for it, 3 us)."""
    return torch._C._cuda_getCurrentRawStream(index)


class Model:
    """Target + drafter weights on the GPU.  ``shape`` has the fields n_layers,
    hidden, n_q, n_kv, head_dim, ffn, vocab, rope_theta, eps; the drafter has
    the target's width and ``draft_layers`` layers."""

    def __init__(self, shape, draft_layers: int, dtype: str, device="cuda", cross_ctx: int = 0):
        self.shape, self.draft_layers, self.dtype = shape, draft_layers, dtype
        self.cross_ctx = cross_ctx  # the drafter's cross-context window (0: whole context)
        self.device = torch.device(device)
        tdt = _DT[dtype][1]
        s = shape
        H, d, F, V = s.hidden, s.head_dim, s.ffn, s.vocab

        def alloc(*sh):
            return torch.empty(sh, dtype=tdt, device=self.device)

        def layer():
            return {"attn_norm": alloc(H), "wqkv": alloc((s.n_q + 2 * s.n_kv) * d, H), "wo": alloc(H, s.n_q * d),
                    "ffn_norm": alloc(H), "w_gate_up": alloc(2 * F, H), "w_down": alloc(H, F)}

        self.embed, self.final_norm, self.lm_head = alloc(V, H), alloc(H), alloc(V, H)
        self.layers = [layer() for _ in range(s.n_layers)]
        self.w_fc, self.fc_norm, self.d_final_norm = alloc(H, 5 * H), alloc(H), alloc(H)
        self.dlayers = [layer() for _ in range(draft_layers)]
        self.w_kv_all = alloc(draft_layers * 2 * s.n_kv * d, H)
        self.capture = capi.dflash_capture_layers(s.n_layers)
        self.mask_id = V - 1
        self._structs = None

    # -------------------------------------------------------------- loading
    def _layer_views(self, lw):
        s, d = self.shape, self.shape.head_dim
        q, kv = s.n_q * d, s.n_kv * d
        return {"attn_norm": lw["attn_norm"], "wq": lw["wqkv"][:q], "wk": lw["wqkv"][q:q + kv],
                "wv": lw["wqkv"][q + kv:], "wo": lw["wo"], "ffn_norm": lw["ffn_norm"],
                "w_gate": lw["w_gate_up"][0::2], "w_up": lw["w_gate_up"][1::2], "w_down": lw["w_down"]}

    def views(self):
        """Canonical name -> view of the packed storage."""
        out = {"embed": self.embed, "final_norm": self.final_norm, "lm_head": self.lm_head,
               "draft.w_fc": self.w_fc, "draft.fc_norm": self.fc_norm, "draft.final_norm": self.d_final_norm}
        for i, lw in enumerate(self.layers):
            for k, v in self._layer_views(lw).items():
                out[f"layers.{i}.{k}"] = v
        for i, lw in enumerate(self.dlayers):
            for k, v in self._layer_views(lw).items():
                out[f"draft.layers.{i}.{k}"] = v
        return out

    def load(self, weights: dict):
        """Copy host arrays (canonical names) into the packed device storage."""
        views = self.views()
        for name, arr in weights.items():
            v = views[name]
            t = torch.from_numpy(np.ascontiguousarray(arr)).to(dtype=v.dtype)
            v.copy_(t.reshape(v.shape))
        self.finalize()

    def set_cross_ctx(self, window: int):
        """Set the drafter's cross-context window (0: whole context)."""
        self.cross_ctx = int(window)
        self._structs = None

    def finalize(self):
        """Gather the drafter's k/v rows for the injection product and build
        the C structs.  Call after every change of the weights."""
        s, d = self.shape, self.shape.head_dim
        q, kv = s.n_q * d, s.n_kv * d
        for i, lw in enumerate(self.dlayers):
            self.w_kv_all[i * 2 * kv:(i + 1) * 2 * kv].copy_(lw["wqkv"][q:q + 2 * kv])
        self._structs = None

    def weight_bytes(self):
        t = sum(x.numel() * x.element_size() for x in (self.embed, self.final_norm, self.lm_head))
        t += sum(x.numel() * x.element_size() for lw in self.layers for x in lw.values())
        dr = sum(x.numel() * x.element_size() for lw in self.dlayers for x in lw.values())
        dr += sum(x.numel() * x.element_size() for x in (self.w_fc, self.fc_norm, self.d_final_norm, self.w_kv_all))
        return t, dr

    # -------------------------------------------------------------- C structs
    def _layer_array(self, layers):
        arr = (capi.LayerW * len(layers))()
        for i, lw in enumerate(layers):
            arr[i] = capi.LayerW(*(lw[k].data_ptr() for k in ("attn_norm", "wqkv", "wo", "ffn_norm", "w_gate_up",
                                                              "w_down")))
        return arr

    def structs(self):
        if self._structs is None:
            tl = self._layer_array(self.layers)
            dl = self._layer_array(self.dlayers)
            tgt = capi.TargetC(desc_of(self.shape, self.dtype), self.embed.data_ptr(), self.final_norm.data_ptr(),
                               self.lm_head.data_ptr(), ctypes.cast(tl, ctypes.POINTER(capi.LayerW)),
                               (ctypes.c_int32 * 5)(*self.capture))
            dr = capi.DraftC(desc_of(self.shape, self.dtype, self.draft_layers), self.w_fc.data_ptr(),
                             self.fc_norm.data_ptr(), self.d_final_norm.data_ptr(),
                             ctypes.cast(dl, ctypes.POINTER(capi.LayerW)), self.w_kv_all.data_ptr(), self.mask_id,
                             self.cross_ctx)
            self._structs = (tgt, dr, tl, dl)  # keep the layer arrays alive
        return self._structs[0], self._structs[1]


class Session:
    """Caches, workspace and device state for ``batch`` sequences."""

    def __init__(self, model: Model, batch=1, capacity=1024, block=16, prefill_chunk=128, stream_cap=None,
                 with_draft=True, tree_budget=0, kv_format="bf16"):
        tree_n = tree_budget + 1 if tree_budget else 0
        if batch * max(block, tree_n) > 128 or prefill_chunk > 128 or tree_n > 64:
            raise ValueError("at most 128 rows per call and 64 tree nodes")
        if kv_format not in ("bf16", "q8"):
            raise ValueError(kv_format)
        self.kv_format = kv_format
        if kv_format == "q8":
            capacity = (capacity + 7) // 8 * 8  # the 8-bit cache's capacity granularity
        self.m, self.batch, self.block, self.capacity = model, batch, block, capacity
        self.chunk = prefill_chunk
        self.stream_cap = stream_cap or capacity
        s = model.shape
        self.tdesc = desc_of(s, model.dtype)
        self.ddesc = desc_of(s, model.dtype, model.draft_layers)
        dev = model.device
        tdt = _DT[model.dtype][1]
        self.tcache = capi.dflash_cache_alloc_ex(self.tdesc, s.n_layers, batch, capacity,
                                                 capi.KV_Q8 if kv_format == "q8" else capi.KV_MODEL)
        self.dcache = capi.dflash_cache_alloc(self.ddesc, model.draft_layers, batch, capacity) if with_draft else None
        self.max_rows = max(batch * block, batch * tree_n, prefill_chunk)
        self.ws = capi.dflash_workspace_alloc(self.tdesc, self.ddesc if with_draft else None, self.max_rows, capacity)
        i32 = dict(dtype=torch.int32, device=dev)
        self.anchor = torch.zeros(batch, **i32)
        self.n_pend = torch.zeros(batch, **i32)
        self.accept_len = torch.zeros(batch, **i32)
        self.draft = torch.zeros(batch, block, **i32)
        self.argmax = torch.zeros(self.max_rows, **i32)
        self.gap = torch.zeros(self.max_rows, dtype=torch.float32, device=dev)
        self.hcap = torch.zeros(self.max_rows, 5 * s.hidden, dtype=tdt, device=dev)
        self.fused = torch.zeros(self.max_rows, s.hidden, dtype=tdt, device=dev)
        self.stream = torch.full((batch, self.stream_cap), -1, **i32)
        self.stream_len = torch.zeros(batch, **i32)
        self.step_ctr = torch.zeros(1, **i32)
        self.ref = self.k_draw = self.r_draw = None
        self.steps_done = 0
        self.rps = block  # rows per sequence of the last verification (the layout of hcap)
        if tree_n:
            self.tree_budget, self.tree_n = tree_budget, tree_n
            self.tree_tokens = torch.zeros(batch, tree_n, **i32)
            self.tree_parent = torch.zeros(batch, tree_n, **i32)
            self.tree_depth = torch.zeros(batch, tree_n, **i32)
            self.tree_mask = torch.zeros(batch, tree_n, dtype=torch.int64, device=dev)  # uint64 bit masks

    def close(self):
        for h, f in ((self.tcache, capi.dflash_cache_free), (self.dcache, capi.dflash_cache_free),
                     (self.ws, capi.dflash_workspace_free)):
            if h:
                f(h)
        self.tcache = self.dcache = self.ws = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    # -------------------------------------------------------------- state
    def target_len(self):
        return capi.dflash_cache_get_lengths(self.tcache, self.batch)

    def draft_len(self):
        return capi.dflash_cache_get_lengths(self.dcache, self.batch)

    def emitted(self):
        torch.cuda.synchronize()
        lens = self.stream_len.cpu().numpy()
        st = self.stream.cpu().numpy()
        return [st[b, :lens[b]].copy() for b in range(self.batch)]

    def status(self):
        return capi.dflash_status(self.ws)

    # -------------------------------------------------------------- prefill
    def prefill(self, prompts, inject=True):
        """Run the target over each sequence's prompt (chunks of <= 128 rows),
        cache its keys/values, emit the first greedy token, and inject every
        prompt row into the drafter cache."""
        tgt, dr = self.m.structs()
        dev = self.m.device
        for b, p in enumerate(prompts):
            toks = torch.as_tensor(np.asarray(p, dtype=np.int32), device=dev)
            tv = capi.dflash_cache_view(self.tcache, b, 1)
            dv = capi.dflash_cache_view(self.dcache, b, 1) if (inject and self.dcache) else None
            try:
                for c0 in range(0, len(p), self.chunk):
                    n = min(self.chunk, len(p) - c0)
                    last = c0 + n == len(p)
                    if last:
                        self._last_chunk_rows = n
                    capi.target_verify(tgt, toks[c0:c0 + n], 1, n, 2 if last else 1, tv, self.argmax, self.gap,
                                       self.hcap if dv else None, self.anchor[b:], self.n_pend[b:],
                                       self.stream[b], self.stream_len[b:], self.stream_cap, self.ws)
                    if dv:
                        capi.dflash_fuse_features(dr, self.hcap, n, self.fused, self.ws)
                        capi.dflash_inject_kv(dr, self.fused, 1, n, self.n_pend[b:], dv, self.ws)
            finally:
                capi.dflash_cache_free(tv)
                if dv:
                    capi.dflash_cache_free(dv)

    def copy_target_from(self, other: "Session"):
        """Take over another session's committed target state (keys/values of
        positions 0..len-1 of every layer, lengths, anchors and emitted
        streams) instead of prefilling the same prompts again."""
        if (other.capacity, other.batch, other.kv_format) == (self.capacity, self.batch, self.kv_format):
            capi.dflash_cache_copy(self.tcache, other.tcache)  # the whole cache in a few copies
        else:
            if self.kv_format != "bf16" or other.kv_format != "bf16":
                raise ValueError("8-bit caches are copied whole, between sessions of the same geometry")
            s = self.m.shape
            lens = other.target_len()
            tdt = _DT[self.m.dtype][1]
            for b, n in enumerate(lens):
                if n == 0:
                    continue
                k = torch.empty(s.n_kv, n, s.head_dim, dtype=tdt, device=self.m.device)
                v = torch.empty_like(k)
                for li in range(s.n_layers):
                    capi.dflash_cache_read(other.tcache, li, b, 0, n, k, v)
                    capi.dflash_cache_write(self.tcache, li, b, 0, n, k, v)
            capi.dflash_cache_set_lengths(self.tcache, lens)
        self.anchor.copy_(other.anchor)
        w = min(self.stream_cap, other.stream_cap)
        self.stream[:, :w].copy_(other.stream[:, :w])
        self.stream_len.copy_(other.stream_len)
        torch.cuda.synchronize()

    # -------------------------------------------------------------- decoding
    def set_teacher(self, ref, k_draw, r_draw):
        """Teacher-forcing inputs: ref [batch][L] greedy streams, draws [steps][batch]."""
        dev = self.m.device
        self.ref = torch.as_tensor(np.ascontiguousarray(ref, dtype=np.int32), device=dev)
        self.k_draw = torch.as_tensor(np.ascontiguousarray(k_draw, dtype=np.int32), device=dev)
        self.r_draw = torch.as_tensor(np.ascontiguousarray(r_draw, dtype=np.int32), device=dev)
        self.step_ctr.zero_()

    def step(self, teacher=False):
        """One DFlash step for every sequence (asynchronous)."""
        tgt, dr = self.m.structs()
        B = self.block
        capi.dflash_fuse_features(dr, self.hcap, self.batch * self.rps, self.fused, self.ws)
        capi.dflash_inject_kv(dr, self.fused, self.batch, self.rps, self.n_pend, self.dcache, self.ws)
        capi.dflash_draft_block(dr, tgt, self.anchor, self.batch, B, self.dcache, self.draft, self.ws)
        self.rps = B
        if teacher:
            capi.dflash_teacher_force(self.draft, self.batch, B, self.ref, self.ref.shape[1], self.ref.shape[1],
                                      self.stream_len, self.k_draw, self.r_draw, self.k_draw.shape[0], self.step_ctr,
                                      self.m.shape.vocab, self.ws)
        capi.target_verify(tgt, self.draft, self.batch, B, 0, self.tcache, self.argmax, self.gap, self.hcap, None,
                           None, None, None, 0, self.ws)
        capi.dflash_accept_rollback(self.draft, self.argmax, self.batch, B, self.tcache, self.anchor, self.n_pend,
                                    self.accept_len, self.stream, self.stream_len, self.stream_cap, self.ws)
        self.steps_done += 1

    def resample_first(self, temperature, v):
        """Sampling mode after prefill: replace each sequence's first emitted
        token (the greedy one) by a draw at `temperature` from the last
        prompt row's logits with the uniform v[batch].  Needs the prefill's
        last chunk to be its only call with that sequence's last row, i.e. a
        single sequence (batch 1)."""
        if self.batch != 1:
            raise ValueError("resample_first draws from the last prefill call's logits: batch 1 only")
        n_last = int(self._last_chunk_rows)
        logits = capi.dflash_workspace_logits(self.ws, n_last, self.m.shape.vocab)[n_last - 1:]
        vv = torch.as_tensor(np.asarray(v, dtype=np.float32).reshape(1), device=self.m.device)
        capi.dflash_sample(logits, 1, self.m.shape.vocab, temperature, vv, self.anchor, self.ws)
        self.stream[:, 0].copy_(self.anchor)

    def step_sampling(self, temperature, w, u, v):
        """One DFlash step in sampling mode (asynchronous): the drafter samples
        its block with w [batch][B-1], the target verifies it by speculative
        sampling with u [batch][B-1] and v [batch] (device float32 uniforms)."""
        tgt, dr = self.m.structs()
        B, V = self.block, self.m.shape.vocab
        capi.dflash_fuse_features(dr, self.hcap, self.batch * self.rps, self.fused, self.ws)
        capi.dflash_inject_kv(dr, self.fused, self.batch, self.rps, self.n_pend, self.dcache, self.ws)
        capi.dflash_draft_block(dr, tgt, self.anchor, self.batch, B, self.dcache, self.draft, self.ws)
        self.rps = B
        capi.dflash_draft_sample(self.batch, B, V, temperature, w, self.draft, self.ws)
        capi.target_verify(tgt, self.draft, self.batch, B, 0, self.tcache, self.argmax, self.gap, self.hcap, None,
                           None, None, None, 0, self.ws)
        capi.dflash_accept_sample(self.draft, self.batch, B, V, temperature, u, v, self.tcache, self.anchor,
                                  self.n_pend, self.accept_len, self.stream, self.stream_len, self.stream_cap, self.ws)
        self.steps_done += 1

    def step_tree(self, topk):
        """One DFlash step with tree verification (asynchronous): the drafter's
        block, the tree of its top-k candidates within the session's budget,
        one ancestor-masked target forward over the tree, the walk and the
        compaction of the accepted path."""
        tgt, dr = self.m.structs()
        B, V, n = self.block, self.m.shape.vocab, self.tree_n
        capi.dflash_fuse_features(dr, self.hcap, self.batch * self.rps, self.fused, self.ws)
        capi.dflash_inject_kv(dr, self.fused, self.batch, self.rps, self.n_pend, self.dcache, self.ws)
        capi.dflash_draft_block(dr, tgt, self.anchor, self.batch, B, self.dcache, self.draft, self.ws)
        capi.dflash_draft_tree(self.anchor, self.batch, B, V, topk, self.tree_budget, self.tree_tokens,
                               self.tree_parent, self.tree_depth, self.tree_mask, self.ws)
        capi.target_verify_tree(tgt, self.tree_tokens, self.tree_depth, self.tree_mask, self.batch, n, self.tcache,
                                self.argmax, self.gap, self.hcap, self.ws)
        capi.dflash_accept_tree(tgt, self.tree_tokens, self.tree_parent, self.argmax, self.batch, n, self.tcache,
                                self.hcap, self.anchor, self.n_pend, self.accept_len, self.stream, self.stream_len,
                                self.stream_cap, self.ws)
        self.rps = n
        self.steps_done += 1

    def ar_step(self):
        """One greedy autoregressive token per sequence: the target forward of
        the anchor, committed."""
        tgt, _ = self.m.structs()
        capi.target_verify(tgt, self.anchor, self.batch, 1, 2, self.tcache, self.argmax, self.gap, None, self.anchor,
                           self.n_pend, self.stream, self.stream_len, self.stream_cap, self.ws)

    def capture_graph(self, fn):
        """Capture ``fn()`` (a step) into a CUDA graph; replay with g.replay()."""
        g = torch.cuda.CUDAGraph()
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.graph(g, stream=s):
            fn()
        torch.cuda.current_stream().wait_stream(s)
        return g


class PagedCache:
    """A pool of KV pages with the append and attention calls on it.

    ``shape`` and ``dtype`` as for ``Model``.  The pool is two tensors ``k`` and
    ``v`` [n_layers][n_pages][n_kv][page_size][head_dim]; pass them (a 4-d pair
    is one layer) or leave them out to have zeroed ones made.  With ``kv_format``
    "q8" they hold uint8 codes, and ``k_scale`` and ``v_scale``
    [n_layers][n_pages][n_kv][page_size] the rows' float32 scales: ``append``
    quantises, ``attention`` and ``read`` take entries as (code - 128) * scale,
    queries and results stay in ``dtype``.  Tables, lengths
    and row counts are the caller's device int32 tensors: ``table``
    [batch][columns] names the page of each ``page_size`` positions, ``lengths``
    [batch] the positions held before a call's rows, ``n_rows`` [batch] the rows
    of each sequence in the call (None: all).  Calls enter the pool's device,
    are asynchronous on its current stream and leave ``lengths`` as it is."""

    def __init__(self, shape, dtype: str, n_pages, page_size, max_pos, max_rows, max_batch=None, n_layers=1, k=None,
                 v=None, device="cuda", kv_format="model", k_scale=None, v_scale=None):
        if kv_format not in ("model", "q8"):
            raise ValueError(kv_format)
        q8 = kv_format == "q8"
        self.dtype, self.tdt, self.kv_format = dtype, _DT[dtype][1], kv_format
        kdt = torch.uint8 if q8 else self.tdt
        self.nq, self.nkv, self.hd = shape.n_q, shape.n_kv, shape.head_dim
        self.page_size, self.max_pos = page_size, max_pos
        self.pages = self.ws = None
        dims = (n_layers, n_pages, self.nkv, page_size, self.hd)
        pools = {"k": k, "v": v}
        if q8:
            pools.update(k_scale=k_scale, v_scale=v_scale)
        elif k_scale is not None or v_scale is not None:
            raise ValueError('scales belong to kv_format "q8"')
        if len({t is None for t in pools.values()}) != 1:
            raise ValueError("pass both pools (with their scales) or none")
        for name in pools:
            t, pdt, pdims = pools[name], torch.float32 if "scale" in name else kdt, dims[:4] if "scale" in name else dims
            if t is None:
                # (code 128 is 0)
                t = pools[name] = torch.full(pdims, 128 if pdt == torch.uint8 else 0, dtype=pdt, device=device)
            if t.dtype != pdt or not t.is_cuda or not t.is_contiguous() or \
                    tuple(t.shape) != (pdims if t.dim() == len(pdims) else pdims[1:]) or \
                    (t.dim() != len(pdims) and n_layers != 1):
                raise ValueError(f"a pool is a contiguous {pdt} tensor {pdims} on the GPU")
        self.k, self.v, self.device = pools["k"], pools["v"], pools["k"].device
        self.k_scale, self.v_scale = pools.get("k_scale"), pools.get("v_scale")
        if any(t.device != self.device for t in pools.values()):
            raise ValueError("the pools are on different devices")
        desc = desc_of(shape, dtype, n_layers)
        with torch.cuda.device(self.device):
            if q8:
                self.pages = capi.dflash_pages_create_q8(desc, n_layers, n_pages, page_size, max_pos, self.k, self.v,
                                                         self.k_scale, self.v_scale)
            else:
                self.pages = capi.dflash_pages_create(desc, n_layers, n_pages, page_size, max_pos, self.k, self.v)
            self.ws = capi.dflash_paged_workspace_alloc(desc, max_batch or max_rows, max_rows)

    def close(self):
        """Frees the handle and the workspace (the pool is torch's).  Work of
        the calls made so far has to be done."""
        if self.pages:
            capi.dflash_pages_free(self.pages)
        if self.ws:
            capi.dflash_paged_workspace_free(self.ws)
        self.pages = self.ws = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def status(self):
        with torch.cuda.device(self.device):
            return capi.dflash_paged_status(self.ws)

    def _index(self, t, what, dims):
        if t.dtype != torch.int32 or t.device != self.device or not t.is_contiguous() or tuple(t.shape) != dims:
            raise ValueError(f"{what} is a contiguous int32 tensor {dims} on {self.device}")
        return t

    def _calls(self, table, lengths, n_rows):
        batch = lengths.shape[0] if lengths.dim() else 0
        if table.dim() != 2:
            raise ValueError("table is [batch][columns]")
        self._index(lengths, "lengths", (batch,))
        self._index(table, "table", (batch, table.shape[1]))
        if n_rows is not None:
            self._index(n_rows, "n_rows", (batch,))
        return batch

    def _rows(self, t, what, batch, n):
        if t.dtype != self.tdt or t.device != self.device or not t.is_contiguous() or \
                t.numel() != batch * n * self.nq * self.hd:
            raise ValueError(f"{what} is a contiguous {self.tdt} tensor [{batch}][{n}][{self.nq}][{self.hd}] on {self.device}")
        return t

    def append(self, layer, qkv, table, lengths, n, q_out=None, n_rows=None):
        """Rotate and append ``n`` rows a sequence.  ``qkv`` [batch * n][...]
        float32 or the model's type, q|k|v heads side by side (k|v without
        ``q_out``); its rows may be apart.  ``q_out`` receives the rotated
        queries."""
        stream = torch.cuda.current_stream()
        if stream.device_index != self.device.index:
            with torch.cuda.device(self.device):
                return self.append(layer, qkv, table, lengths, n, q_out, n_rows)
        batch = self._calls(table, lengths, n_rows)
        width = ((0 if q_out is None else self.nq) + 2 * self.nkv) * self.hd
        if qkv.dim() != 2 or tuple(qkv.shape) != (batch * n, width) or qkv.device != self.device or \
                (qkv.stride(1) != 1 and width > 1) or qkv.dtype not in (torch.float32, self.tdt):
            raise ValueError(f"qkv is a float32 or {self.tdt} tensor [{batch * n}][{width}] on {self.device}, its rows unbroken")
        if q_out is not None:
            self._rows(q_out, "q_out", batch, n)
        ld = qkv.stride(0) if qkv.shape[0] > 1 else width
        capi.dflash_paged_append(self.pages, layer, capi.F32 if qkv.dtype == torch.float32 else capi.BF16, qkv, ld,
                                 batch, n, n_rows, table, table.shape[1], lengths, q_out, self.ws, stream)

    def read(self, layer, table, start, k_out=None, v_out=None, n_rows=None):
        """Rows back out of the pages: positions ``start`` + 0, 1, .. of each
        sequence into ``k_out`` and ``v_out`` [batch][n_kv][n][head_dim], of the
        model's type or float32, both alike; either may be left out.  The first
        ``n_rows`` rows of a sequence are written."""
        if torch.cuda.current_device() != self.device.index:
            with torch.cuda.device(self.device):
                return self.read(layer, table, start, k_out, v_out, n_rows)
        batch = self._calls(table, start, n_rows)
        outs = [t for t in (k_out, v_out) if t is not None]
        if not outs or outs[0].dim() != 4:
            raise ValueError("give k_out or v_out, [batch][n_kv][n][head_dim]")
        n, odt = outs[0].shape[2], outs[0].dtype
        for t in outs:
            if t.dtype != odt or odt not in (torch.float32, self.tdt) or t.device != self.device or \
                    not t.is_contiguous() or tuple(t.shape) != (batch, self.nkv, n, self.hd):
                raise ValueError(f"k_out and v_out are contiguous tensors [{batch}][{self.nkv}][{n}][{self.hd}] of one "
                                 f"type, float32 or {self.tdt}, on {self.device}")
        capi.dflash_paged_read(self.pages, layer, capi.F32 if odt == torch.float32 else capi.BF16, batch, n, n_rows,
                               table, table.shape[1], start, k_out, v_out, self.ws, _raw_stream(self.device.index))

    def attention(self, layer, q, table, lengths, out, causal=True, window=0, sinks=0, n_rows=None, shared_len=None):
        """Attention of ``q`` [batch][n][n_q][head_dim] over the pages into
        ``out``.  ``window`` > 0 hides keys behind it but the first ``sinks``;
        ``shared_len`` (one device int32) says how many first positions all
        sequences share, to be read once for the batch."""
        stream = torch.cuda.current_stream()
        if stream.device_index != self.device.index:
            with torch.cuda.device(self.device):
                return self.attention(layer, q, table, lengths, out, causal, window, sinks, n_rows, shared_len)
        batch = self._calls(table, lengths, n_rows)
        if not batch or q.dim() != 4 or q.shape[0] != batch:
            raise ValueError("q is [batch][n][n_q][head_dim]")
        n = q.shape[1]
        self._rows(q, "q", batch, n)
        self._rows(out, "out", batch, n)
        if shared_len is None:
            capi.dflash_paged_attention(self.pages, layer, q, batch, n, n_rows, int(causal), window, sinks, table,
                                        table.shape[1], lengths, out, self.ws, stream)
        else:
            if shared_len.dtype != torch.int32 or shared_len.device != self.device or shared_len.numel() != 1:
                raise ValueError(f"shared_len is one int32 on {self.device}")
            capi.dflash_paged_attention_shared(self.pages, layer, q, batch, n, n_rows, int(causal), window, sinks, table,
                                               table.shape[1], lengths, shared_len, out, self.ws, stream)


class W4Workspace:
    """Scratch of products with 4-bit weights for up to ``max_rows`` (<= 128)
    rows, for any matrices: one for each stream, and for each of the graphs that
    may run at the same time."""

    def __init__(self, max_rows=128, device="cuda"):
        self.handle, self.max_rows = None, max_rows
        with torch.cuda.device(device):
            self.device = torch.device("cuda", torch.cuda.current_device())
            self.handle = capi.dflash_w4_workspace_alloc(max_rows)

    def status(self):
        with torch.cuda.device(self.device):
            return capi.dflash_w4_status(self.handle)

    def close(self):
        """Frees the scratch.  Work of the calls made so far has to be done."""
        if self.handle:
            capi.dflash_w4_workspace_free(self.handle)
        self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class W4Linear:
    """A weight matrix [M][K] in 4 bits: codes 0..15 with a scale, and where
    ``zeros`` is set a zero point, for each ``group`` (32, 64, 128) columns of a
    row; w = scale * (code - zero), the zero point 8 without.  The codes lie in
    ``packed``, a uint8 tensor in the products' order (pass one to share it)."""

    def __init__(self, M, K, group=128, scale_dtype=torch.bfloat16, zeros=False, device="cuda", packed=None):
        if scale_dtype not in (torch.float32, torch.bfloat16):
            raise ValueError("scales are float32 or bfloat16")
        self.M, self.K, self.group, self.scale_dtype, self.zeros = M, K, group, scale_dtype, bool(zeros)
        self._c = capi.W4C(M, K, group, capi.F32 if scale_dtype == torch.float32 else capi.BF16, int(self.zeros), None)
        n = capi.dflash_w4_bytes(self._c)
        if packed is None:
            packed = torch.empty(n, dtype=torch.uint8, device=device)
        if packed.dtype != torch.uint8 or not packed.is_cuda or not packed.is_contiguous() or packed.numel() != n:
            raise ValueError(f"packed is a contiguous uint8 tensor of {n} bytes on the GPU")
        self.packed, self.device, self._index = packed, packed.device, packed.device.index
        self._c.packed = packed.data_ptr()

    @classmethod
    def from_weight(cls, w, group=128, scale_dtype=torch.bfloat16, zeros=False):
        """The nearest codes of a finite matrix w [M][K], float32 or bfloat16 (its rows may be apart)."""
        if w.dim() != 2 or w.dtype not in (torch.float32, torch.bfloat16) or not w.is_cuda or \
                (w.stride(1) != 1 and w.shape[1] > 1):
            raise ValueError("w is a float32 or bfloat16 matrix on the GPU, its rows unbroken")
        self = cls(w.shape[0], w.shape[1], group, scale_dtype, zeros, w.device)
        with torch.cuda.device(self.device):
            capi.dflash_w4_quantize(self._c, capi.F32 if w.dtype == torch.float32 else capi.BF16, w,
                                    w.stride(0) if w.shape[0] > 1 else w.shape[1])
        return self

    @classmethod
    def from_codes(cls, codes, scales, zeros=None):
        """From codes [M][K / 2] (uint8, the even column's in the low half), scales [M][K / group] (float32 or
        bfloat16) and, if given, zeros [M][K / group] (uint8)."""
        if codes.dim() != 2 or scales.dim() != 2 or codes.shape[0] != scales.shape[0] or scales.shape[1] < 1 or \
                2 * codes.shape[1] % scales.shape[1] != 0:
            raise ValueError("codes are [M][K / 2], scales [M][K / group]")
        if codes.dtype != torch.uint8 or not codes.is_cuda or not codes.is_contiguous() or not scales.is_contiguous() or \
                scales.device != codes.device:
            raise ValueError("codes (uint8) and scales are contiguous tensors on one GPU")
        if zeros is not None and (zeros.dtype != torch.uint8 or zeros.shape != scales.shape or not zeros.is_contiguous() or
                                  zeros.device != codes.device):
            raise ValueError("zeros is a contiguous uint8 tensor of the scales' shape and device")
        K = 2 * codes.shape[1]
        self = cls(codes.shape[0], K, K // scales.shape[1], scales.dtype, zeros is not None, codes.device)
        with torch.cuda.device(self.device):
            capi.dflash_w4_pack(self._c, codes, scales, zeros)
        return self

    def weight(self, dtype=torch.float32):
        """The matrix's values [M][K] (float32 or bfloat16)."""
        if dtype not in (torch.float32, torch.bfloat16):
            raise ValueError("float32 or bfloat16")
        out = torch.empty(self.M, self.K, dtype=dtype, device=self.device)
        with torch.cuda.device(self.device):
            capi.dflash_w4_unpack(self._c, capi.F32 if dtype == torch.float32 else capi.BF16, out)
        return out

    def product(self, x, out, ws, add=None, swiglu=False):
        """``out`` [rows][M] float32 = x w^T (+ ``add``, which may be ``out``), or with ``swiglu`` ``out``
        [rows][M / 2] of x's type, silu(even rows) * odd rows.  ``x`` [rows][K] float32 or bfloat16, its rows may be
        apart.  Asynchronous on the current stream of the weights' device."""
        if torch.cuda.current_device() != self._index:
            with torch.cuda.device(self.device):
                return self.product(x, out, ws, add, swiglu)
        dev, xdt, dims = self.device, x.dtype, x.shape
        if len(dims) != 2 or dims[1] != self.K or (xdt is not torch.bfloat16 and xdt is not torch.float32) or \
                x.device != dev or (x.stride(1) != 1 and self.K > 1):
            raise ValueError(f"x is a float32 or bfloat16 tensor [rows][{self.K}] on {dev}, its rows unbroken")
        rows = dims[0]
        odt, cols = (xdt, self.M // 2) if swiglu else (torch.float32, self.M)
        if out.dtype is not odt or out.shape != (rows, cols) or out.device != dev or not out.is_contiguous():
            raise ValueError(f"out is a contiguous {odt} tensor [{rows}][{cols}] on {dev}")
        if add is not None and (add.dtype is not torch.float32 or add.shape != (rows, self.M) or add.device != dev or
                                not add.is_contiguous()):
            raise ValueError(f"add is a contiguous float32 tensor [{rows}][{self.M}] on {dev}")
        capi.dflash_linear_w4(capi.BF16 if xdt is torch.bfloat16 else capi.F32, x, x.stride(0) if rows > 1 else self.K,
                              self._c, add, int(swiglu), out, rows, ws.handle, _raw_stream(self._index))
