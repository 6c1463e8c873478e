// Attention over pages: the call's geometry, the visible key range of a row,
// and the split of a call's work over CTAs, shared by the tensor-core kernel,
// the CUDA-core kernel and the merge of their partial results.
//
// Work.  The G query heads that share a KV head are stacked: stacked row
// i G + h is head h of block row i.  An item is one KV head and one group of
// stacked rows: a suffix item holds up to `ri` consecutive ones of one
// sequence, a prefix item up to `rp` consecutive ones of the whole batch, whose
// common keys [0, sh) are then read once for all of them.  An item's keys are
// walked in tiles of KT keys at absolute multiples of KT, only those that some
// row of it sees (first tokens that stay visible, then the window).  All tiles
// of all items, in item order, form one line: a tile takes `w` positions and an
// item `oh` more, for its start and its end, in the proportion of their times.
// Prefix items come first, head by head; suffix items follow in order of
// sequence, row group, head.  The line is cut into runs of `quota` positions, a
// run to a CTA, so every CTA has the same work whatever the lengths; a run
// covers the end of one item, whole items, and the start of another.  An item
// inside one run whose rows have no other part is finished there; every other
// piece leaves a partial result (row maximum, sum, unnormalised output).
// Pieces are added up in tile order: by the CTA that finishes an item's last
// one, or, where items have many rows or a shared prefix has left pieces that
// belong to many items, by a second kernel.  The cut depends on all lengths of
// the call: a row's last bits may depend on the batch around it, but the same
// call gives the same bits every time.
#pragma once
#include <stdint.h>

#include "common.cuh"

namespace dfl {

struct PagedGeom {
  int batch, n, nq, nkv, G;
  int ri, rp;            // stacked rows of a suffix / prefix item
  int nrt, nrp;          // row groups of a sequence / of the batch
  int causal, window, sinks;
  int ps, ps_log2, n_pages, table_stride;
  int cap;               // positions that a sequence's table row and the handle can name
  int grid;              // CTAs of the attention kernel
  int min_quota;
  int w_s, oh_s, w_p, oh_p;  // line positions of a tile of a suffix / prefix item, and of an item's start and end
  long long page_row0;   // pool row of (layer, page 0, head 0, slot 0)
  const int32_t* len;
  const int32_t* n_rows; // null: n
  const int32_t* table;
  const int32_t* shared; // null: no shared prefix
  float* part_o;         // suffix slots, then prefix slots
  float2* part_ml;
  long long pre_row0;    // first partial row of the prefix slots
  int slot_s, slot_p;    // partial rows per suffix / prefix slot
  int32_t* plan;         // [kPlanCum + batch] written for the merge kernel
  int32_t* tickets;      // [items] pieces done, zero between calls
  int32_t* records;      // [CTAs][8] items to join after the kernel
  unsigned g_magic;      // ceil(2^32 / G)
  unsigned wait_ns;      // limit of a wait in the tensor-core kernel
  int* status;
};

// Stacked rows (rows x query heads of a KV head) of one item at most, and the largest GQA group.
constexpr int kPagedItemRows = 256;
constexpr int kPagedMaxG = 64;
// CTAs a SM of an attention kernel at most (bounds the partial slots).
constexpr int kPagedMaxCtas = 4;

// plan[]: quota, sh / KT, tiles of a prefix item; then the line position of each
// sequence's first suffix item.
enum { kPlanQuota = 0, kPlanShared = 1, kPlanPre = 2, kPlanCum = 4 };

// `early`: a pass that comes before the call's arrays can be read.  None of them is; every sequence counts as n
// rows behind all the keys that its table can name.
__device__ __forceinline__ int paged_rows(const PagedGeom& g, int b, bool early = false) {
  return g.n_rows && !early ? min(max(g.n_rows[b], 0), g.n) : g.n;
}
__device__ __forceinline__ int paged_len(const PagedGeom& g, int b, bool early = false) {
  return early ? max(g.cap - g.n, 0) : max(g.len[b], 0);
}
__device__ __forceinline__ int paged_shared(const PagedGeom& g, bool early = false) {
  return early ? g.cap : *g.shared;
}

// The sequence's rows lie at positions that there are.
__device__ __forceinline__ bool positions_ok(const PagedGeom& g, int b) {
  const int rows = paged_rows(g, b);
  return rows == 0 || (g.len[b] >= 0 && g.len[b] <= g.cap - rows);
}

// The sequence's keys: those held and those of this call.
__device__ __forceinline__ int key_limit(const PagedGeom& g, int b) {
  return (int)min((long long)paged_len(g, b) + paged_rows(g, b), (long long)g.cap);
}

// First key of the window and end of the always-visible first keys of a row at
// block index i of a sequence holding P keys: visible are [0, sink) and [lo, hi).
__device__ __forceinline__ void row_span(const PagedGeom& g, int P, int rows, int i, int& sink, int& lo, int& hi) {
  P = min(P, g.cap);  // (an overlong sequence is an error; its sums stay in range)
  hi = min(g.causal ? P + i + 1 : P + rows, g.cap);
  lo = 0;
  sink = 0;
  if (g.window > 0) {
    lo = max(0, g.causal ? P + i - g.window + 1 : P - g.window);
    sink = min(g.sinks, lo);
  }
}

// The tiles of an item: [s0, s1) then [w0, w1), all multiples of KT keys.
struct TileSpan {
  int s0, s1, w0, w1;
  __device__ __forceinline__ int count() const { return s1 - s0 + w1 - w0; }
  __device__ __forceinline__ int tile(int t) const { return t < s1 - s0 ? s0 + t : w0 + t - (s1 - s0); }
};

// x / G for stacked row numbers (below 2^26, G <= 64: the error of the inverse stays below 1).
__device__ __forceinline__ int div_g(const PagedGeom& g, int x) {
  return g.G == 1 ? x : (int)__umulhi((unsigned)x, g.g_magic);
}

template <int KT>
__device__ __forceinline__ TileSpan span_of(const PagedGeom& g, int P, int rows, int rt, int sh_tiles) {
  TileSpan s{0, 0, 0, 0};
  const int r0 = rt * g.ri;
  if (r0 >= rows * g.G) return s;
  const int i0 = div_g(g, r0), i1 = div_g(g, min(r0 + g.ri, rows * g.G) - 1);
  int sink, lo, hi, sink1, lo1;
  row_span(g, P, rows, i0, sink, lo, hi);    // the first row's window starts first
  row_span(g, P, rows, i1, sink1, lo1, hi);  // the last row's ends last
  s.w0 = max(lo / KT, sh_tiles);
  s.w1 = max((hi + KT - 1) / KT, s.w0);
  s.s0 = sh_tiles;
  s.s1 = max(s.s0, min((sink1 + KT - 1) / KT, s.w0));
  return s;
}

template <int KT>
__device__ __forceinline__ TileSpan suffix_span(const PagedGeom& g, int b, int rt, int sh_tiles, bool early) {
  return span_of<KT>(g, paged_len(g, b, early), paged_rows(g, b, early), rt, sh_tiles);
}

// The tiles of every prefix item: those below sh that some row of the batch may see
// (min_len: the shortest live sequence).
template <int KT>
__device__ __forceinline__ TileSpan prefix_span(const PagedGeom& g, int sh_tiles, int min_len) {
  TileSpan s{0, 0, 0, sh_tiles};
  if (g.window > 0) {
    const int lo = max(0, g.causal ? min_len - g.window + 1 : min_len - g.window);
    s.w0 = min(lo / KT, sh_tiles);
    s.s1 = min((int)((g.sinks + (long long)KT - 1) / KT), s.w0);
  }
  return s;
}

// An item's place on the line.
struct Span1 {
  int line, total;  // first position, tiles
  int w, oh;        // positions a tile (1 or 2), and before the first one
  __device__ __forceinline__ int end() const { return line + oh + total * w; }
};
// A CTA's piece of one item.
struct Segment {
  bool prefix;
  int b, rt, hk;      // suffix: sequence, row group, head; prefix: row group rt of the batch, keys named by b's table
  TileSpan span;
  int t0, nt, total;  // its tiles [t0, t0 + nt) of the item's `total`
  Span1 at;           // its place on the line
  int ordinal;        // among the prefix or the suffix items
  long long slot_row; // first partial row of this piece
};

// Cuts of the line.  Cut k lies at k quota and divides the item that it falls into at the nearest tile; but
// where that would leave `snap` tiles or fewer on one side, it moves to that end of the item: short pieces do
// not pay for their start, their partial result and joining them.
__device__ __forceinline__ int snap_of(const Span1& s, int quota) {
  if (s.total * s.w <= 2 * quota) return min(3, s.total >> 1);
  const int q = 4 * s.w;  // min(3, quota / q)
  return (quota >= q) + (quota >= 2 * q) + (quota >= 3 * q);
}
// The tile of the item before which a cut at `pos`, inside the item, comes to lie (0 or total: at an end).
__device__ __forceinline__ int cut_at(int pos, const Span1& s, int quota) {
  const int snap = snap_of(s, quota), o = pos - s.line - s.oh + s.w / 2;
  const int t = o <= 0 ? 0 : min(o >> (s.w >> 1), s.total);
  return t <= snap ? 0 : s.total - t <= snap ? s.total : t;
}
// The pieces of an item: from CTA `c0` on, one a CTA.
__device__ __forceinline__ int pieces_of(const Span1& s, int quota, int& c0) {
  const int snap = snap_of(s, quota), at = s.line + s.oh - s.w / 2;
  // the first cut past `snap` tiles, and the first with `snap` or fewer behind it
  const int k0 = (int)((unsigned)(at + (snap + 1) * s.w + quota - 1) / (unsigned)quota);
  const int k1 = (int)((unsigned)(at + (s.total - snap) * s.w + quota - 1) / (unsigned)quota);
  c0 = k0 - 1;
  return max(k1 - k0, 0) + 1;
}

// The line as one CTA sees it.
struct PlanView {
  int T, quota, sh_tiles, min_len, pre_tiles;  // pre_tiles: tiles of one prefix item
  int pre_b;   // the first live sequence: its table names the shared pages
  int b, cum;  // the sequence that holds the CTA's first tile (past the prefix items), and its line position
};

// Line positions of an item of `tiles` tiles.
__device__ __forceinline__ int item_len(int tiles, int w, int oh) { return tiles > 0 ? oh + tiles * w : 0; }
__device__ __forceinline__ int pre_positions(const PagedGeom& g, int pre_tiles) {
  return item_len(pre_tiles, g.w_p, g.oh_p) * g.nrp * g.nkv;
}
template <int KT>
__device__ __forceinline__ int positions_of(const PagedGeom& g, int P, int rows, int sh_tiles) {
  int c = 0;
  for (int rt = 0; rt < g.nrt; ++rt) c += item_len(span_of<KT>(g, P, rows, rt, sh_tiles).count(), g.w_s, g.oh_s);
  return c * g.nkv;
}

// plan_view by one warp for itself, a lane for every few sequences (`write`: it writes the plan).
constexpr int kPlanSmall = 128;
template <int KT>
__device__ __forceinline__ PlanView plan_small(const PagedGeom& g, bool write, bool early) {
  const int lane = threadIdx.x & 31, per = (g.batch + 31) >> 5, b0 = lane * per, b1 = min(b0 + per, g.batch);
  PlanView v;
  v.sh_tiles = v.min_len = v.pre_b = v.pre_tiles = 0;
  const bool in = b0 < g.batch;
  // the lane's first sequence
  const int rows0 = in ? paged_rows(g, b0, early) : 0, P0 = in ? paged_len(g, b0, early) : 0;
  if (g.shared) {
    int m = rows0 > 0 ? min(P0, g.cap) : INT32_MAX, first = rows0 > 0 ? b0 : g.batch;
    for (int b = b0 + 1; b < b1; ++b)
      if (paged_rows(g, b, early) > 0) {
        m = min(m, min(paged_len(g, b, early), g.cap));
        first = min(first, b);
      }
    v.min_len = __reduce_min_sync(0xffffffffu, m);
    first = __reduce_min_sync(0xffffffffu, first);
    if (first < g.batch) {
      v.pre_b = first;
      v.sh_tiles = max(0, min(paged_shared(g, early), v.min_len)) / KT;
      if (v.sh_tiles > 0) v.pre_tiles = prefix_span<KT>(g, v.sh_tiles, v.min_len).count();
    }
  }
  const int pre_total = pre_positions(g, v.pre_tiles);
  const int c0 = positions_of<KT>(g, P0, rows0, v.sh_tiles);
  int c = c0;
  for (int b = b0 + 1; b < b1; ++b)
    c += positions_of<KT>(g, paged_len(g, b, early), paged_rows(g, b, early), v.sh_tiles);
  int inc = c;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += x;
  }
  int at = pre_total + inc - c;
  v.T = pre_total + __shfl_sync(0xffffffffu, inc, 31);
  v.quota = max(g.min_quota, (int)((unsigned)(v.T + g.grid - 1) / (unsigned)g.grid));
  const int start = max((int)min((long long)blockIdx.x * v.quota, (long long)v.T), pre_total);
  write = write && blockIdx.x == 0;
  int hit = start >= at && start < at + c0 ? b0 : -1, hit_at = at;
  if (per > 1 || write) {
    for (int b = b0; b < b1; ++b) {
      const int n =
          b == b0 ? c0 : positions_of<KT>(g, paged_len(g, b, early), paged_rows(g, b, early), v.sh_tiles);
      if (start >= at && start < at + n) {
        hit = b;
        hit_at = at;
      }
      if (write) {
        if (g.shared) g.plan[kPlanCum + b] = at;
        if (!positions_ok(g, b)) set_status(g.status, DFLASH_STATUS_CAPACITY);
      }
      at += n;
    }
  }
  const unsigned here = __ballot_sync(0xffffffffu, hit >= 0);
  const int src = here ? __ffs(here) - 1 : 0;
  v.b = __shfl_sync(0xffffffffu, hit, src);
  v.cum = __shfl_sync(0xffffffffu, hit_at, src);
  if (!here) v.b = g.batch;
  if (write && g.shared && lane == 0) {
    g.plan[kPlanQuota] = v.quota;
    g.plan[kPlanShared] = v.sh_tiles;
    g.plan[kPlanPre] = v.pre_tiles;
  }
  return v;
}

// All threads of the block: the shared prefix, the line's length and where the CTA's run starts.
// red: 2 NT / 32 + 8 ints of shared memory.  With `write`, CTA 0 writes the plan for the merge kernel.
template <int KT, int NT>
__device__ __forceinline__ PlanView plan_view(const PagedGeom& g, int* red, bool write = true) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (g.batch <= kPlanSmall) return plan_small<KT>(g, write && tid < 32, false);
  const bool first_cta = write && blockIdx.x == 0;
  PlanView v;
  const int per = (g.batch + NT - 1) / NT;
  const int b0 = min(tid * per, g.batch), b1 = min(b0 + per, g.batch);
  v.sh_tiles = 0;
  v.min_len = 0;
  v.pre_b = 0;
  int* res = red + 2 * (NT / 32);
  if (g.shared) {
    int m = INT32_MAX, first = g.batch;
    for (int b = b0; b < b1; ++b)
      if (paged_rows(g, b) > 0) {
        m = min(m, min(paged_len(g, b), g.cap));
        first = min(first, b);
      }
    m = __reduce_min_sync(0xffffffffu, m);
    first = __reduce_min_sync(0xffffffffu, first);
    if (lane == 0) {
      red[warp] = m;
      red[NT / 32 + warp] = first;
    }
    __syncthreads();
    for (int w = 0; w < NT / 32; ++w) {
      m = min(m, red[w]);
      first = min(first, red[NT / 32 + w]);
    }
    v.min_len = m;
    if (first < g.batch) {
      v.sh_tiles = max(0, min(paged_shared(g), m)) / KT;
      v.pre_b = first;
    }
    __syncthreads();
  }
  v.pre_tiles = v.sh_tiles > 0 ? prefix_span<KT>(g, v.sh_tiles, v.min_len).count() : 0;
  const int pre_total = pre_positions(g, v.pre_tiles);
  auto tiles_of = [&](int b) { return positions_of<KT>(g, paged_len(g, b), paged_rows(g, b), v.sh_tiles); };
  int sum = 0;
  for (int b = b0; b < b1; ++b) {
    sum += tiles_of(b);
    if (first_cta && !positions_ok(g, b)) set_status(g.status, DFLASH_STATUS_CAPACITY);
  }
  int inc = sum;  // inclusive scan over the block
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += x;
  }
  if (lane == 31) red[warp] = inc;
  __syncthreads();
  int base = pre_total, tot = pre_total;
  for (int w = 0; w < NT / 32; ++w) {
    if (w < warp) base += red[w];
    tot += red[w];
  }
  v.T = tot;
  v.quota = max(g.min_quota, (tot + g.grid - 1) / g.grid);
  const int start = max((int)min((long long)blockIdx.x * v.quota, (long long)tot), pre_total);
  int at = base + inc - sum;
  if (tid == 0) {
    res[0] = g.batch;
    res[1] = tot;
  }
  __syncthreads();
  for (int b = b0; b < b1; ++b) {
    const int c = per == 1 ? sum : tiles_of(b);
    if (first_cta) g.plan[kPlanCum + b] = at;
    if (start >= at && start < at + c) {
      res[0] = b;
      res[1] = at;
    }
    at += c;
  }
  if (first_cta && tid == 0) {
    g.plan[kPlanQuota] = v.quota;
    g.plan[kPlanShared] = v.sh_tiles;
    g.plan[kPlanPre] = v.pre_tiles;
  }
  __syncthreads();
  v.b = res[0];
  v.cum = res[1];
  return v;
}

// Walks a CTA's run piece by piece.
template <int KT>
struct SegmentWalk {
  const PagedGeom& g;
  const PlanView& v;
  int pos, end;       // the run: line positions
  int b, rt, hk;      // the next suffix item
  int item_at;        // its line position
  int pre_total;
  bool at_start;      // the first cut has not been placed yet
  bool early = false; // the lengths are not read
  __device__ __forceinline__ SegmentWalk(const PagedGeom& g_, const PlanView& v_) : g(g_), v(v_) {}
  __device__ __forceinline__ void start() {
    pos = (int)min((long long)blockIdx.x * v.quota, (long long)v.T);
    end = (int)min((long long)pos + v.quota, (long long)v.T);
    pre_total = pre_positions(g, v.pre_tiles);
    b = v.b;
    item_at = v.cum;
    rt = hk = 0;
    at_start = true;
  }
  // The item at `pos` (which lies in it, or where it begins).
  __device__ __forceinline__ bool item(Segment& s) {
    if (pos < pre_total) {
      const int len = item_len(v.pre_tiles, g.w_p, g.oh_p), k = (int)((unsigned)pos / (unsigned)len);
      s.prefix = true;
      s.hk = k / g.nrp;
      s.rt = k - s.hk * g.nrp;
      s.b = v.pre_b;
      s.span = prefix_span<KT>(g, v.sh_tiles, v.min_len);
      s.at = Span1{k * len, v.pre_tiles, g.w_p, g.oh_p};
      s.ordinal = k;
    } else {
      TileSpan sp;
      int c, tiles;
      while (true) {  // (pos < T: some item holds it, unless the lengths changed since the plan)
        if (b >= g.batch || pos < item_at) return false;
        sp = suffix_span<KT>(g, b, rt, v.sh_tiles, early);
        tiles = sp.count();
        c = item_len(tiles, g.w_s, g.oh_s);
        if (pos < item_at + c * g.nkv) break;
        item_at += c * g.nkv;
        if (++rt == g.nrt) {
          rt = 0;
          ++b;
        }
      }
      hk = (int)((unsigned)(pos - item_at) / (unsigned)c);
      s.prefix = false;
      s.b = b;
      s.rt = rt;
      s.hk = hk;
      s.span = sp;
      s.at = Span1{item_at + hk * c, tiles, g.w_s, g.oh_s};
      s.ordinal = (b * g.nrt + rt) * g.nkv + hk;
    }
    return true;
  }
  __device__ __forceinline__ bool next(Segment& s) {
    while (pos < end) {
      if (!item(s)) return false;
      s.t0 = at_start ? cut_at(pos, s.at, v.quota) : 0;  // (the run's first cut)
      at_start = false;
      const int to = end < s.at.end() ? cut_at(end, s.at, v.quota) : s.at.total;
      const bool last = end <= s.at.end();
      pos = last ? end : s.at.end();
      s.total = s.at.total;
      s.nt = to - s.t0;
      if (s.nt <= 0) {
        if (last) return false;
        continue;
      }
      const long long slot = (long long)s.ordinal + blockIdx.x;
      s.slot_row = s.prefix ? g.pre_row0 + slot * g.slot_p : slot * g.slot_s;
      return true;
    }
    return false;
  }
  __device__ __forceinline__ int pieces(const Segment& s, int& c0) const {
    return pieces_of(s.at, v.quota, c0);
  }
  // No other piece contributes to this one's rows.
  __device__ __forceinline__ bool whole(const Segment& s) const {
    return !s.prefix && s.nt == s.total && v.pre_tiles == 0;
  }
};

// Block row and head of an item's stacked row r, numbered from x0 of its sequence (or of the batch), and
// whether it is a row of the call.
struct ItemRow {
  int b, i, head;
  bool live;
};
__device__ __forceinline__ ItemRow item_row(const PagedGeom& g, bool prefix, int b, int hk, int x0, int r) {
  ItemRow w;
  const int x = x0 + r, q = div_g(g, x);
  w.head = hk * g.G + (x - q * g.G);
  w.live = r < (prefix ? g.rp : g.ri);
  if (prefix) {
    w.live = w.live && q < g.batch * g.n;
    const int f = w.live ? q : 0;
    w.b = f / g.n;
    w.i = f - w.b * g.n;
  } else {
    w.b = b;
    w.i = q;
  }
  w.live = w.live && w.i < paged_rows(g, w.b);
  return w;
}

// One warp: a row of HD from `nc` partials, `row_of(c)` the row of the c-th, as
//   sum_c 2^(m_c - m) o_c / sum_c 2^(m_c - m) l_c,  m = max m_c,
// lane l owning HD / 32 dimensions.  Partials are read past L1: other SMs wrote them.
template <typename T, int HD, typename F>
__device__ __forceinline__ void merge_row(const PagedGeom& g, int nc, F row_of, T* __restrict__ dst) {
  constexpr int V = HD / 32;
  const int lane = threadIdx.x & 31;
  float2 ml0 = make_float2(-INFINITY, 0.f);
  if (lane < nc) ml0 = __ldcg(g.part_ml + row_of(lane));
  float m = ml0.x;
  for (int c = 32 + lane; c < nc; c += 32) m = fmaxf(m, __ldcg(g.part_ml + row_of(c)).x);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  float acc[V], lsum = 0.f;
#pragma unroll
  for (int e = 0; e < V; ++e) acc[e] = 0.f;
  for (int cb = 0; cb < nc; cb += 32) {
    float2 ml = ml0;
    if (cb > 0) ml = cb + lane < nc ? __ldcg(g.part_ml + row_of(cb + lane)) : make_float2(-INFINITY, 0.f);
    // (a part whose maximum is NaN keeps its NaN through its sum)
    const float w = ml.x == -INFINITY ? 0.f : exp2f(ml.x - m);
    lsum += w * ml.y;
    const int lim = min(32, nc - cb);
#pragma unroll 1
    for (int c = 0; c < lim; c += 8) {
      float x[8][V];
#pragma unroll
      for (int u = 0; u < 8; ++u)
        if (c + u < lim) {
          const float* src = g.part_o + row_of(cb + c + u) * HD + lane * V;
          if (V == 4) {
            const float4 y = __ldcg(reinterpret_cast<const float4*>(src));
            x[u][0] = y.x, x[u][1] = y.y, x[u][2 % V] = y.z, x[u][3 % V] = y.w;
          } else {
            const float2 y = __ldcg(reinterpret_cast<const float2*>(src));
            x[u][0] = y.x, x[u][1] = y.y;
          }
        }
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const float wc = __shfl_sync(0xffffffffu, w, (c + u) & 31);
        if (c + u < lim) {
#pragma unroll
          for (int e = 0; e < V; ++e) acc[e] += wc * x[u][e];
        }
      }
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) lsum += __shfl_xor_sync(0xffffffffu, lsum, o);
#pragma unroll
  for (int e = 0; e < V; ++e) dst[lane * V + e] = from_f<T>(acc[e] / lsum);
}

// One warp's share (rows w, w + warps, ...) of an item whose `nc` pieces begin with CTA c0's.
// Not inlined: its registers are not to be kept free in the loops that it follows.
template <typename T, int HD>
__device__ __noinline__ void merge_item(const PagedGeom& g, int b, int rt, int hk, int r0, int rows, int nc, int c0,
                                        int w, int warps, T* __restrict__ out) {
  for (int r = r0 + w; r < r0 + rows; r += warps) {
    const int x = rt * g.ri + r, i = div_g(g, x);
    const long long base = ((long long)(b * g.nrt + rt) * g.nkv + hk + c0) * g.slot_s + r;
    merge_row<T, HD>(g, nc, [&](int c) { return base + (long long)c * g.slot_s; },
                     out + ((long long)(b * g.n + i) * g.nq + hk * g.G + x - i * g.G) * HD);
  }
}

cudaError_t rope_table(float2* tab, int max_pos, int half, double theta);
cudaError_t paged_append(int in_dtype, int dtype, const void* qkv, long long ld, int batch, int n, int nq, int nkv,
                         int hd, const int32_t* n_rows, const int32_t* table, int table_stride, const int32_t* len,
                         const float2* tab, int max_pos, int n_pages, int ps, long long page0, void* qout, void* kp,
                         void* vp, int* status, cudaStream_t s);
// How a kernel cuts a call: stacked rows of a suffix / prefix item, keys of a tile, line positions of a tile and of
// an item's start and end.
struct PagedRule {
  int ri, rp, keys, w, oh;
};
PagedRule paged_rule_core(const PagedGeom& g);
PagedRule paged_rule_tc(const PagedGeom& g);
// Whether the line of such a call fits the plan's integers, whatever lengths its tables hold.
bool paged_line_fits(const PagedGeom& g, const PagedRule& r);
// Fills in the split of a call: row groups, the grid, runs of `min_tiles` tiles at least, the partial slots.
// Returns the partial rows that it needs.
long long paged_split(PagedGeom& g, const PagedRule& r, int grid, int min_tiles);
// Keys of a tile of the tensor-core kernel.
constexpr int kPagedTcKeys = 128;
// Merge of the tensor-core kernel's partials.
cudaError_t paged_merge_bf16(int hd, const PagedGeom& g, void* out, cudaStream_t s);
cudaError_t paged_join_bf16(int hd, const PagedGeom& g, void* out, cudaStream_t s);
// Attention of a call described by `g` (geometry, table, lengths; the split is filled in here): float32 on
// the CUDA cores, bf16 on the tensor cores.
cudaError_t paged_attention_core(int hd, const PagedGeom& g, const void* q, const void* kp, const void* vp, void* out,
                                 long long part_rows, cudaStream_t s);
cudaError_t paged_attention_tc(int hd, const PagedGeom& g, const CUtensorMap& tk, const CUtensorMap& tv,
                               long long pool_rows, const void* q, void* out, long long part_rows, cudaStream_t s);
// 2-D maps over a bf16 pool [rows][hd]: boxes of 64 elements (128 B, swizzled) by one page's positions.
bool make_page_maps(const void* k, const void* v, long long rows, int hd, int page_size, CUtensorMap* mk,
                    CUtensorMap* mv);

}  // namespace dfl
