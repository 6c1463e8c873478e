// KV pages: the RoPE table, the append of rotated keys and values, attention
// over pages on the CUDA cores, and the merge of partial attention results.
#include "paged.cuh"

#include <math.h>

#include <algorithm>

#include "common.cuh"
#include "internal.h"

namespace dfl {

// ------------------------------------------------------------------ RoPE table
// cos/sin of pos * theta^(-2 i / hd), angles in double precision.
__global__ void rope_table_kernel(float2* tab, int max_pos, int half, double theta) {
  const long long n = (long long)max_pos * half;
  for (long long t = (long long)blockIdx.x * blockDim.x + threadIdx.x; t < n; t += (long long)gridDim.x * blockDim.x) {
    const int p = (int)(t / half), i = (int)(t - (long long)p * half);
    double s, c;
    sincos((double)p * pow(theta, -(double)i / half), &s, &c);
    tab[t] = make_float2((float)c, (float)s);
  }
}

cudaError_t rope_table(float2* tab, int max_pos, int half, double theta) {
  rope_table_kernel<<<num_sms() * 4, 256>>>(tab, max_pos, half, theta);
  return cudaGetLastError();
}

// ------------------------------------------------------------------ append
// Row (b, j) of the packed q|k|v rows at position p = len[b] + j: q and k are
// rotated in float32 (x_lo c - x_hi s, x_hi c + x_lo s), rounded once, and q
// goes to q_out, k and v to slot p mod ps of page table[b][p / ps].
//
// Bound by the rows' bytes, in and out.  A thread moves 8 entries of the lower
// half and the 8 they rotate with, of HPT heads of one row: their (cos, sin)
// pairs, twice the bytes of a bf16 head's 16 entries, are fetched once for all
// of them, and all their loads are in flight together.  Blocks take `rpb` whole
// rows.  HPT = 1 where the rows do not fill the GPU: more threads, shorter ones.
// 16384 rows of 40 + 2 x 8 heads of 128 in bf16: 79.9 us, 5.88 TB/s of 6.78 that a
// copy reaches (one head a thread, (cos, sin) fetched for each: 96.6 us).
template <typename T>
struct Raw8 {  // 8 entries as they lie in memory
  uint4 v[sizeof(T) / 2];
};

template <typename T>
__device__ __forceinline__ Raw8<T> load8(const T* p, bool vec) {
  Raw8<T> r;
  if (vec) {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) r.v[i] = *(reinterpret_cast<const uint4*>(p) + i);
  } else {
    T x[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = p[e];
    memcpy(&r, x, sizeof(r));
  }
  return r;
}
__device__ __forceinline__ void unpack8(const Raw8<float>& r, float (&x)[8]) { memcpy(x, &r, sizeof(r)); }
__device__ __forceinline__ void unpack8(const Raw8<bf16>& r, float (&x)[8]) {
  const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&r);
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float2 f = __bfloat1622float2(h[e]);
    x[2 * e] = f.x;
    x[2 * e + 1] = f.y;
  }
}

template <typename T>
__device__ __forceinline__ void store8(T* p, const float (&x)[8]) {
  if (sizeof(T) == 4) {
    *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
    *(reinterpret_cast<float4*>(p) + 1) = make_float4(x[4], x[5], x[6], x[7]);
  } else {
    uint4 v;
    __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&v);
#pragma unroll
    for (int e = 0; e < 4; ++e) h[e] = __floats2bfloat162_rn(x[2 * e], x[2 * e + 1]);
    *reinterpret_cast<uint4*>(p) = v;
  }
}

template <typename TI, typename T, int HPT>
__global__ void __launch_bounds__(256)
    paged_append_kernel(const TI* __restrict__ qkv, long long ld, int vec, int rows, int n, int nq, int nkv, int hd,
                        int rpb, const int32_t* __restrict__ n_rows, const int32_t* __restrict__ table,
                        int table_stride, const int32_t* __restrict__ len, const float2* __restrict__ tab, int max_pos,
                        int n_pages, int ps_log2, long long page0, T* __restrict__ qout, T* __restrict__ kp,
                        T* __restrict__ vp, int* status) {
  const int half = hd / 2, lanes = half / 8, heads = nq + 2 * nkv;
  const int groups = (heads + HPT - 1) / HPT;  // group hg takes heads hg, hg + groups, ..
  const int per_row = groups * lanes;
  const int r0 = blockIdx.x * rpb, items = min(rpb, rows - r0) * per_row;
  pdl_launch();
  pdl_wait();
  for (int t = threadIdx.x; t < items; t += 256) {
    const int rr = t / per_row, w = t - rr * per_row, r = r0 + rr;
    const int b = r / n, j = r - b * n;
    if (n_rows && j >= n_rows[b]) continue;
    const int hg = w / lanes, e = (w - hg * lanes) * 8;
    const TI* src = qkv + (long long)r * ld + e;
    Raw8<TI> lo[HPT], hi[HPT];
#pragma unroll
    for (int x = 0; x < HPT; ++x) {
      const int h = hg + x * groups;
      if (h < heads) {
        lo[x] = load8<TI>(src + h * hd, vec);
        hi[x] = load8<TI>(src + h * hd + half, vec);
      }
    }
    const long long pos = (long long)len[b] + j;
    if (pos < 0 || pos >= max_pos || (pos >> ps_log2) >= table_stride) {
      if (w == 0) set_status(status, DFLASH_STATUS_CAPACITY);
      continue;
    }
    const int page = table[(long long)b * table_stride + (pos >> ps_log2)];
    const bool good = (unsigned)page < (unsigned)n_pages;
    if (!good && w == 0) set_status(status, DFLASH_STATUS_BOUNDS);
    const float4* cs = reinterpret_cast<const float4*>(tab + pos * half + e);
    float4 c[4];  // two (cos, sin) pairs each
#pragma unroll
    for (int x = 0; x < 4; ++x) c[x] = __ldg(cs + x);
    // slot (pos mod ps) of the page's first head
    const long long slot = (((page0 + page) * nkv) << ps_log2) + (pos & ((1 << ps_log2) - 1));
#pragma unroll
    for (int x = 0; x < HPT; ++x) {
      const int h = hg + x * groups;
      if (h >= heads) break;
      float a[8], z[8];
      unpack8(lo[x], a);
      unpack8(hi[x], z);
      if (h < nq + nkv) {
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          const float a0 = a[2 * y], z0 = z[2 * y], a1 = a[2 * y + 1], z1 = z[2 * y + 1];
          a[2 * y] = a0 * c[y].x - z0 * c[y].y;
          z[2 * y] = z0 * c[y].x + a0 * c[y].y;
          a[2 * y + 1] = a1 * c[y].z - z1 * c[y].w;
          z[2 * y + 1] = z1 * c[y].z + a1 * c[y].w;
        }
      }
      T* dst;
      if (h < nq) {
        dst = qout + ((long long)r * nq + h) * hd;
      } else {
        if (!good) break;  // (heads ascend: keys and values only from here on)
        const int hk = h - nq < nkv ? h - nq : h - nq - nkv;
        dst = (h - nq < nkv ? kp : vp) + (slot + ((long long)hk << ps_log2)) * hd;
      }
      store8<T>(dst + e, a);
      store8<T>(dst + e + half, z);
    }
  }
}

cudaError_t paged_append(int in_dtype, int dtype, const void* qkv, long long ld, int batch, int n, int nq, int nkv,
                         int hd, const int32_t* n_rows, const int32_t* table, int table_stride, const int32_t* len,
                         const float2* tab, int max_pos, int n_pages, int ps, long long page0, void* qout, void* kp,
                         void* vp, int* status, cudaStream_t s) {
  const size_t es = in_dtype == DFLASH_BF16 ? 2 : 4;
  const int vec = (reinterpret_cast<uintptr_t>(qkv) & 15) == 0 && (ld * es) % 16 == 0;
  const int rows = batch * n, heads = nq + 2 * nkv, lanes = hd / 16, ps_log2 = 31 - __builtin_clz(ps);
  const bool many = (long long)rows * heads * lanes >= (long long)num_sms() * 2048 * 4;
  const int per_row = (heads + (many ? 3 : 0)) / (many ? 4 : 1) * lanes;
  const int rpb = many ? std::max(1, 1024 / per_row) : 1;
  const unsigned grid = (unsigned)((rows + (long long)rpb - 1) / rpb);
#define DFL_APPEND_H(TI, T, H)                                                                                        \
  DFL_RET(launch_pdl(paged_append_kernel<TI, T, H>, dim3(grid), dim3(256), 0, s, (const TI*)qkv, ld, vec, rows, n, nq, \
                     nkv, hd, rpb, n_rows, table, table_stride, len, tab, max_pos, n_pages, ps_log2, page0, (T*)qout,  \
                     (T*)kp, (T*)vp, status))
#define DFL_APPEND(TI, T)      \
  if (many)                    \
    DFL_APPEND_H(TI, T, 4);    \
  else                         \
    DFL_APPEND_H(TI, T, 1)
  if (dtype == DFLASH_F32) {
    DFL_APPEND(float, float);
  } else if (in_dtype == DFLASH_F32) {
    DFL_APPEND(float, bf16);
  } else {
    DFL_APPEND(bf16, bf16);
  }
#undef DFL_APPEND
#undef DFL_APPEND_H
  count_launch();
  return cudaSuccess;
}

// ------------------------------------------------------------------ CUDA-core attention
// One pass over an item's keys in tiles of 32 with the running maximum m, sum l
// and output o of every row: s = q.k scale log2(e), m' = max(m, max s),
// p = 2^(s - m'), l = l 2^(m - m') + sum p, o = o 2^(m - m') + p v.
// MR = 16 MRM stacked rows (row = thread / 16 + 16 x); the 16 threads of a row
// share its keys in the scores and its dimensions in the output.  A hidden
// key's weight is stored as -0, which the masked tiles skip, so that an Inf or
// NaN value behind a mask stays out of the row.  The next tile's keys and values
// are fetched into registers while this one is worked on.  At a drafter's sizes
// (4 sequences, 4 heads of 64, 16 rows over 128 to 1024 keys: 17.4 us, 0.8 at a
// copy's rate) the time is the plan, two tiles' trips to memory and the join.
constexpr int kCoreKeys = 32;
constexpr int kCoreThreads = 256;

template <int HD, int MRM>
struct CoreLayout {
  static constexpr int MR = 16 * MRM;
  static constexpr int kRow = HD + 4;  // padded: the 16 lanes of a row read 16 key rows without bank conflicts
  static constexpr int kK = MR * HD * 4;
  static constexpr int kV = kK + kCoreKeys * kRow * 4;
  static constexpr int kP = kV + kCoreKeys * HD * 4;
  static constexpr int kRed = kP + MR * kCoreKeys * 4;
  static constexpr int kSmem = kRed + (2 * kCoreThreads / 32 + 8) * 4;
};

template <typename T, int HD, int MRM>
__global__ void __launch_bounds__(kCoreThreads)
    paged_attn_core_kernel(const __grid_constant__ PagedGeom g, const T* __restrict__ q, const T* __restrict__ kp,
                           const T* __restrict__ vp, T* __restrict__ out, float scale_log2) {
  typedef CoreLayout<HD, MRM> L;
  extern __shared__ uint8_t smem_raw[];
  float* sq = reinterpret_cast<float*>(smem_raw);
  float* sk = reinterpret_cast<float*>(smem_raw + L::kK);
  float* sv = reinterpret_cast<float*>(smem_raw + L::kV);
  float* sp = reinterpret_cast<float*>(smem_raw + L::kP);
  const int tid = threadIdx.x, l16 = tid & 15, rq = tid >> 4;
  constexpr int NC = HD / 64;  // output: float4 chunks of a thread
  pdl_launch();
  pdl_wait();
  const PlanView v = plan_view<kCoreKeys, kCoreThreads>(g, reinterpret_cast<int*>(smem_raw + L::kRed));
  SegmentWalk<kCoreKeys> walk(g, v);
  walk.start();
  Segment sg;
  while (walk.next(sg)) {
    ItemRow row[MRM];
    int sink[MRM], lo[MRM], hi[MRM];
    float m[MRM], l[MRM], o[MRM][NC * 4];
    __syncthreads();
#pragma unroll
    for (int x = 0; x < MRM; ++x) {
      const int r = rq + 16 * x;
      row[x] = item_row(g, sg.prefix, sg.b, sg.hk, sg.rt * (sg.prefix ? g.rp : g.ri), r);
      sink[x] = lo[x] = hi[x] = 0;
      if (row[x].live) row_span(g, paged_len(g, row[x].b), paged_rows(g, row[x].b), row[x].i, sink[x], lo[x], hi[x]);
      m[x] = -INFINITY;
      l[x] = 0.f;
#pragma unroll
      for (int e = 0; e < NC * 4; ++e) o[x][e] = 0.f;
      for (int d = l16; d < HD; d += 16)
        sq[r * HD + d] = row[x].live ? to_f<T>(q[(((long long)row[x].b * g.n + row[x].i) * g.nq + row[x].head) * HD + d])
                                     : 0.f;
    }
    const int key_lo = sg.prefix ? 0 : v.sh_tiles * kCoreKeys;  // keys below belong to the shared prefix
    const int key_end = sg.prefix ? v.sh_tiles * kCoreKeys : key_limit(g, sg.b);
    // some row of the item sees the keys below seen_sink and those from seen_lo on: its first row's
    int seen_sink, seen_lo, seen_hi;
    row_span(g, sg.prefix ? v.min_len : paged_len(g, sg.b), paged_rows(g, sg.b),
             sg.prefix ? 0 : div_g(g, sg.rt * g.ri), seen_sink, seen_lo, seen_hi);
    // 8 threads a key: its rows of keys and values (keys that no row sees, or in a bad page: zeros), fetched into
    // registers while the tile before is worked on
    Raw8<T> rk[HD / 64], rv[HD / 64];
    auto fetch = [&](int t) {
      const int key = sg.span.tile(t) * kCoreKeys + (tid >> 3), part = tid & 7;
      int page = -1;
      if (key < key_end && (key < seen_sink || key >= seen_lo)) {
        page = g.table[(long long)sg.b * g.table_stride + (key >> g.ps_log2)];
        if ((unsigned)page >= (unsigned)g.n_pages) {
          page = -1;
          set_status(g.status, DFLASH_STATUS_BOUNDS);
        }
      }
      const long long at = (g.page_row0 + ((long long)page * g.nkv + sg.hk) * g.ps + (key & (g.ps - 1))) * HD + part * 8;
#pragma unroll
      for (int e = 0; e < HD / 64; ++e) {
        rk[e] = rv[e] = Raw8<T>{};
        if (page >= 0) {
          rk[e] = load8<T>(kp + at + e * 64, true);
          rv[e] = load8<T>(vp + at + e * 64, true);
        }
      }
    };
    fetch(sg.t0);
    for (int t = sg.t0; t < sg.t0 + sg.nt; ++t) {
      const int k0 = sg.span.tile(t) * kCoreKeys;
      __syncthreads();
#pragma unroll
      for (int e = 0; e < HD / 64; ++e) {
        float x[8];
        unpack8(rk[e], x);
        store8<float>(sk + (tid >> 3) * L::kRow + (tid & 7) * 8 + e * 64, x);
        unpack8(rv[e], x);
        store8<float>(sv + (tid >> 3) * HD + (tid & 7) * 8 + e * 64, x);
      }
      if (t + 1 < sg.t0 + sg.nt) fetch(t + 1);
      __syncthreads();
      float s[MRM][2];
#pragma unroll
      for (int x = 0; x < MRM; ++x) s[x][0] = s[x][1] = 0.f;
#pragma unroll 4
      for (int d = 0; d < HD; d += 4) {
        const float4 ka = *reinterpret_cast<const float4*>(sk + l16 * L::kRow + d);
        const float4 kb = *reinterpret_cast<const float4*>(sk + (l16 + 16) * L::kRow + d);
#pragma unroll
        for (int x = 0; x < MRM; ++x) {
          const float4 a = *reinterpret_cast<const float4*>(sq + (rq + 16 * x) * HD + d);
          s[x][0] = fmaf(a.x, ka.x, fmaf(a.y, ka.y, fmaf(a.z, ka.z, fmaf(a.w, ka.w, s[x][0]))));
          s[x][1] = fmaf(a.x, kb.x, fmaf(a.y, kb.y, fmaf(a.z, kb.z, fmaf(a.w, kb.w, s[x][1]))));
        }
      }
      bool masked = false;
#pragma unroll
      for (int x = 0; x < MRM; ++x) {
        float z[2], mx = -INFINITY;
        bool vis[2];
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          const int key = k0 + l16 + 16 * y;
          vis[y] = key >= key_lo && key < key_end && (key < sink[x] || (key >= lo[x] && key < hi[x]));
          z[y] = vis[y] ? s[x][y] * scale_log2 : -INFINITY;
          mx = fmaxf(mx, z[y]);
          masked |= !vis[y];
        }
#pragma unroll
        for (int w = 8; w > 0; w >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, w));
        const float mn = fmaxf(m[x], mx);
        const float ref = mn == -INFINITY ? 0.f : mn;
        float sum = 0.f;
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          const float p = vis[y] ? exp2f(z[y] - ref) : -0.f;
          sp[(rq + 16 * x) * kCoreKeys + l16 + 16 * y] = p;
          sum += p;
        }
#pragma unroll
        for (int w = 8; w > 0; w >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, w);
        const float f = m[x] == -INFINITY ? 0.f : exp2f(m[x] - ref);
        l[x] = l[x] * f + sum;
        m[x] = mn;
#pragma unroll
        for (int e = 0; e < NC * 4; ++e) o[x][e] *= f;
      }
      masked = __syncthreads_or(masked);
      auto weigh = [&](int x, float p, const float4 (&a)[NC]) {
#pragma unroll
        for (int c = 0; c < NC; ++c) {
          o[x][4 * c] = fmaf(p, a[c].x, o[x][4 * c]);
          o[x][4 * c + 1] = fmaf(p, a[c].y, o[x][4 * c + 1]);
          o[x][4 * c + 2] = fmaf(p, a[c].z, o[x][4 * c + 2]);
          o[x][4 * c + 3] = fmaf(p, a[c].w, o[x][4 * c + 3]);
        }
      };
#pragma unroll 4
      for (int k = 0; k < kCoreKeys; ++k) {
        float4 a[NC];
#pragma unroll
        for (int c = 0; c < NC; ++c) a[c] = *reinterpret_cast<const float4*>(sv + k * HD + c * 64 + l16 * 4);
#pragma unroll
        for (int x = 0; x < MRM; ++x) {
          const float p = sp[(rq + 16 * x) * kCoreKeys + k];
          if (!masked || __float_as_int(p) >= 0) weigh(x, p, a);  // -0: hidden
        }
      }
    }
    const bool whole = walk.whole(sg);
#pragma unroll
    for (int x = 0; x < MRM; ++x) {
      if (!row[x].live) continue;
      const int r = rq + 16 * x;
      if (whole) {
        T* dst = out + (((long long)row[x].b * g.n + row[x].i) * g.nq + row[x].head) * HD;
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
          for (int e = 0; e < 4; ++e) dst[c * 64 + l16 * 4 + e] = from_f<T>(o[x][4 * c + e] / l[x]);
      } else {
        float* dst = g.part_o + (sg.slot_row + r) * HD;
#pragma unroll
        for (int c = 0; c < NC; ++c)
          *reinterpret_cast<float4*>(dst + c * 64 + l16 * 4) =
              make_float4(o[x][4 * c], o[x][4 * c + 1], o[x][4 * c + 2], o[x][4 * c + 3]);
        if (l16 == 0) g.part_ml[sg.slot_row + r] = make_float2(m[x], l[x]);
      }
    }
    if (!whole && v.pre_tiles == 0) {
      int c0;
      const int nc = walk.pieces(sg, c0);
      int* done = reinterpret_cast<int*>(smem_raw + L::kRed);
      __syncthreads();
      if (tid == 0) {
        __threadfence();
        *done = atomicAdd(g.tickets + sg.ordinal, 1) == nc - 1;
      }
      __syncthreads();
      if (*done) {
        __threadfence();
        if (tid == 0) g.tickets[sg.ordinal] = 0;
        merge_item<T, HD>(g, sg.b, sg.rt, sg.hk, 0, min(g.ri, paged_rows(g, sg.b) * g.G - sg.rt * g.ri), nc, c0, tid >> 5,
                          kCoreThreads / 32, out);
      }
    }
  }
}

// ------------------------------------------------------------------ merge
// Calls with a shared prefix: each row from its prefix pieces and its sequence's own, each in tile order.
// One warp per (row, head).  A row that one piece finished has nothing here.
constexpr int kMergeWarps = 8;
template <typename T, int HD, int KT>
__global__ void __launch_bounds__(kMergeWarps * 32)
    paged_merge_kernel(const __grid_constant__ PagedGeom g, T* __restrict__ out) {
  const long long item = (long long)blockIdx.x * kMergeWarps + (threadIdx.x >> 5);
  pdl_launch();
  pdl_wait();
  if (item >= (long long)g.batch * g.n * g.nq) return;
  const int r = (int)(item / g.nq), h = (int)(item - (long long)r * g.nq);
  const int b = r / g.n, i = r - b * g.n;
  const int rows = paged_rows(g, b), P = paged_len(g, b);
  const int quota = g.plan[kPlanQuota], sh = g.plan[kPlanShared], pre = g.plan[kPlanPre];
  int at = g.plan[kPlanCum + b];
  if (i >= rows) return;
  const int hk = div_g(g, h), x = i * g.G + h - hk * g.G, rt = x / g.ri;
  // its sequence's own pieces
  for (int y = 0; y < rt; ++y) at += item_len(span_of<KT>(g, P, rows, y, sh).count(), g.w_s, g.oh_s) * g.nkv;
  const int cnt = span_of<KT>(g, P, rows, rt, sh).count();
  at += hk * item_len(cnt, g.w_s, g.oh_s);
  int c0 = 0, p0 = 0;
  const int ns = cnt > 0 ? pieces_of(Span1{at, cnt, g.w_s, g.oh_s}, quota, c0) : 0;
  if (ns <= 1 && pre == 0) return;
  const long long srow = ((long long)(b * g.nrt + rt) * g.nkv + hk + c0) * g.slot_s + x - rt * g.ri;
  const int xp = r * g.G + h - hk * g.G, rp = xp / g.rp, k = hk * g.nrp + rp;
  const int np = pre > 0 ? pieces_of(Span1{k * item_len(pre, g.w_p, g.oh_p), pre, g.w_p, g.oh_p}, quota, p0) : 0;
  const long long prow = g.pre_row0 + (long long)(k + p0) * g.slot_p + xp - rp * g.rp;
  merge_row<T, HD>(g, np + ns, [&](int c) {
    return c < np ? prow + (long long)c * g.slot_p : srow + (long long)(c - np) * g.slot_s;
  }, out + ((long long)r * g.nq + h) * HD);
}

// Calls without one: block (c, y) joins `per` rows from per y on of the item that CTA c recorded, if it did.
// By itself 10.5 us behind 8 blocks of 16 rows over 4K keys, whose call takes 60 with it.
template <typename T, int HD>
__global__ void __launch_bounds__(kMergeWarps * 32)
    paged_join_kernel(const __grid_constant__ PagedGeom g, int per, T* __restrict__ out) {
  pdl_launch();
  pdl_wait();
  const int4* rec = reinterpret_cast<const int4*>(g.records) + 2 * blockIdx.x;
  const int4 a = rec[0];
  const int c0 = rec[1].x;
  if (a.x <= 0) return;
  const int rows = min(g.ri, paged_rows(g, a.y) * g.G - a.z * g.ri), r0 = per * blockIdx.y;
  if (r0 < rows)
    merge_item<T, HD>(g, a.y, a.z, a.w, r0, min(per, rows - r0), a.x, c0, threadIdx.x >> 5, kMergeWarps, out);
}

cudaError_t paged_join_bf16(int hd, const PagedGeom& g, void* out, cudaStream_t s) {
  // at most 8 blocks an SM: more would run in waves, and most find nothing to do
  const int per = std::max(kMergeWarps, (g.slot_s + 7) / 8);
  const dim3 grid(g.grid, (g.slot_s + per - 1) / per);
  if (hd == 64)
    DFL_RET(launch_pdl(paged_join_kernel<bf16, 64>, grid, dim3(kMergeWarps * 32), 0, s, g, per, (bf16*)out));
  else
    DFL_RET(launch_pdl(paged_join_kernel<bf16, 128>, grid, dim3(kMergeWarps * 32), 0, s, g, per, (bf16*)out));
  count_launch();
  return cudaSuccess;
}

template <typename T, int HD, int KT>
static cudaError_t merge_launch(const PagedGeom& g, void* out, cudaStream_t s) {
  const long long items = (long long)g.batch * g.n * g.nq;
  DFL_RET(launch_pdl(paged_merge_kernel<T, HD, KT>, dim3((unsigned)((items + kMergeWarps - 1) / kMergeWarps)),
                     dim3(kMergeWarps * 32), 0, s, g, (T*)out));
  count_launch();
  return cudaSuccess;
}
cudaError_t paged_merge_bf16(int hd, const PagedGeom& g, void* out, cudaStream_t s) {
  return hd == 64 ? merge_launch<bf16, 64, kPagedTcKeys>(g, out, s) : merge_launch<bf16, 128, kPagedTcKeys>(g, out, s);
}

static int groups_of(int rows, int of) { return (rows + of - 1) / of; }

long long paged_split(PagedGeom& g, const PagedRule& r, int grid, int min_tiles) {
  g.ri = r.ri;
  g.rp = r.rp;
  g.w_s = g.w_p = r.w;
  g.oh_s = g.oh_p = r.oh;
  g.g_magic = (unsigned)(((1ull << 32) + g.G - 1) / g.G);
  g.nrt = groups_of(g.n * g.G, r.ri);
  g.nrp = groups_of(g.batch * g.n * g.G, r.rp);
  g.grid = grid;
  g.min_quota = min_tiles * r.w;
  g.slot_s = std::min(g.n * g.G, r.ri);
  g.slot_p = std::min(g.batch * g.n * g.G, r.rp);
  g.pre_row0 = ((long long)g.batch * g.nrt * g.nkv + grid) * g.slot_s;
  return g.pre_row0 + (g.shared ? ((long long)g.nrp * g.nkv + grid) * g.slot_p : 0);
}

// Below 2^30 positions every sum and product on the line (a position and a run, an item's tiles by its heads) fits
// an int.  16384 rows of 32 / 8 heads in 8 sequences behind tables of 131072 positions: 4.2 million.
bool paged_line_fits(const PagedGeom& g, const PagedRule& r) {
  const double items =
      (double)g.batch * groups_of(g.n * g.G, r.ri) + (g.shared ? groups_of(g.batch * g.n * g.G, r.rp) : 0);
  return items * g.nkv * (((double)g.cap / r.keys + 2) * r.w + r.oh) < 1073741824.0;
}

// Few stacked rows: the 16-row tile spends fewer products on padding.
static bool core_small(const PagedGeom& g) { return (g.shared ? g.batch : 1) * g.n * g.G <= 16; }
PagedRule paged_rule_core(const PagedGeom& g) {
  const int rows = core_small(g) ? 16 : 64;
  return PagedRule{rows, rows, kCoreKeys, 1, 0};
}

template <typename T, int HD, int MRM>
static cudaError_t core_launch(PagedGeom g, const void* q, const void* kp, const void* vp, void* out,
                               long long part_rows, cudaStream_t s) {
  typedef CoreLayout<HD, MRM> L;
  static PerDevice ctas;
  int per_sm = 0;
  DFL_RET(ctas.get(&per_sm, [](int, int* v) {
    DFL_RET(cudaFuncSetAttribute(paged_attn_core_kernel<T, HD, MRM>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 L::kSmem));
    DFL_RET(cudaOccupancyMaxActiveBlocksPerMultiprocessor(v, paged_attn_core_kernel<T, HD, MRM>, kCoreThreads,
                                                          L::kSmem));
    *v = std::min(std::max(*v, 1), kPagedMaxCtas);
    return cudaSuccess;
  }));
  const PagedRule rule = paged_rule_core(g);
  if (rule.ri != L::MR) return cudaErrorInvalidValue;
  // runs of two tiles at least: 4 blocks of 16 rows over up to 1K keys take 17.4 us, 22.4 in runs of four
  if (paged_split(g, rule, num_sms() * per_sm, 2) > part_rows) return cudaErrorInvalidValue;
  const float scale_log2 = 1.4426950408889634f / sqrtf((float)HD);
  DFL_RET(launch_pdl(paged_attn_core_kernel<T, HD, MRM>, dim3(g.grid), dim3(kCoreThreads), L::kSmem, s, g, (const T*)q,
                     (const T*)kp, (const T*)vp, (T*)out, scale_log2));
  count_launch();
  return g.shared ? merge_launch<T, HD, kCoreKeys>(g, out, s) : cudaSuccess;  // (else the CTAs join their pieces)
}

cudaError_t paged_attention_core(int hd, const PagedGeom& g, const void* q, const void* kp, const void* vp,
                                 void* out, long long part_rows, cudaStream_t s) {
#define DFL_CORE(HD)                                                                         \
  return core_small(g) ? core_launch<float, HD, 1>(g, q, kp, vp, out, part_rows, s)          \
                       : core_launch<float, HD, 4>(g, q, kp, vp, out, part_rows, s)
  if (hd == 64) DFL_CORE(64);
  DFL_CORE(128);
#undef DFL_CORE
}

}  // namespace dfl
