// Attention over 8-bit pages (bf16 queries) on tensor cores fed from registers.
//
//   z_j = scale ks_j sum_d q_d (u_jd - 128),  o = sum_j 2^(z_j - m) vs_j (v_jd - 128) / sum_j 2^(z_j - m)   (log2 units)
//
// Codes less 128 are exact in half precision: the bytes 0x64 and u are the half
// 1024 + u, and 1152 taken off it leaves u - 128, so two codes take one byte
// permutation and one packed subtraction.  The queries are half too, each row
// scaled by a power of two to a largest entry of 2^7..2^8 (exact but for entries
// 2^25 below it).  The scales stay in float32: ks multiplies the scores, vs the
// weights.  A weight enters the product with the values as a pair of halves, w =
// 2^(z - m) vs f rounded and what that leaves: off by 2^-22 of itself, or by 2^-25, so
// that the outputs' own rounding is what tells (one half alone is off by 2^-11, and the
// outputs differed by 0.0009 from those of float32 weights, 0.0001 now).  f is a factor
// of the row that keeps its largest weight between 2^7 and 2^15, whatever size the scales
// have down to 2^-112; values of zero leave it at its most, so that the first other one
// sets it.  m and f move only when a weight outgrows that range (or a score m by 64),
// which a vote finds; the sum of weights is taken in float32 before vs and f.
//
// A step is 16 keys, always inside one page.  The products run over dimensions
// and keys in the order that suits the loads: a lane takes 16 consecutive bytes of
// a key row, swizzled against bank conflicts, and the queries, scores and outputs
// follow that order; nothing is shuffled between the two products.
//
// An item is up to 32 stacked rows, held by each of a CTA's four warps.  Up to 8 leave
// half of a row tile free: the second halves of the weights take it, and no product
// is added for them.  The warps take the steps of a run in turn, each with its own ring
// of stages (16-byte asynchronous copies) and its own running sums, so they run without
// a barrier; their sums are joined at a piece's end.  The split of a call over CTAs is
// that of paged.cuh, in tiles of 64 keys.
//
// Few rows are bound by the keys' bytes and by issue, most of it the codes' way to
// halves.  Up to 32 rows share that in pairs of row tiles; more go to the kernel that
// expands a key once for 128 rows.
//
// Measured: 32 tokens over 0.5K..36K keys, 40 / 8 heads, 190 us for 1.12 GB: 5.9 TB/s,
// 86% of the copy rate, 54% of the issue slots taken by 12 warps a multiprocessor (168
// registers).  (With both halves of the row tile computed and one half a weight: 213.)
// 8 blocks of 4 rows over 2K..6K keys, 32 / 8 heads, two products a tile of values:
// 38 us; of 8 rows 54.
#include <math.h>

#include <algorithm>
#include <type_traits>

#include "common.cuh"
#include "internal.h"
#include "paged.cuh"

namespace dfl {

namespace {
constexpr int kQ8Threads = 128;
constexpr int kQ8Keys = kPagedQ8Keys;
constexpr int kStep = 16;     // keys of a step
constexpr float kFactorLog2 = 120.f;  // a row's factor lies within 2^-120 and 2^120

// ROWS: stacked rows of an item, 8, 16 or 32.
template <int HD, int ROWS>
struct Q8Layout {
  static constexpr int kWarps = kQ8Threads / 32;
  static constexpr int kRows = ROWS;
  static constexpr int kTiles = ROWS == 32 ? 2 : 1;  // of 16 rows
  static constexpr int kHalves = ROWS == 8 ? 1 : 2;  // of a tile that hold rows
  static constexpr int kStages = 4;
  static constexpr int kStage = 2 * kStep * HD + 2 * kStep * 4;  // codes of keys and values, their scales
  static constexpr int kRing = kWarps * kStages * kStage;
  static constexpr int kQRow = HD * 2 + 16;               // padded: 8 rows of 16 bytes fall into 32 banks
  static constexpr int kPer = (HD / 4 + 2) * kHalves * 32;  // floats of a warp's sums of a row tile
  static constexpr int kJoin = (kWarps - 1) * kTiles * kPer * 4;  // those of the warps but the first, over the ring
  static constexpr int kRingEnd = kRing > kJoin ? kRing : kJoin;
  static constexpr int kQ = kRingEnd;
  static constexpr int kRf = kQ + kRows * kQRow;
  static constexpr int kSpan = kRf + kRows * 4;           // [rows] sink, lo, hi
  static constexpr int kRed = kSpan + kRows * 16;
  static constexpr int kSmem = kRed + (2 * kQ8Threads / 32 + 8) * 4;
  static constexpr int kCtas = ROWS <= 16 ? 3 : 2;
};

__device__ __forceinline__ void cp16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
// The upper 8 rows of the tile are zero.
__device__ __forceinline__ void ldsm2(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x2.shared.b16 {%0, %1}, [%2];" : "=r"(r[0]), "=r"(r[2]) : "r"(addr) : "memory");
  r[1] = r[3] = 0u;
}
__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// c = a b
__device__ __forceinline__ void mma_f16_first(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, "
      "%10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}
// Two codes (bytes 0 and 1, or 2 and 3 of w) less 128 as halves.
template <int HI>
__device__ __forceinline__ uint32_t two_codes(uint32_t w) {
  uint32_t d;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(__byte_perm(w, 0x64646464u, HI ? 0x4342 : 0x4140)), "r"(0x64806480u));
  return d;
}
__device__ __forceinline__ uint32_t half2_of(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// What rounding a pair of weights to the halves `hi` leaves.  (kInf: nothing where a half is infinite.)
template <bool kInf>
__device__ __forceinline__ uint32_t rest_of(float a, float b, uint32_t hi) {
  const float2 h = __half22float2(*reinterpret_cast<const __half2*>(&hi));
  if (kInf) return half2_of(isinf(h.x) ? 0.f : a - h.x, isinf(h.y) ? 0.f : b - h.y);
  return half2_of(a - h.x, b - h.y);
}
__device__ __forceinline__ float quad_max(float x) {
  x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
  return fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
}
__device__ __forceinline__ float quad_sum(float x) {
  x += __shfl_xor_sync(0xffffffffu, x, 1);
  return x + __shfl_xor_sync(0xffffffffu, x, 2);
}
// The key (of 8) that is column n of a score tile.
template <int HD>
__host__ __device__ __forceinline__ constexpr int key_of(int n) {
  return HD == 128 ? (n & 1) << 2 | n >> 1 : n;
}
// Byte offset of 16-byte chunk c of key row r: rows of 128 (64) bytes, chunks swizzled.
template <int HD>
__device__ __forceinline__ int chunk_at(int r, int c) {
  return HD == 128 ? r * 128 + ((c ^ (r & 7)) << 4) : r * 64 + ((c ^ ((r >> 1) & 3)) << 4);
}
}  // namespace

template <int HD, int ROWS>
__global__ void __launch_bounds__(kQ8Threads, (Q8Layout<HD, ROWS>::kCtas))
    paged_attn_q8_kernel(const __grid_constant__ PagedGeom g, const bf16* __restrict__ q,
                         const uint8_t* __restrict__ kp, const uint8_t* __restrict__ vp, bf16* __restrict__ out,
                         float scale_log2) {
  typedef Q8Layout<HD, ROWS> L;
  constexpr int KW = L::kWarps, S = L::kStages, NT = HD / 8, KS = HD / 16;  // output tiles, steps of 16 dimensions
  constexpr int MT = L::kTiles, YS = L::kHalves;
  extern __shared__ __align__(128) uint8_t smem[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, gr = lane >> 2, t = lane & 3;
  float* rfs = reinterpret_cast<float*>(smem + L::kRf);
  uint8_t* ring = smem + warp * S * L::kStage;
  const uint32_t ring_u = smem_u32(ring);
  pdl_launch();
  pdl_wait();
  const PlanView pv = plan_view<kQ8Keys, kQ8Threads>(g, reinterpret_cast<int*>(smem + L::kRed));
  SegmentWalk<kQ8Keys> walk(g, pv);
  walk.start();
  Segment sg;
  while (walk.next(sg)) {
    // ------------------------------------------------------------ queries: half, each row by a power of two
    __syncthreads();
    constexpr int kLanes = HD / 16;  // a lane takes 16 entries of a row
    for (int r = tid / kLanes; r < L::kRows; r += kQ8Threads / kLanes) {
      const ItemRow row = item_row(g, sg.prefix, sg.b, sg.hk, sg.rt * (sg.prefix ? g.rp : g.ri), r);
      const int c = tid % kLanes;
      float x[16];
      uint4 raw[2] = {make_uint4(0u, 0u, 0u, 0u), make_uint4(0u, 0u, 0u, 0u)};
      if (row.live) {
        const uint4* src =
            reinterpret_cast<const uint4*>(q + (((long long)row.b * g.n + row.i) * g.nq + row.head) * HD + 16 * c);
        raw[0] = src[0];
        raw[1] = src[1];
      }
      const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(raw);
      float most = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float2 f = __bfloat1622float2(h[e]);
        x[2 * e] = f.x;
        x[2 * e + 1] = f.y;
        most = fmaxf(most, fmaxf(fabsf(f.x), fabsf(f.y)));
      }
#pragma unroll
      for (int o = 1; o < kLanes; o <<= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
      // 2^up brings the largest entry to 2^7..2^8 (a row of zeros, or one that holds Inf: as it is)
      const int ex = (int)(__float_as_uint(most) >> 23);  // biased; 0: subnormal or zero
      const int up = ex > 0 && ex < 255 ? 134 - ex : ex == 0 && most > 0.f ? 133 : 0;
      // (up to 2^133: in two factors)
      const float u1 = exp2f((float)(up / 2)), u2 = exp2f((float)(up - up / 2));
      uint8_t* dst = smem + L::kQ + r * L::kQRow + ((c >> 2) * 64 + (c & 3) * 2) * 2;
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        *reinterpret_cast<uint32_t*>(dst + s * 32) = half2_of(x[4 * s] * u1 * u2, x[4 * s + 1] * u1 * u2);
        *reinterpret_cast<uint32_t*>(dst + s * 32 + 16) = half2_of(x[4 * s + 2] * u1 * u2, x[4 * s + 3] * u1 * u2);
      }
      if (c == 0) {
        int4 v = make_int4(0, 0, INT32_MAX, 0);
        if (row.live) row_span(g, paged_len(g, row.b), paged_rows(g, row.b), row.i, v.x, v.y, v.z);
        reinterpret_cast<int4*>(smem + L::kSpan)[r] = v;
        rfs[r] = exp2f((float)-up);
      }
    }
    __syncthreads();
    // ------------------------------------------------------------ the rows
    const uint32_t q_at = smem_u32(smem + L::kQ) +
                          (YS == 1 ? (uint32_t)((lane & 7) * L::kQRow + 16 * ((lane >> 3) & 1))
                                   : (uint32_t)(((lane & 7) + 8 * ((lane >> 3) & 1)) * L::kQRow + 16 * (lane >> 4)));
    const int key_lo = sg.prefix ? 0 : pv.sh_tiles * kQ8Keys;
    const int key_end = sg.prefix ? pv.sh_tiles * kQ8Keys : key_limit(g, sg.b);
    const int4* spans = reinterpret_cast<const int4*>(smem + L::kSpan) + gr;
    int all_lo = key_lo, all_hi = key_end;  // keys that every row sees
    float rf[MT][YS], m[MT][YS], l[MT][YS], f[MT][YS];
    float o[MT][NT][4];  // (YS == 1: the last two are the sums of the weights' second halves)
#pragma unroll
    for (int a = 0; a < MT; ++a)
#pragma unroll
      for (int y = 0; y < YS; ++y) {
        const int4 v = spans[a * 16 + 8 * y];
        all_lo = max(all_lo, v.y);
        all_hi = min(all_hi, v.z);
        rf[a][y] = rfs[a * 16 + gr + 8 * y];
        m[a][y] = -INFINITY;
        l[a][y] = 0.f;
        f[a][y] = 1.f;
      }
    all_lo = __reduce_max_sync(0xffffffffu, all_lo);
    all_hi = __reduce_min_sync(0xffffffffu, all_hi);
#pragma unroll
    for (int a = 0; a < MT; ++a)
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[a][i][e] = 0.f;
    // some row of the item sees the keys below seen_sink and those from seen_lo on: its first row's
    int seen_sink, seen_lo, seen_hi;
    row_span(g, sg.prefix ? pv.min_len : paged_len(g, sg.b), paged_rows(g, sg.b),
             sg.prefix ? 0 : div_g(g, sg.rt * g.ri), seen_sink, seen_lo, seen_hi);
    // ------------------------------------------------------------ the ring
    const int steps = sg.nt * (kQ8Keys / kStep) / KW;  // of this warp: warp, warp + KW, ..
    auto first_key = [&](int j) {
      const int s = j * KW + warp;
      return sg.span.tile(sg.t0 + s / (kQ8Keys / kStep)) * kQ8Keys + s % (kQ8Keys / kStep) * kStep;
    };
    const int32_t* trow = g.table + (long long)sg.b * g.table_stride;
    int pages = -1;        // lane x: the page of step x of the 32 at hand (-1: none, or no row sees a key of it)
    uint32_t there = 0u;   // bit j % 32: step j has been asked for
    const uint32_t put0 = chunk_at<HD>(lane / (HD / 16), lane % (HD / 16));
    uint32_t ask_slot = 0, slot = 0;
    auto ask = [&](int j) {
      if (j < steps) {
        if ((j & 31) == 0) {
          const int k0 = j + lane < steps ? first_key(j + lane) : INT32_MAX;
          pages = -1;
          if (k0 < key_end && (k0 < seen_sink || k0 + kStep > seen_lo)) {
            pages = trow[k0 >> g.ps_log2];
            if ((unsigned)pages >= (unsigned)g.n_pages) {
              pages = -1;
              set_status(g.status, DFLASH_STATUS_BOUNDS);
            }
          }
        }
        const int page = __shfl_sync(0xffffffffu, pages, j & 31);
        there = (there & ~(1u << (j & 31))) | (uint32_t)(page >= 0) << (j & 31);
        if (page >= 0) {
          // (pool rows are below 2^31)
          const int row = (int)g.page_row0 + (page * g.nkv + sg.hk) * g.ps + (first_key(j) & (g.ps - 1));
          const uint32_t at = ring_u + ask_slot * L::kStage;
          const long long src = (long long)row * HD + lane * 16;
#pragma unroll
          for (int x = 0; x < kStep * HD / 512; ++x) {
            // row lane / (HD / 16) + x 512 / HD: the swizzle changes with x only where 4 rows a load are 128 bytes each
            const uint32_t to = at + (HD == 128 && (x & 1) ? put0 ^ 64u : put0) + x * 512;
            cp16(to, kp + src + x * 512);
            cp16(to + kStep * HD, vp + src + x * 512);
          }
          if (lane < 8) cp16(at + 2 * kStep * HD + lane * 16, (lane < 4 ? g.ks : g.vs) + row + 4 * (lane & 3));
        }
      }
      if (++ask_slot == S) ask_slot = 0;
      cp_commit();
    };
#pragma unroll 1
    for (int j = 0; j < S - 1; ++j) ask(j);
#pragma unroll 1
    for (int j = 0; j < steps; ++j) {
      cp_wait<S - 2>();
      __syncwarp();
      ask(j + S - 1);
      const uint8_t* kb = ring + slot * L::kStage;
      if (++slot == S) slot = 0;
      if (!(there >> (j & 31) & 1u)) continue;
      const uint8_t* vb = kb + kStep * HD;
      const float* sc = reinterpret_cast<const float*>(vb + kStep * HD);
      const int k0 = first_key(j);
      // ---------------------------------------------------------- scores
      float c[MT][2][4];
      uint4 kc[2][HD / 64];
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int h = 0; h < HD / 64; ++h)
          kc[n][h] = *reinterpret_cast<const uint4*>(kb + chunk_at<HD>(8 * n + key_of<HD>(gr), t + 4 * h));
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        uint32_t b[2][2];
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          const uint4 v = kc[n][s >> 2];
          const uint32_t word = (s & 3) == 0 ? v.x : (s & 3) == 1 ? v.y : (s & 3) == 2 ? v.z : v.w;
          b[n][0] = two_codes<0>(word);
          b[n][1] = two_codes<1>(word);
        }
#pragma unroll
        for (int a = 0; a < MT; ++a) {
          uint32_t x[4];
          if (YS == 1)
            ldsm2(x, q_at + s * 32);
          else
            ldsm4(x, q_at + a * 16 * L::kQRow + s * 32);
#pragma unroll
          for (int n = 0; n < 2; ++n)
            if (s == 0)
              mma_f16_first(c[a][n], x, b[n][0], b[n][1]);
            else
              mma_f16(c[a][n], x, b[n][0], b[n][1]);
        }
      }
      // ---------------------------------------------------------- weights
      // this lane's keys: columns 2 t, 2 t + 1 of both score tiles
      const int kx[4] = {key_of<HD>(2 * t), key_of<HD>(2 * t + 1), 8 + key_of<HD>(2 * t), 8 + key_of<HD>(2 * t + 1)};
      float ks[4], vs[4];
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        ks[x] = sc[kx[x]] * scale_log2;
        vs[x] = sc[kStep + kx[x]];
      }
      const bool part = k0 < all_lo || k0 + kStep > all_hi;
      uint32_t p[MT][4], pl[MT][4];  // weights: their first halves and (YS == 2) their second ones
      auto weights = [&](auto masked) {
        constexpr bool kMasked = decltype(masked)::value;
        uint32_t hidden = 0u;  // bit 8 a + 4 y + x
#pragma unroll
        for (int a = 0; a < MT; ++a)
#pragma unroll
          for (int i = 0; i < 4 * YS; ++i) {
            const int y = i >> 2, x = i & 3;
            const int4 see = kMasked ? spans[a * 16 + 8 * y] : make_int4(0, 0, 0, 0);
            float& z = c[a][x >> 1][2 * y + (x & 1)];
            z *= ks[x];
            if (kMasked) {
              const int key = k0 + kx[x];
              if (!(key >= key_lo && key < key_end && (key < see.x || (key >= see.y && key < see.z)))) {
                z = -INFINITY;
                hidden |= 1u << (8 * a + i);
              }
            }
          }
        float sum[MT][YS];
        // Weights as the rows' references and factors have them; true if some row's have to move.  (Without a
        // reference every score that is seen makes one.)
        auto weigh = [&](auto again) {
          constexpr bool kInf = decltype(again)::value;
          bool move = false;
#pragma unroll
          for (int a = 0; a < MT; ++a)
#pragma unroll
            for (int y = 0; y < YS; ++y) {
              const bool none = m[a][y] == -INFINITY;
              const float off = none ? 0.f : -m[a][y] * rf[a][y];
              float w[4], e[4];
              sum[a][y] = 0.f;
#pragma unroll
              for (int x = 0; x < 4; ++x) {
                e[x] = fmaf(c[a][x >> 1][2 * y + (x & 1)], rf[a][y], off);
                const float pr = ex2f(e[x]);
                sum[a][y] += pr;
                const bool hide = kMasked && (hidden >> (8 * a + 4 * y + x) & 1u);
                // (the scale first: a factor for small values, times the scale of a large one that has next to no
                // weight, may be past float32)
                w[x] = pr * (hide ? 0.f : vs[x]) * f[a][y];
              }
              move |= fmaxf(fmaxf(e[0], e[1]), fmaxf(e[2], e[3])) > (none ? -INFINITY : 64.f);
              move |= fmaxf(fmaxf(fabsf(w[0]), fabsf(w[1])), fmaxf(fabsf(w[2]), fabsf(w[3]))) > 32768.f;
              p[a][y] = half2_of(w[0], w[1]);
              p[a][2 + y] = half2_of(w[2], w[3]);
              uint32_t(&lo)[4] = YS == 1 ? p[a] : pl[a];
              lo[YS == 1 ? 1 : y] = rest_of<kInf>(w[0], w[1], p[a][y]);
              lo[YS == 1 ? 3 : 2 + y] = rest_of<kInf>(w[2], w[3], p[a][2 + y]);
            }
          return move;
        };
        if (__any_sync(0xffffffffu, weigh(std::false_type()))) {  // (an infinite weight too)
#pragma unroll
          for (int a = 0; a < MT; ++a)
#pragma unroll
            for (int y = 0; y < YS; ++y) {
              float z[4], zm = -INFINITY;
#pragma unroll
              for (int x = 0; x < 4; ++x) {
                z[x] = c[a][x >> 1][2 * y + (x & 1)];
                zm = fmaxf(zm, z[x]);
              }
              const float mn = fmaxf(m[a][y], quad_max(zm)), r = rf[a][y];
              const bool has = mn > -INFINITY, first = m[a][y] == -INFINITY;
              float tm = 0.f;
#pragma unroll
              for (int x = 0; x < 4; ++x)
                tm = fmaxf(tm, kMasked && (hidden >> (8 * a + 4 * y + x) & 1u)
                                   ? 0.f
                                   : ex2f((z[x] - (has ? mn : 0.f)) * r) * fabsf(vs[x]));
              tm = quad_max(tm);
              const float dm = first || !has ? 0.f : (mn - m[a][y]) * r;  // (in log2 units)
              // this step's weights are brought within 2^8 (values of zero leave the factor at its most, so that the
              // next ones set it); those before it keep their factor unless it has to fall
              const float want = tm > 0.f ? 8.f - log2f(tm) : kFactorLog2, was = log2f(f[a][y]);
              const float keep = first ? want : was + dm;
              const bool fall = !first && tm > 0.f && exp2f(fminf(keep, 126.f)) * tm > 32768.f;
              const float to = fminf(fmaxf(fall ? want : keep, -kFactorLog2), kFactorLog2);
              const float os = first ? 1.f : exp2f(to - keep);
              if (has) {
                l[a][y] *= ex2f(-dm);
                m[a][y] = mn;
                if (to != was) f[a][y] = exp2f(to);
#pragma unroll
                for (int i = 0; i < NT; ++i)
#pragma unroll
                  for (int e = 0; e < 4 / YS; ++e) o[a][i][2 * y + e] *= os;
              }
            }
          weigh(std::true_type());
        }
#pragma unroll
        for (int a = 0; a < MT; ++a)
#pragma unroll
          for (int y = 0; y < YS; ++y) l[a][y] += sum[a][y];
      };
      if (part)
        weights(std::true_type());
      else
        weights(std::false_type());
      // ---------------------------------------------------------- values
      if constexpr (HD == 128) {
        uint4 vc[4];
#pragma unroll
        for (int x = 0; x < 4; ++x)
          vc[x] = *reinterpret_cast<const uint4*>(vb + chunk_at<HD>(kx[x], (gr & 1) << 2 | gr >> 1));
#pragma unroll
        for (int d = 0; d < 4; ++d) {  // 4 dimensions
          uint32_t word[4];
#pragma unroll
          for (int x = 0; x < 4; ++x) word[x] = d == 0 ? vc[x].x : d == 1 ? vc[x].y : d == 2 ? vc[x].z : vc[x].w;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t ab = __byte_perm(word[0], word[1], h ? 0x7362 : 0x5140);
            const uint32_t cd = __byte_perm(word[2], word[3], h ? 0x7362 : 0x5140);
            const uint32_t b0 = two_codes<0>(ab), b1 = two_codes<0>(cd), b2 = two_codes<1>(ab), b3 = two_codes<1>(cd);
#pragma unroll
            for (int a = 0; a < MT; ++a) {
              mma_f16(o[a][4 * d + 2 * h], p[a], b0, b1);
              mma_f16(o[a][4 * d + 2 * h + 1], p[a], b2, b3);
              if (YS == 2) {
                mma_f16(o[a][4 * d + 2 * h], pl[a], b0, b1);
                mma_f16(o[a][4 * d + 2 * h + 1], pl[a], b2, b3);
              }
            }
          }
        }
      } else {
        uint2 vc[4];
#pragma unroll
        for (int x = 0; x < 4; ++x)
          vc[x] = *reinterpret_cast<const uint2*>(vb + chunk_at<HD>(kx[x], gr >> 1) + (gr & 1) * 8);
#pragma unroll
        for (int d = 0; d < 2; ++d) {
          uint32_t word[4];
#pragma unroll
          for (int x = 0; x < 4; ++x) word[x] = d ? vc[x].y : vc[x].x;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t ab = __byte_perm(word[0], word[1], h ? 0x7362 : 0x5140);
            const uint32_t cd = __byte_perm(word[2], word[3], h ? 0x7362 : 0x5140);
            const uint32_t b0 = two_codes<0>(ab), b1 = two_codes<0>(cd), b2 = two_codes<1>(ab), b3 = two_codes<1>(cd);
#pragma unroll
            for (int a = 0; a < MT; ++a) {
              mma_f16(o[a][4 * d + 2 * h], p[a], b0, b1);
              mma_f16(o[a][4 * d + 2 * h + 1], p[a], b2, b3);
              if (YS == 2) {
                mma_f16(o[a][4 * d + 2 * h], pl[a], b0, b1);
                mma_f16(o[a][4 * d + 2 * h + 1], pl[a], b2, b3);
              }
            }
          }
        }
      }
    }
    cp_wait<0>();
    // ------------------------------------------------------------ the rows' sums: (m, l, o) with o as m has it
#pragma unroll
    for (int a = 0; a < MT; ++a)
#pragma unroll
      for (int y = 0; y < YS; ++y) {
        l[a][y] = quad_sum(l[a][y]);
        m[a][y] = m[a][y] == -INFINITY ? -INFINITY : m[a][y] * rf[a][y];
        const float back = 1.f / f[a][y];
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
          for (int e = 0; e < 2; ++e) o[a][i][2 * y + e] = (YS == 1 ? o[a][i][e] + o[a][i][2 + e] : o[a][i][2 * y + e]) * back;
      }
    __syncthreads();  // (the rings are free)
    float* join = reinterpret_cast<float*>(smem);
    constexpr int kPer = L::kPer;
    if (warp > 0) {
#pragma unroll
      for (int a = 0; a < MT; ++a) {
        float* dst = join + ((warp - 1) * MT + a) * kPer + lane;
#pragma unroll
        for (int i = 0; i < NT * 2 * YS; ++i) dst[i * 32] = o[a][i / (2 * YS)][i % (2 * YS)];
#pragma unroll
        for (int y = 0; y < YS; ++y) {
          dst[(NT * 2 * YS + y) * 32] = m[a][y];
          dst[(NT * 2 * YS + YS + y) * 32] = l[a][y];
        }
      }
    }
    __syncthreads();
    if (warp == 0) {
#pragma unroll
      for (int a = 0; a < MT; ++a)
#pragma unroll 1
        for (int k = 0; k < KW - 1; ++k) {
          const float* src = join + (k * MT + a) * kPer + lane;
          float x0[YS], x1[YS];
#pragma unroll
          for (int y = 0; y < YS; ++y) {
            const float m1 = src[(NT * 2 * YS + y) * 32], l1 = src[(NT * 2 * YS + YS + y) * 32];
            const float mn = fmaxf(m[a][y], m1);
            x0[y] = m[a][y] == -INFINITY ? 0.f : ex2f(m[a][y] - mn);
            x1[y] = m1 == -INFINITY ? 0.f : ex2f(m1 - mn);
            l[a][y] = l[a][y] * x0[y] + l1 * x1[y];
            m[a][y] = mn;
          }
#pragma unroll
          for (int i = 0; i < NT * 2 * YS; ++i) {
            const int e = i % (2 * YS), y = e >> 1;
            float& sum = o[a][i / (2 * YS)][e];
            sum = sum * x0[y] + src[i * 32] * x1[y];
          }
        }
    }
    const bool whole = walk.whole(sg);
    if (warp == 0) {
#pragma unroll
      for (int a = 0; a < MT; ++a)
#pragma unroll
        for (int y = 0; y < YS; ++y) {
          const int r = a * 16 + gr + 8 * y;
          const ItemRow row = item_row(g, sg.prefix, sg.b, sg.hk, sg.rt * (sg.prefix ? g.rp : g.ri), r);
          if (!row.live) continue;
          // dimension 16 t + i of output tile i in column 2 t, and column 2 t + 1: 64 further (HD = 64: 8 further)
          constexpr int kFar = HD == 128 ? 64 : 8;
          if (whole) {
            const float inv = 1.f / l[a][y];
            bf16* dst = out + (((long long)row.b * g.n + row.i) * g.nq + row.head) * HD + 16 * t;
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
              for (int i = 0; i < NT; i += 8) {
                uint4 v;
                __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&v);
#pragma unroll
                for (int x = 0; x < 4; ++x)
                  h[x] = __floats2bfloat162_rn(o[a][i + 2 * x][2 * y + e] * inv, o[a][i + 2 * x + 1][2 * y + e] * inv);
                *reinterpret_cast<uint4*>(dst + e * kFar + i) = v;
              }
          } else {
            float* dst = g.part_o + (sg.slot_row + r) * HD + 16 * t;
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
              for (int i = 0; i < NT; i += 4)
                *reinterpret_cast<float4*>(dst + e * kFar + i) = make_float4(
                    o[a][i][2 * y + e], o[a][i + 1][2 * y + e], o[a][i + 2][2 * y + e], o[a][i + 3][2 * y + e]);
            if (t == 0) g.part_ml[sg.slot_row + r] = make_float2(m[a][y], l[a][y]);
          }
        }
    }
    if (!whole && pv.pre_tiles == 0) {
      int c0;
      const int nc = walk.pieces(sg, c0);
      int* done = reinterpret_cast<int*>(smem + L::kRed);
      __syncthreads();
      if (tid == 0) {
        __threadfence();
        *done = atomicAdd(g.tickets + sg.ordinal, 1) == nc - 1;
      }
      __syncthreads();
      if (*done) {
        __threadfence();
        if (tid == 0) g.tickets[sg.ordinal] = 0;
        merge_item<bf16, HD>(g, sg.b, sg.rt, sg.hk, 0, min(g.ri, paged_rows(g, sg.b) * g.G - sg.rt * g.ri), nc, c0, warp,
                             kQ8Threads / 32, out);
      }
    }
  }
}

// Stacked rows that one sequence's queries, or the batch's behind a shared prefix, make.  (The batch's choose for the
// sequences' own keys too: 32 tokens behind 64 common keys and 2K..8K of their own take 216 us, without the shared
// length 68.)
static int q8_stack(const PagedGeom& g) { return (g.shared ? g.batch : 1) * g.n * g.G; }
// Up to 32 rows a key's codes are expanded for one or two row tiles; beyond, once for 128 rows.  At 32 rows (8 sequences,
// 2K..6K keys) 54 us here and 58 there, at 30 over 0.5K..36K keys 147 and 179, at 16 38 and 56; at 64 83 (in groups of
// warps, with one half a weight) and 63.
constexpr int kFewRows = 32;
PagedRule paged_rule_q8(const PagedGeom& g) {
  const int rows = q8_stack(g);
  if (rows > kFewRows) return paged_rule_q8_tc();
  const int of = rows <= 8 ? 8 : rows <= 16 ? 16 : 32;
  return PagedRule{of, of, kQ8Keys, 1, 2};
}

template <int HD, int ROWS>
static cudaError_t q8_launch(PagedGeom g, const void* q, const void* kp, const void* vp, void* out, long long part_rows,
                             cudaStream_t s) {
  typedef Q8Layout<HD, ROWS> L;
  static_assert(L::kSmem * L::kCtas <= 232448, "shared memory per multiprocessor");
  static PerDevice smem;
  DFL_RET(smem.once([] {
    return cudaFuncSetAttribute(paged_attn_q8_kernel<HD, ROWS>, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kSmem);
  }));
  if (paged_split(g, paged_rule_q8(g), num_sms() * L::kCtas, 2) > part_rows || g.ri != L::kRows)
    return cudaErrorInvalidValue;
  const float scale_log2 = 1.4426950408889634f / sqrtf((float)HD);
  DFL_RET(launch_pdl(paged_attn_q8_kernel<HD, ROWS>, dim3(g.grid), dim3(kQ8Threads), L::kSmem, s, g, (const bf16*)q,
                     (const uint8_t*)kp, (const uint8_t*)vp, (bf16*)out, scale_log2));
  count_launch();
  return g.shared ? paged_merge_q8(HD, g, out, s) : cudaSuccess;  // (else the CTAs join their pieces)
}

template <int HD>
static cudaError_t q8_pick(const PagedGeom& g, const void* q, const void* kp, const void* vp, void* out,
                           long long part_rows, cudaStream_t s) {
  const int rows = q8_stack(g);
  return rows <= 8    ? q8_launch<HD, 8>(g, q, kp, vp, out, part_rows, s)
         : rows <= 16 ? q8_launch<HD, 16>(g, q, kp, vp, out, part_rows, s)
                      : q8_launch<HD, 32>(g, q, kp, vp, out, part_rows, s);
}

cudaError_t paged_attention_q8(int hd, const PagedGeom& g, const void* q, const void* kp, const void* vp, void* out,
                               long long part_rows, cudaStream_t s) {
  if (q8_stack(g) > kFewRows) return paged_attention_q8_tc(hd, g, q, kp, vp, out, part_rows, s);
  return hd == 64 ? q8_pick<64>(g, q, kp, vp, out, part_rows, s) : q8_pick<128>(g, q, kp, vp, out, part_rows, s);
}

}  // namespace dfl
