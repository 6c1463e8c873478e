// Attention of many rows over 8-bit pages (bf16 queries) on the 5th-generation
// tensor cores.
//
//   z_j = scale ks_j sum_d q_d (u_jd - 128),  o = sum_j 2^(z_j - m) vs_j (v_jd - 128) / sum_j 2^(z_j - m)   (log2 units)
//
// The arithmetic is that of the kernel for few rows: codes less 128 are exact in
// half precision, queries are half, each row scaled by a power of two, ks
// multiplies the scores in float32, and a weight enters the product with the values
// as half(2^(z - m) vs f), f a factor of the row that keeps the largest below 2^15.
//
// An item is up to 128 stacked rows, one to a thread.  A tile of 64 keys goes
//   pages -> registers (one tile ahead; the pages' numbers two ahead)
//         -> halves in shared memory, two buffers, K and V rows alike, swizzled
//   S = Q K^T   128 rows by 64 keys in TMEM: a thread reads its row
//   O += P V    P as halves in TMEM, O in TMEM
// so a key's codes are expanded once for all rows, while the products of the tile
// before run.  One barrier a tile; two CTAs share an SM, and one's products run
// under the other's exponentials.  The split of a call over CTAs is that of
// paged.cuh; pieces of items are joined by a second kernel.
//
// Every wait is bounded (PagedGeom::wait_ns); one that gives up sets
// DFLASH_STATUS_TIMEOUT, and the CTA drains its products, whatever the limit, and
// ends.
#include <math.h>

#include <algorithm>

#include "common.cuh"
#include "internal.h"
#include "paged.cuh"

namespace dfl {

namespace {
constexpr int kThreads = 128;
constexpr int kKeys = kPagedQ8Keys;
constexpr int kRows = 128;
constexpr uint64_t kDrainNs = 125000000ull;

template <int HD>
struct Q8TcLayout {
  static constexpr int kHalves = HD / 64;              // 64 dimensions: rows of 128 bytes
  static constexpr int kTile = kHalves * kKeys * 128;  // 64 keys or values
  static constexpr int kQ = 0;
  static constexpr int kK = kHalves * kRows * 128;     // [2]
  static constexpr int kV = kK + 2 * kTile;            // [2]
  static constexpr int kScales = kV + 2 * kTile;       // [2][ks, vs][64]
  static constexpr int kRed = kScales + 2 * 2 * kKeys * 4;
  static constexpr int kUsed = kRed + (2 * kThreads / 32 + 8) * 4;
  static constexpr int kSmem = kUsed + 1024;
};

__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("mul.rn.f32x2 %0, %1, %2;"
      : "=l"(reinterpret_cast<uint64_t&>(d))
      : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("add.rn.f32x2 %0, %1, %2;"
      : "=l"(reinterpret_cast<uint64_t&>(d))
      : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)));
  return d;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ uint32_t half2_of(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// 16 codes less 128 as halves: two 16-byte chunks.
__device__ __forceinline__ void halves_of(const uint4& u, uint4 (&h)[2]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
  uint32_t* out = reinterpret_cast<uint32_t*>(h);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    uint32_t d;
    asm("sub.rn.f16x2 %0, %1, %2;"
        : "=r"(d)
        : "r"(__byte_perm(w[i >> 1], 0x64646464u, i & 1 ? 0x4342 : 0x4140)), "r"(0x64806480u));
    out[i] = d;
  }
}
// Bits [a, b) of a word, clamped to it.
__device__ __forceinline__ uint32_t bits_of(int a, int b) {
  a = max(a, 0);
  b = min(b, 32);
  if (a >= b) return 0u;
  return (b >= 32 ? 0xffffffffu : (1u << b) - 1u) & ~((1u << a) - 1u);
}
// A phase is over, waited for up to the limit (0: it has expired).
__device__ __forceinline__ bool over(uint64_t* bar, uint32_t parity, unsigned limit_ns) {
  if (limit_ns != 0 && mbar_try_wait(bar, parity)) return true;
  return mbar_wait(bar, parity, limit_ns);
}
}  // namespace

template <int HD>
__global__ void __launch_bounds__(kThreads, 2)
    paged_attn_q8_tc_kernel(const __grid_constant__ PagedGeom g, const bf16* __restrict__ q,
                            const uint8_t* __restrict__ kp, const uint8_t* __restrict__ vp, bf16* __restrict__ out,
                            float scale_log2) {
  typedef Q8TcLayout<HD> L;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t s_done, pv_done;
  __shared__ uint32_t tmem_slot;
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  float* scales = reinterpret_cast<float*>(sm + L::kScales);
  if (tid == 0) {
    mbar_init(&s_done, 1);
    mbar_init(&pv_done, 1);
    fence_barrier_init();
  }
  if (warp == 0) {
    __syncwarp();
    tmem_alloc(&tmem_slot, 256);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot, tO = tmem, tS = tmem + 128, tP = tmem + 192;
  const uint32_t lanes = (uint32_t)(32 * warp) << 16;
  pdl_launch();
  pdl_wait();
  const PlanView pv = plan_view<kKeys, kThreads>(g, reinterpret_cast<int*>(sm + L::kRed));
  SegmentWalk<kKeys> walk(g, pv);
  walk.start();
  Segment sg;
  int seg = 0;
  uint32_t s_n = 0, pv_n = 0;  // score products and value products asked for
  bool ok = true;
  constexpr uint32_t idS = idesc_f16_f32(128, kKeys), idO = idesc_f16_f32(128, HD) | (1u << 16);  // values MN-major
  while (true) {
    const bool more = walk.next(sg);
    if (seg == 0 && !g.shared) {
      // the item that this CTA's run begins inside of, when it is the second to hold a piece of it
      int c0 = 0, nc = 0;
      if (more && sg.t0 > 0) nc = walk.pieces(sg, c0);
      if (c0 + 1 != (int)blockIdx.x) nc = 0;
      int4* rec = reinterpret_cast<int4*>(g.records) + 2 * blockIdx.x;
      if (tid == 0) {
        rec[0] = make_int4(nc, sg.b, sg.rt, sg.hk);
        rec[1].x = c0;
      }
    }
    if (!more) break;
    ++seg;
    const int x0 = sg.rt * (sg.prefix ? g.rp : g.ri);
    const ItemRow mine = item_row(g, sg.prefix, sg.b, sg.hk, x0, tid);
    // ------------------------------------------------------------ queries: half, each row by a power of two
    float rf = 1.f;
    int sink = 0, lo = 0, hi = INT32_MAX;
    {
      const uint4* src = reinterpret_cast<const uint4*>(
          q + (((long long)mine.b * g.n + mine.i) * g.nq + mine.head) * HD);
      float most = 0.f;
      if (mine.live) {
        row_span(g, paged_len(g, mine.b), paged_rows(g, mine.b), mine.i, sink, lo, hi);
#pragma unroll 4
        for (int c = 0; c < HD / 8; ++c) {
          const uint4 u = src[c];
          const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&u);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 f = __bfloat1622float2(h[e]);
            most = fmaxf(most, fmaxf(fabsf(f.x), fabsf(f.y)));
          }
        }
      }
      // 2^up brings the largest entry to 2^7..2^8 (a row of zeros, or one that holds Inf: as it is)
      const int ex = (int)(__float_as_uint(most) >> 23);
      const int up = ex > 0 && ex < 255 ? 134 - ex : ex == 0 && most > 0.f ? 133 : 0;
      const float u1 = exp2f((float)(up / 2)), u2 = exp2f((float)(up - up / 2));
      rf = exp2f((float)-up);
#pragma unroll 4
      for (int c = 0; c < HD / 8; ++c) {
        uint4 u = make_uint4(0u, 0u, 0u, 0u);
        if (mine.live) u = src[c];
        const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&u);
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 f = __bfloat1622float2(h[e]);
          w[e] = half2_of(f.x * u1 * u2, f.y * u1 * u2);
        }
        *reinterpret_cast<uint4*>(sm + L::kQ + (c >> 3) * (kRows * 128) + tid * 128 + (((c & 7) ^ (tid & 7)) << 4)) =
            make_uint4(w[0], w[1], w[2], w[3]);
      }
    }
    const int key_lo = sg.prefix ? 0 : pv.sh_tiles * kKeys;
    const int key_end = sg.prefix ? pv.sh_tiles * kKeys : key_limit(g, sg.b);
    const int all_lo = __reduce_max_sync(0xffffffffu, max(key_lo, lo));
    const int all_hi = __reduce_min_sync(0xffffffffu, min(key_end, hi));
    const bool idle = __all_sync(0xffffffffu, !mine.live);  // none of the warp's rows is one
    int seen_sink, seen_lo, seen_hi;
    row_span(g, sg.prefix ? pv.min_len : paged_len(g, sg.b), paged_rows(g, sg.b),
             sg.prefix ? 0 : div_g(g, sg.rt * g.ri), seen_sink, seen_lo, seen_hi);
    // ------------------------------------------------------------ keys and values
    // A thread takes 16 bytes of every kStep-th key row: whole rows by neighbours.  Every 16 keys lie in one page.
    constexpr int kLanes = HD / 16, kStep = kThreads / kLanes, KU = kKeys / kStep;
    const int kr = tid / kLanes, kc16 = tid % kLanes;
    const int32_t* trow = g.table + (long long)sg.b * g.table_stride;
    // The page of the 16 keys 16 (lane % 4) .. of tile i (-1: no row sees one of them): asked for a tile before it is
    // looked at.
    auto key_of = [&](int i) { return sg.span.tile(sg.t0 + i) * kKeys + 16 * (lane & 3); };
    auto page_of = [&](int i) {
      if (i >= sg.nt) return -1;
      const int key = key_of(i);
      return key >= key_end || (key >= seen_sink && key + 16 <= seen_lo) ? -1 : trow[key >> g.ps_log2];
    };
    uint4 kc[KU], vc[KU];
    float sc = 0.f;
    // (Keys that no row sees, and those of a bad page: some row of the pool; what they hold is masked, or the sequence's
    // result unspecified.)
    auto fetch = [&](int i, int page) {
      if (i >= sg.nt) return;
      int first = 0;  // the pool row of the 16 keys (below 2^31)
      if ((unsigned)page < (unsigned)g.n_pages)
        first = (int)g.page_row0 + (page * g.nkv + sg.hk) * g.ps + (key_of(i) & (g.ps - 1));
      else if (page != -1)
        set_status(g.status, DFLASH_STATUS_BOUNDS);
#pragma unroll
      for (int u = 0; u < KU; ++u) {
        const int key = kr + kStep * u;
        const long long at = (long long)(__shfl_sync(0xffffffffu, first, key >> 4) + (key & 15)) * HD + 16 * kc16;
        kc[u] = __ldg(reinterpret_cast<const uint4*>(kp + at));
        vc[u] = __ldg(reinterpret_cast<const uint4*>(vp + at));
      }
      const int key = tid & 63;
      sc = __ldg((tid < 64 ? g.ks : g.vs) + __shfl_sync(0xffffffffu, first, key >> 4) + (key & 15));
    };
    auto expand = [&](int buf) {
      // 16 codes are two chunks of 16 bytes; lanes of the upper half of a row write theirs the other way round, so
      // that the 8 lanes of a row fill all banks
      const int c = 2 * (kc16 & 3), far = kc16 >> 2;
#pragma unroll
      for (int u = 0; u < KU; ++u) {
        const int key = kr + kStep * u;
        uint8_t* base = sm + far * (kKeys * 128) + buf * L::kTile + key * 128;
        const int p0 = ((c + far) ^ (key & 7)) << 4, p1 = ((c + 1 - far) ^ (key & 7)) << 4;
        uint4 h[2];
        halves_of(kc[u], h);
        *reinterpret_cast<uint4*>(base + L::kK + p0) = far ? h[1] : h[0];
        *reinterpret_cast<uint4*>(base + L::kK + p1) = far ? h[0] : h[1];
        halves_of(vc[u], h);
        *reinterpret_cast<uint4*>(base + L::kV + p0) = far ? h[1] : h[0];
        *reinterpret_cast<uint4*>(base + L::kV + p1) = far ? h[0] : h[1];
      }
      scales[2 * buf * kKeys + tid] = tid < 64 ? sc * scale_log2 : sc;
    };
    auto scores = [&](int buf) {  // one thread
      const uint64_t dq = smem_desc_sw128(sm + L::kQ), dk = smem_desc_sw128(sm + L::kK + buf * L::kTile);
#pragma unroll
      for (int k = 0; k < HD / 16; ++k)
        tc_mma_f16(tS, dq + (uint64_t)((k >> 2) * (kRows * 128 / 16) + 2 * (k & 3)),
                   dk + (uint64_t)((k >> 2) * (kKeys * 128 / 16) + 2 * (k & 3)), idS, k > 0);
      tc_commit(&s_done);
    };
    int next_page = page_of(0);
    fetch(0, next_page);
    next_page = page_of(1);
    expand(0);
    fetch(1, next_page);
    next_page = page_of(2);
    fence_proxy_async_smem();
    tc_fence_before();
    if (__syncthreads_or(!ok)) break;
    if (warp == 0) {
      if (elect_one()) {
        tc_fence_after();
        scores(0);
      }
      __syncwarp();
    }
    ++s_n;
    float m = -INFINITY, l = 0.f, f = 1.f;
    for (int i = 0; i < sg.nt; ++i) {
      // the value products of tile i - 1: their weights, their values and the other keys' buffer are free
      if (i > 0) ok = ok && over(&pv_done, (pv_n - 1) & 1u, g.wait_ns);
      if (i + 1 < sg.nt) {
        expand((i + 1) & 1);
        fetch(i + 2, next_page);
        next_page = page_of(i + 3);
      }
      ok = ok && over(&s_done, (s_n - 1) & 1u, g.wait_ns);
      ok = __all_sync(0xffffffffu, ok);
      tc_fence_after();
      if (ok && !idle) {
        const float* ks = scales + 2 * (i & 1) * kKeys;
        const float* vs = ks + kKeys;
        const int k0 = sg.span.tile(sg.t0 + i) * kKeys;
        uint32_t s[2][32];
        tmem_ld32(tS + lanes, s[0]);
        tmem_ld32(tS + 32 + lanes, s[1]);
        // the largest scale of the tile's values (of hidden slots too: it only says when to look closer)
        const float va = fabsf(vs[lane]), vb = fabsf(vs[lane + 32]);
        const float vmax = __uint_as_float(__reduce_max_sync(
            0xffffffffu, max(va < INFINITY ? __float_as_uint(va) : 0u, vb < INFINITY ? __float_as_uint(vb) : 0u)));
        const bool whole_tile = k0 >= all_lo && k0 + kKeys <= all_hi;  // every row sees every key
        // a hidden value's scale that is not finite would reach this row through its weight of 0
        const bool bad = !whole_tile && __any_sync(0xffffffffu, !(va < INFINITY && vb < INFINITY));
        tmem_ld_wait();
        float2* z = reinterpret_cast<float2*>(s);
        const float2 rf2 = make_float2(rf, rf);
        const float4* ks4 = reinterpret_cast<const float4*>(ks);
        const float4* vs4 = reinterpret_cast<const float4*>(vs);
        // scores in log2 units
#pragma unroll
        for (int x = 0; x < 16; ++x) {
          const float4 k4 = ks4[x];
          z[2 * x] = mul2(z[2 * x], mul2(make_float2(k4.x, k4.y), rf2));
          z[2 * x + 1] = mul2(z[2 * x + 1], mul2(make_float2(k4.z, k4.w), rf2));
        }
        uint32_t see[2] = {0xffffffffu, 0xffffffffu};  // the tile's keys that this row sees
        if (!whole_tile) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int b = k0 + 32 * h;
            see[h] = (bits_of(lo - b, hi - b) | bits_of(-b, sink - b)) & bits_of(key_lo - b, key_end - b);
#pragma unroll
            for (int x = 0; x < 16; ++x) {
              float2& y = z[16 * h + x];
              y.x = see[h] >> (2 * x) & 1u ? y.x : -INFINITY;
              y.y = see[h] >> (2 * x + 1) & 1u ? y.y : -INFINITY;
            }
          }
        }
        float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int x = 0; x < 32; ++x) top[x & 3] = max3(top[x & 3], z[x].x, z[x].y);
        const float zmax = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
        const bool none = m == -INFINITY;
        const bool move = none ? zmax > -INFINITY : zmax - m > 64.f || ex2f(zmax - m) * (f * vmax) > 32768.f;
        if (__any_sync(0xffffffffu, move)) {
          const float mn = fmaxf(m, zmax);
          const bool has = mn > -INFINITY;
          const float ref = has ? mn : 0.f;
          float tm = 0.f;
#pragma unroll
          for (int x = 0; x < 16; ++x) {  // (a hidden key: 0, or a NaN that the maximum passes over)
            const float4 v4 = vs4[x];
            tm = max3(tm, ex2f(z[2 * x].x - ref) * fabsf(v4.x), ex2f(z[2 * x].y - ref) * fabsf(v4.y));
            tm = max3(tm, ex2f(z[2 * x + 1].x - ref) * fabsf(v4.z), ex2f(z[2 * x + 1].y - ref) * fabsf(v4.w));
          }
          const float dm = none || !has ? 0.f : mn - m;
          const float want = tm > 0.f ? 8.f - log2f(tm) : 0.f;
          // this tile's weights are brought within 2^8; those before it keep their factor unless it has to fall
          const float keep = none ? want : log2f(f) + dm;
          const bool fall = !none && tm > 0.f && exp2f(fminf(keep, 126.f)) * tm > 32768.f;
          const float to = fminf(fmaxf(fall ? want : keep, -120.f), 120.f);
          const float os = none ? 1.f : exp2f(to - keep);
          if (has) {
            l *= ex2f(-dm);
            m = mn;
            f = exp2f(to);
          }
          if (i > 0 && __any_sync(0xffffffffu, has && os != 1.f)) {
            const float by = has ? os : 1.f;
#pragma unroll 1
            for (int c = 0; c < HD; c += 16) {
              uint32_t o[16];
              tmem_ld16u(tO + lanes + c, o);
              tmem_ld_wait();
#pragma unroll
              for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * by);
              tmem_st16(tO + lanes + c, o);
            }
            tmem_st_wait();
          }
        }
        const float off = m == -INFINITY ? 0.f : -m;
        const float2 off2 = make_float2(off, off), f2 = make_float2(f, f);
        float2 sum = make_float2(0.f, 0.f);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t p[16];
#pragma unroll
          for (int y = 0; y < 8; ++y) {
            const int x = 8 * h + y;
            const float4 v4 = vs4[x];
            const float2 va2 = mul2(make_float2(v4.x, v4.y), f2), vb2 = mul2(make_float2(v4.z, v4.w), f2);
            float2 a = add2(z[2 * x], off2), b = add2(z[2 * x + 1], off2);
            a = make_float2(ex2f(a.x), ex2f(a.y));
            b = make_float2(ex2f(b.x), ex2f(b.y));
            sum = add2(sum, add2(a, b));
            a = mul2(a, va2);
            b = mul2(b, vb2);
            p[2 * y] = half2_of(a.x, a.y);
            p[2 * y + 1] = half2_of(b.x, b.y);
          }
          if (bad) {
#pragma unroll
            for (int y = 0; y < 16; ++y)
              p[y] &= (see[h] >> (2 * y) & 1u ? 0xffffu : 0u) | (see[h] >> (2 * y + 1) & 1u ? 0xffff0000u : 0u);
          }
          tmem_st16(tP + 16 * h + lanes, p);
        }
        l += sum.x + sum.y;
        tmem_st_wait();
      }
      fence_proxy_async_smem();
      tc_fence_before();
      if (__syncthreads_or(!ok)) {
        ok = false;
        break;
      }
      if (warp == 0) {
        if (elect_one()) {
          tc_fence_after();
          const uint32_t vt = smem_u32(sm + L::kV + (i & 1) * L::kTile);
#pragma unroll
          for (int k = 0; k < kKeys / 16; ++k)
            tc_mma_f16_tmem_a(tO, tP + 8 * k, smem_desc_mn(vt + k * 2048, kKeys * 128), idO, (i | k) != 0);
          tc_commit(&pv_done);
        }
        __syncwarp();
      } else if (warp == 1 && i + 1 < sg.nt) {  // (by another warp: a product takes 30 to 60 cycles to ask for)
        if (elect_one()) {
          tc_fence_after();
          scores((i + 1) & 1);
        }
        __syncwarp();
      }
      ++pv_n;
      if (i + 1 < sg.nt) ++s_n;
    }
    if (!ok) break;
    // ------------------------------------------------------------ the rows' results
    ok = over(&pv_done, (pv_n - 1) & 1u, g.wait_ns);
    if (__syncthreads_or(!ok)) {
      ok = false;
      break;
    }
    tc_fence_after();
    const bool whole = walk.whole(sg);
    if (!idle) {
      const float inv = whole ? 1.f / (f * l) : 1.f / f;
      bf16* dst = out + (((long long)mine.b * g.n + mine.i) * g.nq + mine.head) * HD;
      float* pdst = g.part_o + (sg.slot_row + tid) * HD;
#pragma unroll 1
      for (int c = 0; c < HD; c += 16) {
        uint32_t o[16];
        tmem_ld16u(tO + lanes + c, o);
        tmem_ld_wait();
        float x[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) x[e] = __uint_as_float(o[e]) * inv;
        if (mine.live) {
          if (whole) {
#pragma unroll
            for (int e = 0; e < 16; e += 8) {
              uint4 v;
              __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&v);
#pragma unroll
              for (int y = 0; y < 4; ++y) h[y] = __floats2bfloat162_rn(x[e + 2 * y], x[e + 2 * y + 1]);
              *reinterpret_cast<uint4*>(dst + c + e) = v;
            }
          } else {
#pragma unroll
            for (int e = 0; e < 16; e += 4)
              *reinterpret_cast<float4*>(pdst + c + e) = make_float4(x[e], x[e + 1], x[e + 2], x[e + 3]);
          }
        }
      }
      if (mine.live && !whole) g.part_ml[sg.slot_row + tid] = make_float2(m, l);
    }
    tc_fence_before();
    __syncthreads();
  }
  if (!ok) {
    // (some thread's wait ran out: all of them are here) products in flight end before their operands go away
    if (tid == 0) {
      set_status(g.status, DFLASH_STATUS_TIMEOUT);
      if (s_n > 0) mbar_wait(&s_done, (s_n - 1) & 1u, kDrainNs);
      if (pv_n > 0) mbar_wait(&pv_done, (pv_n - 1) & 1u, kDrainNs);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, 256);
  }
}

PagedRule paged_rule_q8_tc() { return PagedRule{kRows, kRows, kKeys, 1, 2}; }

template <int HD>
static cudaError_t q8_tc_launch(PagedGeom g, const void* q, const void* kp, const void* vp, void* out,
                                long long part_rows, cudaStream_t s) {
  typedef Q8TcLayout<HD> L;
  static_assert(2 * L::kSmem <= 232448 - 2048, "two CTAs a multiprocessor");
  static PerDevice smem;
  DFL_RET(smem.once([] {
    return cudaFuncSetAttribute(paged_attn_q8_tc_kernel<HD>, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kSmem);
  }));
  if (paged_split(g, paged_rule_q8_tc(), num_sms() * 2, 2) > part_rows) return cudaErrorInvalidValue;
  const float scale_log2 = 1.4426950408889634f / sqrtf((float)HD);
  DFL_RET(launch_pdl(paged_attn_q8_tc_kernel<HD>, dim3(g.grid), dim3(kThreads), L::kSmem, s, g, (const bf16*)q,
                     (const uint8_t*)kp, (const uint8_t*)vp, (bf16*)out, scale_log2));
  count_launch();
  return g.shared ? paged_merge_q8(HD, g, out, s) : paged_join_bf16(HD, g, out, s);
}

cudaError_t paged_attention_q8_tc(int hd, const PagedGeom& g, const void* q, const void* kp, const void* vp, void* out,
                                  long long part_rows, cudaStream_t s) {
  return hd == 64 ? q8_tc_launch<64>(g, q, kp, vp, out, part_rows, s)
                  : q8_tc_launch<128>(g, q, kp, vp, out, part_rows, s);
}

}  // namespace dfl
