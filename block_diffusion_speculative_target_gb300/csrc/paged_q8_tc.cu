// Attention of many rows over 8-bit pages (bf16 queries) on the 5th-generation
// tensor cores.
//
//   z_j = scale ks_j sum_d q_d (u_jd - 128),  o = sum_j 2^(z_j - m) vs_j (v_jd - 128) / sum_j 2^(z_j - m)   (log2 units)
//
// The arithmetic is that of the kernel for few rows: codes less 128 are exact in
// half precision, queries are half, each row scaled by a power of two, ks
// multiplies the scores in float32, and a weight enters the product with the values
// as a pair of halves, 2^(z - m) vs f rounded and what that leaves (off by 2^-22 of
// itself, or by 2^-25), f a factor of the row that keeps its largest weight between
// 2^7 and 2^15.
//
// An item is up to 128 stacked rows.  A tile of 64 keys goes
//   pages -> codes in shared memory by bulk copies of 16 keys (one tile ahead; the
//            pages' numbers two ahead)
//         -> halves in shared memory, K once and V in two buffers, swizzled
//   S = Q K^T   128 rows by 64 keys in TMEM, two buffers
//   O += P V    P as two halves over the scores they come from, O in TMEM
// so a key's codes are expanded once for all rows.  Warps 0..3 take the exponentials,
// a row a thread; warps 4..7 fetch and expand the next tile meanwhile, and two of them
// issue the products.  Measured: 128 rows behind 36K keys, 40 / 8 heads, 244 us (400
// TFLOP/s, 20% of the products' floor); 8 blocks of 16 rows over 2K..6K keys, 32 / 8
// heads, 63 us; 15-row blocks in a window of 4096 58 us.  Bound by latency: 39% of the
// issue slots and 26% of the tensor pipe are taken, a tile takes a CTA about 2.9 us, and a
// CTA's exponentials (a chain of TMEM load, scales, maximum, weights, TMEM store) cannot
// begin before its scores nor end a tile before the next one's.  The weights' second
// halves cost 12% of the chunk (217 us without them).  Before them, one group of 128 threads for everything took 238 us,
// codes through registers instead of bulk copies 239, one buffer of scores 228.
// Two CTAs share an SM.  The split of a call over CTAs is that of
// paged.cuh; pieces of items are joined by a second kernel.
//
// Every wait is bounded (PagedGeom::wait_ns); one that gives up sets
// DFLASH_STATUS_TIMEOUT, the CTA stops, drains its products, whatever the limit, and
// ends.  No wait can be lapped by a whole phase: what completes a barrier's next phase
// needs every warp that waits for this one (named at the barriers).
#include <math.h>

#include <algorithm>

#include "common.cuh"
#include "internal.h"
#include "paged.cuh"

namespace dfl {

namespace {
constexpr int kThreads = 256;
constexpr int kGroup = 128;  // threads of the exponentials, and of the expansion
constexpr int kKeys = kPagedQ8Keys;
constexpr int kRows = 128;
constexpr float kFactorLog2 = 120.f;  // a row's factor lies within 2^-120 and 2^120
constexpr uint64_t kDrainNs = 125000000ull;

template <int HD>
struct Q8TcLayout {
  static constexpr int kHalves = HD / 64;              // 64 dimensions: rows of 128 bytes
  static constexpr int kTile = kHalves * kKeys * 128;  // 64 keys or values
  static constexpr int kQ = 0;
  static constexpr int kK = kHalves * kRows * 128;
  static constexpr int kV = kK + kTile;                // [2]
  static constexpr int kCodes = kV + 2 * kTile;        // [K, V][64][HD] as in the pages
  static constexpr int kCodeScales = kCodes + 2 * kKeys * HD;   // [ks, vs][64]
  static constexpr int kScales = kCodeScales + 2 * kKeys * 4;   // [2][ks, vs][64]
  static constexpr int kSpan = kScales + 2 * 2 * kKeys * 4;  // [rows] sink, lo, hi, 2^-up of the queries' factor
  static constexpr int kRed = kSpan + kRows * 16;
  static constexpr int kUsed = kRed + (2 * kThreads / 32 + 8) * 4;
  static constexpr int kSmem = kUsed + 1024;
};

// What both halves of the CTA need to know of a piece.
struct Q8Piece {
  int nt, prefix, b, rt, hk, whole;
  int s0, sn, w0, t0;                 // tile t is t0 + t of the item's: s0 + t below sn, then w0 + t - sn
  int key_lo, key_end;
  int seen_sink, seen_lo;             // some row sees the keys below the one, and those from the other on
  long long slot_row;
  __device__ __forceinline__ int tile(int t) const {
    t += t0;
    return t < sn ? s0 + t : w0 + t - sn;
  }
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
// What rounding a pair of weights to the halves `hi` leaves.
__device__ __forceinline__ uint32_t rest_of(float2 w, uint32_t hi) {
  const float2 h = __half22float2(*reinterpret_cast<const __half2*>(&hi));
  const float2 d = add2(w, make_float2(-h.x, -h.y));
  return half2_of(d.x, d.y);
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
}  // namespace

template <int HD>
__global__ void __launch_bounds__(kThreads, 2)
    paged_attn_q8_tc_kernel(const __grid_constant__ PagedGeom g, const bf16* __restrict__ q,
                            const uint8_t* __restrict__ kp, const uint8_t* __restrict__ vp, bf16* __restrict__ out,
                            float scale_log2) {
  typedef Q8TcLayout<HD> L;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  // kv_full: a tile's keys and values are expanded (4 warps, which have waited for the last scores and for the pv_done
  // of two tiles before).  s_done: its scores are there, in buffer T % 2; the next ones of a buffer are asked for after
  // the kv_full of two tiles on, so after all have waited for these.  p_full: its weights are there (4 warps, which
  // have waited for the last pv_done).  pv_done: their product with the values is done; it is asked for after p_full
  // and the next tile's kv_full, whose warps have waited for the one before it.
  // codes_full: a tile's codes are there.  codes_free: and have been read (4 warps; so all have waited for codes_full).
  __shared__ __align__(8) uint64_t kv_full, s_done[2], p_full, pv_done, codes_full, codes_free, drain[2];
  __shared__ uint32_t tmem_slot;
  __shared__ volatile int abort_s;
  __shared__ Q8Piece pc;
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  float* scales = reinterpret_cast<float*>(sm + L::kScales);
  int4* spans = reinterpret_cast<int4*>(sm + L::kSpan);
  if (tid == 0) {
    mbar_init(&kv_full, 4);
    mbar_init(&s_done[0], 1);
    mbar_init(&s_done[1], 1);
    mbar_init(&p_full, 4);
    mbar_init(&pv_done, 1);
    mbar_init(&codes_full, 1);
    mbar_init(&codes_free, 4);
    mbar_init(&drain[0], 1);
    mbar_init(&drain[1], 1);
    abort_s = 0;
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
  const uint32_t tmem = tmem_slot, tO = tmem, tS = tmem + 128;  // scores of tile T (and its weights): 64 T % 2 further
  pdl_launch();
  pdl_wait();
  const PlanView pv = plan_view<kKeys, kThreads>(g, reinterpret_cast<int*>(sm + L::kRed));
  // Waits for phase `n` of a barrier, giving up on the CTA's abort flag or after the limit (then raising the flag).
  // A warp's lanes wait together and agree.
  auto wait = [&](uint64_t* bar, int n) {
    const uint32_t parity = (uint32_t)n & 1u;
    if (g.wait_ns != 0 && __all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
    bool ok = false;
    if (g.wait_ns != 0) {
      const uint32_t t0 = global_ns_lo();
      while (true) {
#pragma unroll 1
        for (int i = 0; i < 64 && !ok; ++i) ok = mbar_try_wait(bar, parity);
        if (ok || abort_s || global_ns_lo() - t0 > g.wait_ns) break;
      }
    }
    if (__any_sync(0xffffffffu, !ok)) {
      if (lane == 0) {
        if (!abort_s) set_status(g.status, DFLASH_STATUS_TIMEOUT);
        abort_s = 1;
      }
      return false;
    }
    return true;
  };
  auto arrive = [&](uint64_t* bar) {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar);
  };
  // All threads of the CTA, from either group's code.
  auto cta_sync = [&] {
    __syncwarp();
    asm volatile("barrier.cta.sync 0, %0;" ::"n"(kThreads) : "memory");
  };
  // The piece's queries: half, each row by a power of two.
  auto load_queries = [&] {
    const int x0 = pc.rt * (pc.prefix ? g.rp : g.ri);
    constexpr int kLanes = HD / 16;  // a lane takes 16 entries of a row
    const int c = tid % kLanes;
#pragma unroll 2
    for (int r = tid / kLanes; r < kRows; r += kThreads / kLanes) {
      const ItemRow row = item_row(g, pc.prefix, pc.b, pc.hk, x0, r);
      uint4 raw[2] = {make_uint4(0u, 0u, 0u, 0u), make_uint4(0u, 0u, 0u, 0u)};
      int4 span = make_int4(0, 0, INT32_MAX, 0);
      if (row.live) {
        const uint4* src =
            reinterpret_cast<const uint4*>(q + (((long long)row.b * g.n + row.i) * g.nq + row.head) * HD + 16 * c);
        raw[0] = src[0];
        raw[1] = src[1];
        if (c == 0) row_span(g, paged_len(g, row.b), paged_rows(g, row.b), row.i, span.x, span.y, span.z);
      }
      const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(raw);
      float most = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float2 f = __bfloat1622float2(h[e]);
        most = fmaxf(most, fmaxf(fabsf(f.x), fabsf(f.y)));
      }
#pragma unroll
      for (int o = 1; o < kLanes; o <<= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
      // 2^up brings the largest entry to 2^7..2^8 (a row of zeros, or one that holds Inf: as it is)
      const int ex = (int)(__float_as_uint(most) >> 23);
      const int up = ex > 0 && ex < 255 ? 134 - ex : ex == 0 && most > 0.f ? 133 : 0;
      const float u1 = exp2f((float)(up / 2)), u2 = exp2f((float)(up - up / 2));
      uint32_t w[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float2 f = __bfloat1622float2(h[e]);
        w[e] = half2_of(f.x * u1 * u2, f.y * u1 * u2);
      }
      uint8_t* dst = sm + L::kQ + (c >> 2) * (kRows * 128) + r * 128;
#pragma unroll
      for (int e = 0; e < 2; ++e)
        *reinterpret_cast<uint4*>(dst + (((2 * (c & 3) + e) ^ (r & 7)) << 4)) =
            make_uint4(w[4 * e], w[4 * e + 1], w[4 * e + 2], w[4 * e + 3]);
      if (c == 0) {
        span.w = __float_as_int(exp2f((float)-up));
        spans[r] = span;
      }
    }
    fence_proxy_async_smem();
  };
  int done = 0;  // tiles of the pieces before
  if (warp >= 4) {
    // ------------------------------------------------------------ keys and values, and the products
    asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
    int asked = 0;  // tiles that warp 6 has asked for
    while (true) {
      cta_sync();
      const int nt = pc.nt;
      if (nt == 0) break;
      load_queries();
      cta_sync();
      // A thread takes 16 bytes of every kStep-th key row: whole rows by neighbours.  Every 16 keys lie in one page.
      constexpr int kLanes = HD / 16, kStep = kGroup / kLanes, KU = kKeys / kStep;
      const int et = tid - kGroup, kr = et / kLanes, kc16 = et % kLanes;
      const int hk = pc.hk, key_end = pc.key_end, seen_sink = pc.seen_sink, seen_lo = pc.seen_lo;
      const int32_t* trow = g.table + (long long)pc.b * g.table_stride;
      // The page of the 16 keys 16 (lane % 4) .. of tile i (the pool's first where no row sees one of them): asked for a
      // tile before it is looked at.
      auto key_of = [&](int i) { return pc.tile(i) * kKeys + 16 * (lane & 3); };
      auto page_of = [&](int i) {
        if (i >= nt) return 0;
        const int key = key_of(i);
        return key >= key_end || (key >= seen_sink && key + 16 <= seen_lo) ? 0 : trow[key >> g.ps_log2];
      };
      // Tile i's codes: a lane of warp 6 brings 16 keys, their values and the scales of both.
      // (Of a bad page: the pool's first rows; the sequence's result is unspecified.)
      auto fetch = [&](int i, int page) {
        asked = done + i + 1;
        if (lane == 0) mbar_arrive_expect_tx(&codes_full, 2 * kKeys * (HD + 4));
        __syncwarp();
        if (lane < 4) {
          long long first = 0;  // the pool row of the 16 keys
          if ((unsigned)page < (unsigned)g.n_pages)
            first = g.page_row0 + ((long long)page * g.nkv + hk) * g.ps + (key_of(i) & (g.ps - 1));
          else
            set_status(g.status, DFLASH_STATUS_BOUNDS);
          uint8_t* codes = sm + L::kCodes + lane * 16 * HD;
          uint8_t* cs = sm + L::kCodeScales + lane * 64;
          bulk_load(codes, kp + first * HD, 16 * HD, &codes_full);
          bulk_load(codes + kKeys * HD, vp + first * HD, 16 * HD, &codes_full);
          bulk_load(cs, g.ks + first, 64, &codes_full);
          bulk_load(cs + kKeys * 4, g.vs + first, 64, &codes_full);
        }
        __syncwarp();
      };
      // 16 codes are two chunks of 16 bytes; lanes of the upper half of a row write theirs the other way round, so
      // that the 8 lanes of a row fill all banks
      const int c = 2 * (kc16 & 3), far = kc16 >> 2;
      auto expand = [&](const uint4 (&codes)[KU], uint8_t* dst) {
#pragma unroll
        for (int u = 0; u < KU; ++u) {
          const int key = kr + kStep * u;
          uint8_t* base = dst + far * (kKeys * 128) + key * 128;
          const uint4 w = codes[u];
          uint4 h[2];
          halves_of(far ? make_uint4(w.z, w.w, w.x, w.y) : w, h);
          *reinterpret_cast<uint4*>(base + (((c + far) ^ (key & 7)) << 4)) = h[0];
          *reinterpret_cast<uint4*>(base + (((c + 1 - far) ^ (key & 7)) << 4)) = h[1];
        }
      };
      constexpr uint32_t idS = idesc_f16_f32(128, kKeys), idO = idesc_f16_f32(128, HD) | (1u << 16);  // values MN-major
      int next_page = 0;
      if (warp == 6) {
        fetch(0, page_of(0));
        next_page = page_of(1);
      }
      for (int i = 0; i <= nt; ++i) {
        const int T = done + i;  // tile i's number
        if (i < nt) {
          if (!wait(&codes_full, T)) break;
          const uint4* raw = reinterpret_cast<const uint4*>(sm + L::kCodes) + et;
          uint4 kc[KU], vc[KU];
#pragma unroll
          for (int u = 0; u < KU; ++u) {
            kc[u] = raw[kGroup * u];
            vc[u] = raw[kGroup * u + kKeys * HD / 16];
          }
          const float sc = reinterpret_cast<const float*>(sm + L::kCodeScales)[et];
          arrive(&codes_free);
          if (warp == 6 && i + 1 < nt) {
            if (!wait(&codes_free, T)) break;
            fetch(i + 1, next_page);
            next_page = page_of(i + 2);
          }
          // the last scores have been computed; the buffer's last values and scales have been read (the piece before has
          // ended)
          if (i >= 1 && !wait(&s_done[(T - 1) & 1], (T - 1) >> 1)) break;
          expand(kc, sm + L::kK);
          if (i >= 2 && !wait(&pv_done, T - 2)) break;
          expand(vc, sm + L::kV + (T & 1) * L::kTile);
          scales[2 * (T & 1) * kKeys + et] = et < kKeys ? sc * scale_log2 : sc;
          fence_proxy_async_smem();
          arrive(&kv_full);
        }
        if (warp == 4 && i < nt) {
          if (!wait(&kv_full, T)) break;
          tc_fence_after();
          if (elect_one()) {
            const uint64_t dq = smem_desc_sw128(sm + L::kQ), dk = smem_desc_sw128(sm + L::kK);
#pragma unroll
            for (int k = 0; k < HD / 16; ++k)
              tc_mma_f16(tS + 64 * (T & 1), dq + (uint64_t)((k >> 2) * (kRows * 128 / 16) + 2 * (k & 3)),
                         dk + (uint64_t)((k >> 2) * (kKeys * 128 / 16) + 2 * (k & 3)), idS, k > 0);
            tc_commit(&s_done[T & 1]);
          }
          __syncwarp();
        }
        if (warp == 5 && i > 0) {  // (of the tile before)
          if ((i < nt && !wait(&kv_full, T)) || !wait(&p_full, T - 1)) break;
          tc_fence_after();
          if (elect_one()) {
            const uint32_t vt = smem_u32(sm + L::kV + ((T - 1) & 1) * L::kTile);
#pragma unroll
            for (int k = 0; k < 2 * (kKeys / 16); ++k)  // the weights' first halves, then their second ones
              tc_mma_f16_tmem_a(tO, tS + 64 * ((T - 1) & 1) + 8 * k,
                                smem_desc_mn(vt + k % (kKeys / 16) * 2048, kKeys * 128), idO, i > 1 || k > 0);
            tc_commit(&pv_done);
          }
          __syncwarp();
        }
      }
      cta_sync();
      if (abort_s) break;
      done += nt;
    }
    if (abort_s && warp < 6) {
      // products in flight end before their operands go away
      if (elect_one()) tc_commit(&drain[warp - 4]);
      __syncwarp();
      mbar_wait(&drain[warp - 4], 0, kDrainNs);
    }
    // so do copies
    if (abort_s && warp == 6 && asked > 0) mbar_wait(&codes_full, (uint32_t)(asked - 1) & 1u, kDrainNs);
  } else {
    // ------------------------------------------------------------ exponentials
    asm volatile("setmaxnreg.inc.sync.aligned.u32 176;");
    SegmentWalk<kKeys> walk(g, pv);
    walk.start();
    bool first = true;
    while (true) {
      if (warp == 0) {
        Segment sg;
        const bool more = walk.next(sg);
        if (first && !g.shared) {
          // the item that this CTA's run begins inside of, when it is the second to hold a piece of it
          int c0 = 0, nc = 0;
          if (more && sg.t0 > 0) nc = walk.pieces(sg, c0);
          if (c0 + 1 != (int)blockIdx.x) nc = 0;
          int4* rec = reinterpret_cast<int4*>(g.records) + 2 * blockIdx.x;
          if (lane == 0) {
            rec[0] = make_int4(nc, sg.b, sg.rt, sg.hk);
            rec[1].x = c0;
          }
        }
        if (lane == 0) {
          pc.nt = more ? sg.nt : 0;
          if (more) {
            pc.prefix = sg.prefix;
            pc.b = sg.b;
            pc.rt = sg.rt;
            pc.hk = sg.hk;
            pc.whole = walk.whole(sg);
            pc.s0 = sg.span.s0;
            pc.sn = sg.span.s1 - sg.span.s0;
            pc.w0 = sg.span.w0;
            pc.t0 = sg.t0;
            pc.key_lo = sg.prefix ? 0 : pv.sh_tiles * kKeys;
            pc.key_end = sg.prefix ? pv.sh_tiles * kKeys : key_limit(g, sg.b);
            int hi;
            row_span(g, sg.prefix ? pv.min_len : paged_len(g, sg.b), paged_rows(g, sg.b),
                     sg.prefix ? 0 : div_g(g, sg.rt * g.ri), pc.seen_sink, pc.seen_lo, hi);
            pc.slot_row = sg.slot_row;
          }
        }
      }
      first = false;
      cta_sync();
      const int nt = pc.nt;
      if (nt == 0) break;
      load_queries();
      cta_sync();
      const uint32_t lanes = (uint32_t)(32 * warp) << 16;
      const int4 span = spans[tid];
      const int sink = span.x, lo = span.y, hi = span.z, key_lo = pc.key_lo, key_end = pc.key_end;
      const float rf = __int_as_float(span.w);
      const int all_lo = __reduce_max_sync(0xffffffffu, max(key_lo, lo));
      const int all_hi = __reduce_min_sync(0xffffffffu, min(key_end, hi));
      const ItemRow mine = item_row(g, pc.prefix, pc.b, pc.hk, pc.rt * (pc.prefix ? g.rp : g.ri), tid);
      const bool idle = __all_sync(0xffffffffu, !mine.live);  // none of the warp's rows is one
      float m = -INFINITY, l = 0.f, f = 1.f;
      bool ok = true;
      for (int i = 0; i < nt; ++i) {
        const int T = done + i;
        if (!(ok = wait(&s_done[T & 1], T >> 1))) break;
        tc_fence_after();
        if (idle) {  // (in step with the others: an arrival must not count for the phase before)
          if (i > 0 && !(ok = wait(&pv_done, T - 1))) break;
          arrive(&p_full);
          continue;
        }
        const float* ks = scales + 2 * (T & 1) * kKeys;
        const float* vs = ks + kKeys;
        const int k0 = pc.tile(i) * kKeys;
        uint32_t s[2][32];
        const uint32_t ts = tS + 64 * (T & 1) + lanes;
        tmem_ld32(ts, s[0]);
        tmem_ld32(ts + 32, s[1]);
        // the largest scale of the tile's values (of hidden slots too: it only says when to look closer)
        const float va = fabsf(vs[lane]), vb = fabsf(vs[lane + 32]);
        const float vmax = __uint_as_float(__reduce_max_sync(
            0xffffffffu, max(va < INFINITY ? __float_as_uint(va) : 0u, vb < INFINITY ? __float_as_uint(vb) : 0u)));
        const bool whole_tile = k0 >= all_lo && k0 + kKeys <= all_hi;  // every row sees every key
        // a hidden value's scale that is not finite would reach this row through its weight of 0
        const bool bad = __any_sync(0xffffffffu, !(va < INFINITY && vb < INFINITY));
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
        const bool move = none ? zmax > -INFINITY : zmax - m > 64.f || ex2f(zmax - m) * vmax * f > 32768.f;
        // the last weights have been multiplied: the outputs' sums may be moved
        if (i > 0 && !(ok = wait(&pv_done, T - 1))) break;
        tc_fence_after();
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
          // this tile's weights are brought within 2^8 (values of zero leave the factor at its most, so that the next
          // ones set it); those before it keep their factor unless it has to fall
          const float want = tm > 0.f ? 8.f - log2f(tm) : kFactorLog2, was = log2f(f);
          const float keep = none ? want : was + dm;
          const bool fall = !none && tm > 0.f && exp2f(fminf(keep, 126.f)) * tm > 32768.f;
          const float to = fminf(fmaxf(fall ? want : keep, -kFactorLog2), kFactorLog2);
          const float os = none ? 1.f : exp2f(to - keep);
          if (has) {
            l *= ex2f(-dm);
            m = mn;
            if (to != was) f = exp2f(to);
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
          uint32_t p[16], rest[16];
#pragma unroll
          for (int y = 0; y < 8; ++y) {
            const int x = 8 * h + y;
            const float4 v4 = vs4[x];
            float2 a = add2(z[2 * x], off2), b = add2(z[2 * x + 1], off2);
            a = make_float2(ex2f(a.x), ex2f(a.y));
            b = make_float2(ex2f(b.x), ex2f(b.y));
            sum = add2(sum, add2(a, b));
            // (the scale first: a hidden key's weight of 0 stays 0 whatever finite scale its slot holds, where the scale
            // times the factor may be past float32)
            a = mul2(mul2(a, make_float2(v4.x, v4.y)), f2);
            b = mul2(mul2(b, make_float2(v4.z, v4.w)), f2);
            p[2 * y] = half2_of(a.x, a.y);
            p[2 * y + 1] = half2_of(b.x, b.y);
            rest[2 * y] = rest_of(a, p[2 * y]);
            rest[2 * y + 1] = rest_of(b, p[2 * y + 1]);
          }
          if (bad) {
#pragma unroll
            for (int y = 0; y < 16; ++y) {
              const uint32_t on = (see[h] >> (2 * y) & 1u ? 0xffffu : 0u) | (see[h] >> (2 * y + 1) & 1u ? 0xffff0000u : 0u);
              // (an infinite weight leaves nothing)
              const uint32_t fine = ((p[y] & 0x7c00u) != 0x7c00u ? 0xffffu : 0u) |
                                    ((p[y] & 0x7c000000u) != 0x7c000000u ? 0xffff0000u : 0u);
              p[y] &= on;
              rest[y] &= on & fine;
            }
          }
          tmem_st16(ts + 16 * h, p);
          tmem_st16(ts + 32 + 16 * h, rest);
        }
        l += sum.x + sum.y;
        tmem_st_wait();
        tc_fence_before();
        arrive(&p_full);
      }
      // ---------------------------------------------------------- the rows' results
      if (ok) ok = wait(&pv_done, done + nt - 1);
      tc_fence_after();
      if (ok && !idle) {
        const bool whole = pc.whole;
        // (two quotients: a factor for tiny values times the sum may be past float32)
        const float back = 1.f / f, inv = 1.f / l;
        bf16* dst = out + (((long long)mine.b * g.n + mine.i) * g.nq + mine.head) * HD;
        float* pdst = g.part_o + (pc.slot_row + tid) * HD;
#pragma unroll 1
        for (int c = 0; c < HD; c += 32) {
          uint32_t o[32];
          tmem_ld32(tO + lanes + c, o);
          tmem_ld_wait();
          if (mine.live) {
            if (whole) {
#pragma unroll
              for (int e = 0; e < 32; e += 8) {
                uint4 v;
                __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&v);
#pragma unroll
                for (int y = 0; y < 4; ++y)
                  h[y] = __floats2bfloat162_rn(__uint_as_float(o[e + 2 * y]) * back * inv,
                                               __uint_as_float(o[e + 2 * y + 1]) * back * inv);
                *reinterpret_cast<uint4*>(dst + c + e) = v;
              }
            } else {
#pragma unroll
              for (int e = 0; e < 32; e += 4)
                *reinterpret_cast<float4*>(pdst + c + e) =
                    make_float4(__uint_as_float(o[e]) * back, __uint_as_float(o[e + 1]) * back,
                                __uint_as_float(o[e + 2]) * back, __uint_as_float(o[e + 3]) * back);
            }
          }
        }
        if (mine.live && !whole) g.part_ml[pc.slot_row + tid] = make_float2(m, l);
      }
      tc_fence_before();
      cta_sync();
      if (abort_s) break;
      done += nt;
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, 256);
  }
}

// (An item's start and end weigh as three tiles in the split: as two, the chunk takes 218 us instead of 215; as six 213, but
// 8 blocks of 16 rows 60 instead of 58.)
PagedRule paged_rule_q8_tc() { return PagedRule{kRows, kRows, kKeys, 1, 3}; }

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
