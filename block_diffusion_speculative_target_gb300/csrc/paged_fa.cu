// Attention over pages on the 5th-generation tensor cores (bf16, head_dim 64
// or 128): one persistent CTA a SM walks its run of key tiles (paged.cuh).
//
// Two groups of four softmax warps work independently, each with a score
// buffer S and an output accumulator O in TMEM and a warp that issues its
// products, so one group's exponentials run under the other's products:
//   S = Q K_t^T            128 stacked rows by 128 keys, fp32 in TMEM
//   reference max M: the row's first tile sets it, a later tile raises it only
//     when its own max exceeds M by more than 8 (log2 units); then O and the
//     row sum L are rescaled by 2^(M_old - M_new)
//   P = 2^(s - M)          <= 2^8, written over S as bf16
//   O += P V_t             A operand from TMEM, fp32 in TMEM
// An item of at most 128 stacked rows (few rows against many keys) has one
// query tile; the groups take its key tiles in turn and their (M, L, O) are
// joined at the end.  There P is kept as a bf16 pair hi + lo (about 2^-17
// relative) and multiplied in two passes: such items wait for keys, not for
// products.  An item of more rows has two query tiles, one a group, that share
// every key tile, which halves the traffic from L2; there the products bound,
// and P is rounded to bf16 once (2^-9 relative a weight, the size of the
// result's own rounding).
//
// Warps: 0 streams the pages (TMA, one box a page and 64 dimensions) through a
// ring of key and value tiles; 1 and 2 issue the groups' products; 3 owns TMEM
// and brings the query rows (16-byte asynchronous copies, swizzled by hand:
// stacked rows of any GQA group are packed without gaps); 4..7 and 8..11 are
// the softmax groups, a thread a row.
//
// A hidden key's weight is 0, and 0 times an Inf or NaN value would reach rows
// that do not see it.  So in a tile that some row sees only in part, the group
// looks through the values first; a value that is not finite is taken out of
// the tile and added with its weight to the accumulators of the rows that do
// see it.
//
// Every wait is bounded; one that gives up sets DFLASH_STATUS_TIMEOUT, the CTA
// stops, and drains its copies and products before it releases TMEM.
#include <math.h>

#include <algorithm>
#include <type_traits>

#include "common.cuh"
#include "internal.h"
#include "paged.cuh"

namespace dfl {

namespace {
constexpr int kTcThreads = 384;
constexpr uint64_t kTcWaitNs = 500000000ull;

template <int HD>
struct TcLayout {
  static constexpr int kHalves = HD / 64;               // 64-dimension halves: 128-byte rows
  static constexpr uint32_t kTile = kHalves * 16384;    // 128 rows
  static constexpr int kSlots = HD == 128 ? 5 : 8;
  static constexpr uint32_t kQ = 0;                     // two query tiles
  static constexpr uint32_t kRing = 2 * kTile;
  static constexpr uint32_t kXch = kRing + kSlots * kTile;  // [128] (M, L) of group 1
  static constexpr uint32_t kBar = kXch + 1024;
  static constexpr int kBars = 2 * kSlots + 21;
  static constexpr uint32_t kMisc = kBar + kBars * 8;   // TMEM slot, abort flag, per-group words, scan scratch
  static constexpr int kSmem = kMisc + 256 + 1024;      // + alignment slack
  static_assert(kSmem <= 232448, "shared memory per block");
  static_assert(kMisc % 8 == 0, "alignment");
};

__device__ __forceinline__ uint32_t tmem_ld1(uint32_t taddr) {
  uint32_t r;
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=r"(r) : "r"(taddr) : "memory");
  return r;
}
__device__ __forceinline__ void cp_async16(void* smem_dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(smem_dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void reg_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void reg_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}

// Waits for a phase, giving up on the CTA's abort flag or after the limit (then raising the flag).
__device__ __forceinline__ bool wait_phase(uint64_t* bar, uint32_t parity, volatile int* abort_f, int* status) {
#pragma unroll 1
  for (int i = 0; i < 64; ++i)
    if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = global_ns();
  while (true) {
#pragma unroll 1
    for (int i = 0; i < 64; ++i)
      if (mbar_try_wait(bar, parity)) return true;
    if (*abort_f) return false;
    if (global_ns() - t0 > kTcWaitNs) {
      *abort_f = 1;
      set_status(status, DFLASH_STATUS_TIMEOUT);
      return false;
    }
  }
}

__device__ __forceinline__ bool nonfinite2(uint32_t w) {  // either of two bf16
  return (w & 0x7f800000u) == 0x7f800000u || (w & 0x7f80u) == 0x7f80u;
}
// Bits [a, b) of a word, clamped to it.
__device__ __forceinline__ uint32_t bits_of(int a, int b) {
  a = max(a, 0);
  b = min(b, 32);
  if (a >= b) return 0u;
  const uint32_t below = b >= 32 ? 0xffffffffu : (1u << b) - 1u;
  return below & ~((1u << a) - 1u);
}
}  // namespace

template <int HD>
__global__ void __launch_bounds__(kTcThreads, 1)
    paged_attn_tc_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                         const __grid_constant__ PagedGeom g, int pool_rows, const bf16* __restrict__ q,
                         bf16* __restrict__ out, float scale_log2) {
  typedef TcLayout<HD> L;
  constexpr int KT = kPagedTcKeys, NS = L::kSlots;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bar = reinterpret_cast<uint64_t*>(sm + L::kBar);
  uint64_t* full = bar;              // [NS] a key or value tile has landed
  uint64_t* empty = bar + NS;        // [NS] both issuing warps are done with it
  uint64_t* q_full = bar + 2 * NS;   // [2]
  uint64_t* q_empty = q_full + 2;    // [2] two arrivals
  uint64_t* s_full = q_full + 4;     // [2] scores of the group's tile in TMEM
  uint64_t* p_full = q_full + 6;     // [2] its weights (four warps)
  uint64_t* pv_done = q_full + 8;    // [2] its product with the values is done
  uint64_t* o_free = q_full + 10;    // [2] the accumulator has been read (four warps)
  uint64_t* fix = q_full + 12;       // [3] value scan: group 0, group 1 (four warps), both (eight)
  uint64_t* x_full = q_full + 15;    // group 1's M and L are written (four warps)
  uint64_t* x_free = q_full + 16;    // and read
  uint64_t* drain = q_full + 17;     // [2] every product a warp issued is done
  uint64_t* v_ready = q_full + 19;   // [2] the values of the group's tile have landed
  uint32_t* misc = reinterpret_cast<uint32_t*>(sm + L::kMisc);
  uint32_t* tslot = misc;
  volatile int* abort_f = reinterpret_cast<volatile int*>(misc + 1);
  volatile uint32_t* acc_first = misc + 2;  // [2] the first product of an item adds to O instead of setting it
  volatile uint32_t* bad_w = misc + 4;      // [2][4] keys of the tile with a value that is not finite
  int* red = reinterpret_cast<int*>(misc + 12);
  float2* xch = reinterpret_cast<float2*>(sm + L::kXch);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
    for (int i = 0; i < NS; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 2);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&q_full[i], 1);
      mbar_init(&q_empty[i], 2);
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], 4);
      mbar_init(&pv_done[i], 1);
      mbar_init(&o_free[i], 4);
      mbar_init(&fix[i], 4);
      mbar_init(&drain[i], 1);
      mbar_init(&v_ready[i], 1);
    }
    mbar_init(&fix[2], 8);
    mbar_init(x_full, 4);
    mbar_init(x_free, 4);
    *abort_f = 0;
    fence_barrier_init();
  }
  if (warp == 3) {
    tmem_alloc(tslot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tslot;
  pdl_launch();
  pdl_wait();
  const PlanView pv = plan_view<KT, kTcThreads>(g, red);
  SegmentWalk<KT> walk(g, pv);
  Segment sg;
  // stacked rows of a piece's item, and whether it has two query tiles
  auto item_rows = [&](const Segment& s) {
    return s.prefix ? min(g.rp, g.batch * g.n * g.G - s.rt * g.rp) : min(g.ri, paged_rows(g, s.b) * g.G - s.rt * g.ri);
  };
  // query buffers: an item with one tile takes the buffer after the last one's, an item with two both
  int seg = 0, qt = 0, qn0 = 0, qn1 = 0;
  int tiles = 0;  // key tiles before the current piece
  auto stop = [&](bool ok) { return __any_sync(0xffffffffu, !ok); };

  if (warp < 4) {
    reg_dec<64>();
    if (warp == 0) {
      // ---------------------------------------------------------- pages
      const int per = KT >> g.ps_log2;  // pages a tile
      const bool mine = lane < per;
      int at = 0;  // tiles issued
      bool ok = true;
      while (ok && walk.next(sg)) {
        const int key_end = sg.prefix ? pv.sh_tiles * KT : key_limit(g, sg.b);
        const int32_t* trow = g.table + (long long)sg.b * g.table_stride;
        // pool row of this lane's page of tile t (past the keys or a bad page: past the pool, read as zeros)
        auto page_row = [&](int t) {
          if (!mine || t >= sg.t0 + sg.nt) return pool_rows;
          const int key = sg.span.tile(t) * KT + (lane << g.ps_log2);
          if (key >= key_end) return pool_rows;
          const int page = trow[key >> g.ps_log2];
          if ((unsigned)page >= (unsigned)g.n_pages) {
            set_status(g.status, DFLASH_STATUS_BOUNDS);
            return pool_rows;
          }
          return (int)(g.page_row0 + ((long long)page * g.nkv + sg.hk) * g.ps);
        };
        int row = page_row(sg.t0);
        for (int t = sg.t0; t < sg.t0 + sg.nt; ++t) {
          const int next_row = page_row(t + 1);
#pragma unroll
          for (int kv = 0; kv < 2; ++kv) {
            const int x = 2 * at + kv, s = x % NS;
            if (x >= NS && stop(wait_phase(&empty[s], (uint32_t)(x / NS - 1) & 1u, abort_f, g.status))) {
              ok = false;
              break;
            }
            uint8_t* dst = sm + L::kRing + s * L::kTile;
            if (lane == 0) mbar_arrive_expect_tx(&full[s], L::kTile);
            __syncwarp();
            if (mine) {
#pragma unroll
              for (int dh = 0; dh < L::kHalves; ++dh)
                tma_load_2d(dst + dh * 16384 + ((lane << g.ps_log2) << 7), kv == 0 ? &tmK : &tmV, &full[s], dh * 64, row);
            }
            tiles = x + 1;  // (slots filled)
          }
          if (!ok) break;
          row = next_row;
          ++at;
        }
      }
      // the last copies land before the CTA leaves, whatever became of their readers
      for (int x = max(0, tiles - NS); x < tiles; ++x) mbar_wait(&full[x % NS], (uint32_t)(x / NS) & 1u, kTcWaitNs / 4);
    } else if (warp < 3) {
      // ---------------------------------------------------------- products of group gq
      const int gq = warp - 1;
      if (lane == 0) {
        const uint32_t idS = idesc_bf16_f32(128, 128), idO = idesc_bf16_f32(128, HD) | (1u << 16);  // values MN-major
        const uint32_t tS = tmem + gq * 128, tO = tmem + 256 + gq * 128;
        int job = 0;
        bool ok = true;
        // Both issuing warps see every tile land and release it: a slot is refilled only after both have
        // been past it, so a wait never looks at a phase two fills away.
        while (ok && walk.next(sg)) {
          const bool two = item_rows(sg) > 128;
          const int buf = two ? gq : qt;
          if (two || qt == 0) ok = wait_phase(&q_full[0], (uint32_t)qn0 & 1u, abort_f, g.status);
          if (ok && (two || qt == 1)) ok = wait_phase(&q_full[1], (uint32_t)qn1 & 1u, abort_f, g.status);
          const int t0 = two ? 0 : gq, step = two ? 1 : 2;
          if (ok && t0 >= sg.nt) {  // no tile for this group
            if (seg > 0) ok = wait_phase(&o_free[gq], (uint32_t)(seg - 1) & 1u, abort_f, g.status);
            if (ok) mbar_arrive(&q_empty[buf]);
          }
          const uint8_t* qs = sm + L::kQ + buf * L::kTile;
          for (int t = 0; ok && t < sg.nt; ++t) {
            const int xk = 2 * (tiles + t), sk = xk % NS, sv = (xk + 1) % NS;
            const uint32_t pk = (uint32_t)(xk / NS) & 1u, pv_ = (uint32_t)((xk + 1) / NS) & 1u;
            ok = wait_phase(&full[sk], pk, abort_f, g.status);
            if (!ok) break;
            if (!two && (t & 1) != gq) {  // the other group's tile
              mbar_arrive(&empty[sk]);
              ok = wait_phase(&full[sv], pv_, abort_f, g.status);
              if (ok) mbar_arrive(&empty[sv]);
              continue;
            }
            // P of the last tile lies over S until its product is done
            if (job > 0) ok = wait_phase(&pv_done[gq], (uint32_t)(job - 1) & 1u, abort_f, g.status);
            if (!ok) break;
            tc_fence_after();
            const uint8_t* kt = sm + L::kRing + sk * L::kTile;
#pragma unroll
            for (int kk = 0; kk < HD / 16; ++kk) {
              const uint64_t off = (uint64_t)(((kk & 3) * 32) >> 4);
              tc_mma_f16(tS, smem_desc_sw128(qs + (kk >> 2) * 16384) + off,
                         smem_desc_sw128(kt + (kk >> 2) * 16384) + off, idS, kk > 0 ? 1u : 0u);
            }
            tc_commit(&s_full[gq]);
            tc_commit(&empty[sk]);
            if (t + step >= sg.nt) {  // the last scores of the piece: the query tile is free after them
              tc_commit(&q_empty[buf]);
              if (two) tc_commit(&q_empty[buf]);
            }
            ok = wait_phase(&full[sv], pv_, abort_f, g.status);
            if (ok) mbar_arrive(&v_ready[gq]);
            ok = ok && wait_phase(&p_full[gq], (uint32_t)job & 1u, abort_f, g.status);
            if (ok && t == t0 && seg > 0) ok = wait_phase(&o_free[gq], (uint32_t)(seg - 1) & 1u, abort_f, g.status);
            if (!ok) break;
            tc_fence_after();
            const uint32_t acc0 = t == t0 ? acc_first[gq] : 1u;
            const uint32_t vt = smem_u32(sm + L::kRing + sv * L::kTile);
#pragma unroll
            for (int kk = 0; kk < 8; ++kk)
              tc_mma_f16_tmem_a(tO, tS + kk * 8, smem_desc_mn(vt + kk * 2048, 16384), idO, kk > 0 ? 1u : acc0);
            if (!two) {
#pragma unroll
              for (int kk = 0; kk < 8; ++kk)
                tc_mma_f16_tmem_a(tO, tS + 64 + kk * 8, smem_desc_mn(vt + kk * 2048, 16384), idO, 1u);
            }
            tc_commit(&pv_done[gq]);
            tc_commit(&empty[sv]);
            ++job;
          }
          tiles += sg.nt;
          ++seg;
          if (two || qt == 0) ++qn0;
          if (two || qt == 1) ++qn1;
          if (!two) qt ^= 1;
        }
        tc_commit(&drain[gq]);
        mbar_wait(&drain[gq], 0, kTcWaitNs / 4);
      }
      __syncwarp();
    } else {
      // ---------------------------------------------------------- query rows
      bool ok = true;
      while (ok && walk.next(sg)) {
        const int rows = item_rows(sg);
        const bool two = rows > 128;
        for (int w = 0; ok && w < (two ? 2 : 1); ++w) {
          const int buf = two ? w : qt;
          int& used = buf ? qn1 : qn0;
          if (used > 0) ok = !stop(wait_phase(&q_empty[buf], (uint32_t)(used - 1) & 1u, abort_f, g.status));
          if (!ok) break;
          constexpr int kChunks = HD / 8, kLanes = 32 / kChunks;  // 16-byte chunks a row, rows an iteration
          const int c = lane % kChunks;
          int r = lane / kChunks;
          const int x = sg.rt * (sg.prefix ? g.rp : g.ri) + w * 128 + r;
          int row = x / g.G, h = x - row * g.G;
          if (!sg.prefix) row += sg.b * g.n;
          uint8_t* dst = sm + L::kQ + buf * L::kTile + (c >> 3) * 16384;
          for (const int lim = min(128, rows - w * 128); r < lim; r += kLanes) {
            cp_async16(dst + r * 128 + (((c & 7) ^ (r & 7)) << 4),
                       q + ((long long)row * g.nq + sg.hk * g.G + h) * HD + c * 8);
            h += kLanes;
            while (h >= g.G) {
              h -= g.G;
              ++row;
            }
          }
          cp_async_wait_all();
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&q_full[buf]);
          ++used;
        }
        if (!two) qt ^= 1;
      }
    }
  } else {
    // ------------------------------------------------------------ softmax
    reg_inc<216>();
    const int gq = (warp - 4) >> 2, qr = warp & 3;  // TMEM lane quarter
    const int r = qr * 32 + lane;
    const uint32_t lanes = (uint32_t)(qr * 32) << 16;
    const uint32_t tS = tmem + lanes + gq * 128, tO = tmem + lanes + 256 + gq * 128;
    int job = 0, xn = 0, fn = 0, fb = 0;  // tiles done; joins; phases of the scan barriers
    bool ok = true;
    while (ok && walk.next(sg)) {
      const int rows = item_rows(sg);
      const bool two = rows > 128;
      const int step = two ? 1 : 2, t0 = two ? 0 : gq;
      const int rr = r + (two ? gq * 128 : 0);  // the item's stacked row
      const ItemRow me = item_row(g, sg, rr);
      const bool warp_live = (rr - lane) < rows;  // uniform: some row of the warp belongs to the item
      int sink = 0, lo = 0, hi = 0;
      if (me.live) row_span(g, paged_len(g, me.b), paged_rows(g, me.b), me.i, sink, lo, hi);
      const int key_lo = sg.prefix ? 0 : pv.sh_tiles * KT;
      const int key_end = sg.prefix ? pv.sh_tiles * KT : key_limit(g, sg.b);
      lo = max(lo, key_lo);
      hi = min(hi, key_end);
      sink = min(sink, key_end);
      // keys that every row of the item sees: [all_lo, all_hi)
      int all_lo = 0, all_hi = key_end;
      if (!sg.prefix) {
        int a, b, c;
        const int P = paged_len(g, sg.b), n = paged_rows(g, sg.b), x = sg.rt * g.ri;
        row_span(g, P, n, (x + rows - 1) / g.G, a, all_lo, c);
        row_span(g, P, n, x / g.G, a, b, all_hi);
        all_lo = max(all_lo, key_lo);
        all_hi = min(all_hi, key_end);
      } else if (g.window > 0) {
        all_hi = 0;
      }
      float M = -INFINITY, Ls = 0.f;
      for (int t = t0; ok && t < sg.nt; t += step) {
        const int k0 = sg.span.tile(sg.t0 + t) * KT;
        const bool inner = k0 >= all_lo && k0 + KT <= all_hi;  // the same for all warps of the item
        if (stop(wait_phase(&s_full[gq], (uint32_t)job & 1u, abort_f, g.status))) {
          ok = false;
          break;
        }
        tc_fence_after();
        uint32_t v[128];
        uint32_t vw[4] = {0u, 0u, 0u, 0u};  // visible keys of the tile
        float Mn = M, f = 1.f;
        bool wfull = true;
        if (!inner) {
          const bool row_full = k0 >= key_lo && ((lo <= k0 && hi >= k0 + KT) || sink >= k0 + KT);
          wfull = __all_sync(0xffffffffu, !me.live || row_full);
          if (me.live) {
#pragma unroll
            for (int w = 0; w < 4; ++w)
              vw[w] = bits_of(lo - k0 - 32 * w, hi - k0 - 32 * w) | bits_of(key_lo - k0 - 32 * w, sink - k0 - 32 * w);
          }
        }
        auto vis = [&](int e) { return ((vw[e >> 5] >> (e & 31)) & 1u) != 0u; };
        if (warp_live) {
#pragma unroll
          for (int c = 0; c < 4; ++c) tmem_ld32(tS + c * 32, *reinterpret_cast<uint32_t(*)[32]>(&v[c * 32]));
          tmem_ld_wait();
          float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
          if (wfull) {
#pragma unroll
            for (int e = 0; e < 128; ++e) mx[e & 3] = fmaxf(mx[e & 3], __uint_as_float(v[e]));
          } else {
#pragma unroll
            for (int e = 0; e < 128; ++e) mx[e & 3] = fmaxf(mx[e & 3], vis(e) ? __uint_as_float(v[e]) : -INFINITY);
          }
          const float m = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
          bool raise = false;
          if (m != -INFINITY) {
            const float mt = m * scale_log2;
            if (M == -INFINITY) {
              Mn = mt;
            } else if (mt > M + 8.f) {
              Mn = mt;
              raise = true;
            }
          }
          if (__any_sync(0xffffffffu, raise)) {  // the group's earlier products are done: S came after them
            f = raise ? ex2f(M - Mn) : 1.f;
#pragma unroll 1
            for (int c = 0; c < HD; c += 16) {
              uint32_t o[16];
              tmem_ld16u(tO + c, o);
              tmem_ld_wait();
#pragma unroll
              for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
              tmem_st16(tO + c, o);
            }
            tmem_st_wait();
          }
        }
        const float negm = Mn == -INFINITY ? 0.f : -Mn;
        uint32_t first_acc = 0u;
        if (!inner) {
          // values that are not finite, a key a thread
          uint8_t* vt = sm + L::kRing + (2 * (tiles + t) + 1) % NS * L::kTile;
          auto chunk = [&](int key, int c) {
            return reinterpret_cast<uint4*>(vt + (c >> 3) * 16384 + key * 128 + (((c & 7) ^ (key & 7)) << 4));
          };
          uint64_t* fx = two ? &fix[2] : &fix[gq];
          int& ph = two ? fb : fn;
          ok = !stop(wait_phase(&v_ready[gq], (uint32_t)job & 1u, abort_f, g.status));
          if (!ok) break;
          uint32_t bad = 0u;
#pragma unroll
          for (int c = 0; c < HD / 8; ++c) {
            const uint4 w = *chunk(r, c);
            bad |= nonfinite2(w.x) | nonfinite2(w.y) | nonfinite2(w.z) | nonfinite2(w.w);
          }
          const uint32_t word = __ballot_sync(0xffffffffu, bad != 0u);
          if (lane == 0) {
            bad_w[gq * 4 + qr] = word;
            mbar_arrive(fx);
          }
          ok = !stop(wait_phase(fx, (uint32_t)ph & 1u, abort_f, g.status));
          ++ph;
          if (!ok) break;
          const uint32_t bw[4] = {bad_w[gq * 4], bad_w[gq * 4 + 1], bad_w[gq * 4 + 2], bad_w[gq * 4 + 3]};
          if (bw[0] | bw[1] | bw[2] | bw[3]) {  // uniform over the group
            const bool first = t == t0;
            if (first && warp_live) {
              // O starts here instead of in the first product, which must not overtake its last reader
              if (seg > 0) ok = !stop(wait_phase(&o_free[gq], (uint32_t)(seg - 1) & 1u, abort_f, g.status));
              if (!ok) break;
              tc_fence_after();
              uint32_t z[16];
#pragma unroll
              for (int e = 0; e < 16; ++e) z[e] = 0u;
              for (int c = 0; c < HD; c += 16) tmem_st16(tO + c, z);
              tmem_st_wait();
            }
            first_acc = 1u;
            if (warp_live) {
#pragma unroll 1
              for (int key = 0; key < KT; ++key) {
                auto word_of = [&](const uint32_t (&w)[4]) {
                  return key < 64 ? (key < 32 ? w[0] : w[1]) : (key < 96 ? w[2] : w[3]);
                };
                if (!((word_of(bw) >> (key & 31)) & 1u)) continue;
                const float s = __uint_as_float(tmem_ld1(tS + key));
                tmem_ld_wait();
                const bool see = (word_of(vw) >> (key & 31)) & 1u;
                const float p = ex2f(fmaf(s, scale_log2, negm));
#pragma unroll 1
                for (int c = 0; c < HD; c += 16) {
                  uint32_t o[16];
                  tmem_ld16u(tO + c, o);
                  tmem_ld_wait();
                  const uint4 w[2] = {*chunk(key, c >> 3), *chunk(key, (c >> 3) + 1)};
                  const uint32_t* x = reinterpret_cast<const uint32_t*>(w);
#pragma unroll
                  for (int e = 0; e < 16; ++e) {
                    const uint32_t hbits = (e & 1) ? x[e >> 1] & 0xffff0000u : x[e >> 1] << 16;
                    if (see && (hbits & 0x7f800000u) == 0x7f800000u)
                      o[e] = __float_as_uint(fmaf(p, __uint_as_float(hbits), __uint_as_float(o[e])));
                  }
                  tmem_st16(tO + c, o);
                  tmem_st_wait();
                }
              }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(fx);  // every row has taken what it sees
            ok = !stop(wait_phase(fx, (uint32_t)ph & 1u, abort_f, g.status));
            ++ph;
            if (!ok) break;
            if (bad) {
#pragma unroll 1
              for (int c = 0; c < HD / 8; ++c) {
                uint4 w = *chunk(r, c);
                uint32_t* x = reinterpret_cast<uint32_t*>(&w);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  if ((x[e] & 0x7f800000u) == 0x7f800000u) x[e] &= 0xffffu;
                  if ((x[e] & 0x7f80u) == 0x7f80u) x[e] &= 0xffff0000u;
                }
                *chunk(r, c) = w;
              }
            }
            fence_proxy_async_smem();
          }
        }
        if (warp_live) {
          float sum[4] = {0.f, 0.f, 0.f, 0.f};
          const float sl = scale_log2;
          // a loop each for the four kinds of tile: hidden keys or none, P as a pair or rounded once
          auto weights = [&](auto all, auto pair) {
#pragma unroll
            for (int c = 0; c < 4; ++c) {  // 32 keys
              uint32_t hi16[16], lo16[16];
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                const int k = c * 32 + 2 * e;
                float a = fmaf(__uint_as_float(v[k]), sl, negm), b = fmaf(__uint_as_float(v[k + 1]), sl, negm);
                if (!decltype(all)::value) {
                  a = vis(k) ? a : -INFINITY;
                  b = vis(k + 1) ? b : -INFINITY;
                }
                a = ex2f(a);
                b = ex2f(b);
                sum[(2 * e) & 3] += a;
                sum[(2 * e + 1) & 3] += b;
                if (decltype(pair)::value) {
                  pack_bf16_hilo(a, b, hi16[e], lo16[e]);
                } else {
                  const __nv_bfloat162 h2 = __floats2bfloat162_rn(a, b);
                  hi16[e] = *reinterpret_cast<const uint32_t*>(&h2);
                }
              }
              tmem_st16(tS + c * 16, hi16);
              if (decltype(pair)::value) tmem_st16(tS + 64 + c * 16, lo16);
            }
          };
          if (two) {
            if (wfull)
              weights(std::true_type{}, std::false_type{});
            else
              weights(std::false_type{}, std::false_type{});
          } else if (wfull) {
            weights(std::true_type{}, std::true_type{});
          } else {
            weights(std::false_type{}, std::true_type{});
          }
          Ls = fmaf(Ls, f, (sum[0] + sum[1]) + (sum[2] + sum[3]));
          M = Mn;
          tmem_st_wait();
        }
        if (t == t0 && r == 0) acc_first[gq] = first_acc;
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[gq]);
        ++job;
      }
      if (!ok) break;
      const bool has = t0 < sg.nt;
      if (has && stop(wait_phase(&pv_done[gq], (uint32_t)(job - 1) & 1u, abort_f, g.status))) break;
      // ---- the piece's end: group 0 joins both groups' parts of a single query tile, else each has its own
      float2 other = make_float2(-INFINITY, 0.f);
      if (!two) {
        if (gq == 1) {
          if (xn > 0 && stop(wait_phase(x_free, (uint32_t)(xn - 1) & 1u, abort_f, g.status))) break;
          xch[r] = make_float2(M, Ls);
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(x_full);
        } else {
          if (stop(wait_phase(x_full, (uint32_t)xn & 1u, abort_f, g.status))) break;
          other = xch[r];
          __syncwarp();
          if (lane == 0) mbar_arrive(x_free);
        }
        ++xn;
      }
      if (two || gq == 0) {
        tc_fence_after();
        const bool both = !two && sg.nt > 1;
        const float Mx = fmaxf(M, other.x);
        const float ref = Mx == -INFINITY ? 0.f : Mx;
        // (a part whose maximum is NaN keeps its NaN through its sum)
        const float wa = M == -INFINITY ? (both ? 0.f : 1.f) : ex2f(M - ref);
        const float wb = other.x == -INFINITY ? 0.f : ex2f(other.x - ref);
        const float Lt = fmaf(wb, other.y, wa * Ls);
        const bool whole = walk.whole(sg);
        const float inv = whole ? 1.f / Lt : 1.f;
        if (warp_live) {
          bf16* dst = out + (((long long)me.b * g.n + me.i) * g.nq + me.head) * HD;
          float* pdst = g.part_o + (sg.slot_row + rr) * HD;
#pragma unroll 1
          for (int c = 0; c < HD; c += 32) {
            uint32_t a[32], b[32];
            tmem_ld32(tO + c, a);
            if (both) tmem_ld32(tO + 128 + c, b);
            tmem_ld_wait();
            float x[32];
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              x[e] = __uint_as_float(a[e]);
              if (both) x[e] = fmaf(wb, __uint_as_float(b[e]), wa * x[e]);
            }
            if (me.live) {
              if (whole) {
#pragma unroll
                for (int e = 0; e < 32; e += 8) {
                  uint4 w;
                  __nv_bfloat162* h2 = reinterpret_cast<__nv_bfloat162*>(&w);
#pragma unroll
                  for (int i = 0; i < 4; ++i) h2[i] = __floats2bfloat162_rn(x[e + 2 * i] * inv, x[e + 2 * i + 1] * inv);
                  *reinterpret_cast<uint4*>(dst + c + e) = w;
                }
              } else {
#pragma unroll
                for (int e = 0; e < 32; e += 4)
                  *reinterpret_cast<float4*>(pdst + c + e) = make_float4(x[e], x[e + 1], x[e + 2], x[e + 3]);
              }
            }
          }
          if (me.live && !whole) g.part_ml[sg.slot_row + rr] = make_float2(both ? Mx : M, both ? Lt : Ls);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&o_free[gq]);
          if (!two) mbar_arrive(&o_free[1]);
        }
      }
      tiles += sg.nt;
      ++seg;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 3) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int HD>
static cudaError_t tc_launch(PagedGeom g, const CUtensorMap& tk, const CUtensorMap& tv, long long pool_rows,
                             const void* q, void* out, long long part_rows, cudaStream_t s) {
  typedef TcLayout<HD> L;
  static bool set = false;
  if (!set) {
    DFL_RET(cudaFuncSetAttribute(paged_attn_tc_kernel<HD>, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kSmem));
    set = true;
  }
  // items of two query tiles where there are rows for them
  const int ri = g.n * g.G > 128 ? 256 : 128, rp = g.batch * g.n * g.G > 128 ? 256 : 128;
  if (paged_split(g, ri, rp, num_sms(), 2) > part_rows) return cudaErrorInvalidValue;
  const float scale_log2 = 1.4426950408889634f / sqrtf((float)HD);
  DFL_RET(launch_pdl(paged_attn_tc_kernel<HD>, dim3(g.grid), dim3(kTcThreads), L::kSmem, s, tk, tv, g, (int)pool_rows,
                     (const bf16*)q, (bf16*)out, scale_log2));
  count_launch();
  return paged_merge_bf16(HD, g, out, s);
}

cudaError_t paged_attention_tc(int hd, const PagedGeom& g, const CUtensorMap& tk, const CUtensorMap& tv,
                               long long pool_rows, const void* q, void* out, long long part_rows, cudaStream_t s) {
  return hd == 64 ? tc_launch<64>(g, tk, tv, pool_rows, q, out, part_rows, s)
                  : tc_launch<128>(g, tk, tv, pool_rows, q, out, part_rows, s);
}

}  // namespace dfl
