// Attention over pages on the 5th-generation tensor cores (bf16, head_dim 64
// or 128): one persistent CTA a SM walks its run of key tiles (paged.cuh).
//
// Two groups of four softmax warps work independently, each with a score
// buffer S and an output accumulator O in TMEM and a warp that issues its
// products, so one group's exponentials run under the other's products.
// For every row a reference M: the row's first visible keys set it, a tile
// raises it only when its own max exceeds M by more than 8 (log2 units); then O
// and the row sum L are rescaled by 2^(M_old - M_new).  The weights are
// p = 2^(s - M) <= 2^8.  An item runs in one of two layouts:
//
// rows as columns (at most 64 stacked rows: single tokens, blocks)
//   S = K_t Q^T            128 keys by NR = 16, 32 or 64 rows: a thread holds a key's scores
//   O += V_t^T P           dims by rows, both operands from shared memory
//   The products' M dimension is filled with keys and dimensions, so few rows
//   cost few columns, and all 128 threads of a group share the exponentials of
//   however few rows there are.  Whether a row's reference has to move is one
//   vote a tile.  With 16 and 32 rows P is kept as a bf16 pair hi + lo in
//   neighbouring columns (2^-16 relative): the product has 64 columns anyway, and
//   splitting the weights costs 1 to 3% (with 32 rows: 8 blocks of 8 over 2K..6K
//   keys 50.5 -> 51.9 us, 32 of them 123 -> 127).  With 64 the pair would take 128
//   columns, and P is rounded once.  S has two buffers, and K runs two tiles ahead
//   of V in the ring: the next scores are there before a tile's weights are done.
//   An item's key tiles are taken by the groups in turn.
// rows as rows (more rows: chunks, shared prefixes)
//   S = Q K_t^T            128 rows by 64 keys (half a tile), two buffers: a thread
//                          holds one row
//   O += P V_t             P as bf16 over S in TMEM
//   An item of at most 128 rows has one query tile, whose key tiles the groups
//   take in turn; one of more rows has two, a group each, that share every key
//   tile, which halves the traffic from L2.
// P rounded to bf16 once (more than 32 rows) is off by 2^-8 relative a weight,
// the size of the result's own rounding: relative errors against 64 bits are
// 0.0023 there and 0.0017, the result's rounding alone, where P is a pair.  L
// sums the weights before it.  Where both groups work on the same rows, their
// (M, L, O) are joined at the item's end.
//
// Warps: 0 streams the pages (TMA, one box a page and 64 dimensions) through a
// ring of key and value tiles; 1 and 2 issue the groups' products; 3 owns TMEM
// and brings the query rows (16-byte asynchronous copies, swizzled by hand:
// stacked rows of any GQA group are packed without gaps); 4..7 and 8..11 are
// the softmax groups.
//
// A hidden key's weight is 0, and 0 times an Inf or NaN value would reach rows
// that do not see it.  So in a tile that some row sees only in part, the group
// looks through the values first; a value that is not finite is taken out of
// the tile and added with its weight to the accumulators of the rows that do
// see it.
//
// What bounds it, measured on inputs larger than L2, us a call (bytes at a copy's
// 6.78 TB/s, products at 1.92 PFLOP/s):
//   32 sequences, one token, 512 to 36K keys, 40 / 8 heads   396 (381): the bytes
//   one token over 4K keys, 32 / 8 heads                    16.9 (2.5): the start (5.5 us to the first weights),
//     one piece of two or three tiles a CTA, writing and joining the pieces (5)
//   8 blocks of 16 rows over 2K..6K keys, 32 / 8 heads      61.4 (22): the start (10 us to the first weights),
//     14 tiles a CTA at 2.5 us a tile and group, the piece (5.6), the joining kernel (10.5 by itself)
//   128 rows over 36K keys, 40 / 8 heads                     126 (51): 2.7 us a tile of 256 rows and 128 keys
//     (products alone 1.3), a row's 128 exponentials by one thread
// Rows as columns and not as rows for up to 64 rows: 128 rows' worth of exponentials would be computed for 4.
//
// Every wait is bounded (PagedGeom::wait_ns); one that gives up sets
// DFLASH_STATUS_TIMEOUT, the CTA stops, and drains its copies and products,
// whatever the limit, before it releases TMEM.
#include <math.h>

#include <algorithm>
#include <type_traits>

#include "common.cuh"
#include "internal.h"
#include "paged.cuh"

namespace dfl {

namespace {
constexpr int kTcThreads = 384;
constexpr uint64_t kTcDrainNs = 125000000ull;
constexpr float kNoRef = 3e38f;  // -M of a row that has seen no key: every score lies more than 8 above it

template <int HD>
struct TcLayout {
  static constexpr int kHalves = HD / 64;               // 64-dimension halves: 128-byte rows
  static constexpr uint32_t kTile = kHalves * 16384;    // 128 keys
  static constexpr int kSlots = HD == 128 ? 5 : 8;
  // two query buffers: a tile of 128 rows, or 64 rows and, behind them, a group's P of 128 keys x 64 rows
  static constexpr uint32_t kQ = kSlots * kTile;
  static constexpr uint32_t kQBuf = 32768;
  static constexpr uint32_t kP = 16384;                 // P within a buffer
  static constexpr uint32_t kXch = kQ + 2 * kQBuf;      // [128] (M, L) of group 1
  static constexpr uint32_t kRef = kXch + 1024;         // [2][64] row references of the rows-as-columns layout
  static constexpr uint32_t kBar = kRef + 512;
  static constexpr int kBars = 2 * kSlots + 35;
  static constexpr uint32_t kMisc = kBar + kBars * 8;   // TMEM slot, abort flag, per-group words, scan scratch
  static constexpr uint32_t kPieces = kMisc + 256;      // [4] pieces
  static constexpr int kUsed = kPieces + 4 * 96;
  static constexpr int kSmem = kUsed + 512;             // room for a base off the 1024-byte grid
  static_assert(kSmem <= 232448, "shared memory per block");
  static_assert(kMisc % 16 == 8 || kMisc % 16 == 0, "alignment");
};

// One 32-byte store (a whole sector; the address 32-byte aligned).
__device__ __forceinline__ void store32(void* dst, const uint32_t (&w)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(w[0]), "r"(w[1]), "r"(w[2]),
               "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}
// One piece of the CTA's run, as every role needs it; the last one of the run is followed by one without tiles.
struct Piece {
  int nt, prefix, two, whole;     // key tiles; both groups on each of them; no other piece has its rows
  int b, hk, rt, ordinal;         // as in Segment
  int rows, x0;                   // stacked rows of the item, the first one's number
  int s0, sn, w0, t0;             // tile t of the piece is t0 + t of the item's: s0 + t below sn, then w0 + t - sn
  int key_lo, key_end;            // keys of the item: [key_lo, key_end)
  int all_lo, all_hi;             // those that every row of it sees
  int P, n;                       // the sequence's keys before this call, its rows
  int nc, c0;                     // pieces of the item, the first one's CTA
  long long slot_row;
  __device__ __forceinline__ int tile(int t) const {
    t += t0;
    return t < sn ? s0 + t : w0 + t - sn;
  }
};
static_assert(sizeof(Piece) == 96, "a slot of the ring");

// max of three
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
// Two float32 lanes at once.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(reinterpret_cast<uint64_t&>(d))
      : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)), "l"(reinterpret_cast<uint64_t&>(c)));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("add.rn.f32x2 %0, %1, %2;"
      : "=l"(reinterpret_cast<uint64_t&>(d))
      : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)));
  return d;
}
// Sum (or maximum) over the warp's lanes of N values a lane: each step exchanges half of what is left with
// the lane `o` away.  A lane ends with N / 32 results (N = 16: one, in two lanes), those from scatter_row on.
template <int N, bool kMax>
__device__ __forceinline__ void warp_scatter(float (&x)[N], int lane) {
  int n = N;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    if (n > 1) {
      n >>= 1;
      const bool up = lane & o;
#pragma unroll
      for (int e = 0; e < N / 2; ++e)
        if (e < n) {
          const float mine = up ? x[e + n] : x[e], theirs = __shfl_xor_sync(0xffffffffu, up ? x[e] : x[e + n], o);
          x[e] = kMax ? fmaxf(mine, theirs) : mine + theirs;
        }
    } else {
      const float theirs = __shfl_xor_sync(0xffffffffu, x[0], o);
      x[0] = kMax ? fmaxf(x[0], theirs) : x[0] + theirs;
    }
  }
}
// (lane bits 16, 8, ... select halves: the first row of a lane's results)
template <int N>
__device__ __forceinline__ int scatter_row(int lane) {
  int row = 0, n = N;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    if (n > 1) {
      n >>= 1;
      if (lane & o) row += n;
    }
  return row;
}

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

__device__ __forceinline__ bool give_up(volatile int* abort_f, const PagedGeom& g) {
  *abort_f = 1;
  set_status(g.status, DFLASH_STATUS_TIMEOUT);
  return false;
}
// Waits for a phase, giving up on the CTA's abort flag or after the limit (then raising the flag).
__device__ __forceinline__ bool wait_phase(uint64_t* bar, uint32_t parity, volatile int* abort_f,
                                           const PagedGeom& g) {
#pragma unroll 1
  for (int i = 0; i < 64; ++i)
    if (mbar_try_wait(bar, parity)) return true;
  const uint32_t t0 = global_ns_lo();
  while (true) {
#pragma unroll 1
    for (int i = 0; i < 64; ++i)
      if (mbar_try_wait(bar, parity)) return true;
    if (*abort_f) return false;
    if (global_ns_lo() - t0 > g.wait_ns) return give_up(abort_f, g);
  }
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

// NR: rows of the rows-as-columns layout (0: it is not used); TS, TP: suffix / prefix items use it.
template <int HD, int NR, bool TS, bool TP>
__global__ void __launch_bounds__(kTcThreads, 1)
    paged_attn_tc_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                         const __grid_constant__ PagedGeom g, int pool_rows, const bf16* __restrict__ q,
                         bf16* __restrict__ out, float scale_log2) {
  typedef TcLayout<HD> L;
  constexpr int KT = kPagedTcKeys, NS = L::kSlots;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  if (sm - smem_raw > L::kSmem - L::kUsed) {  // (the base is on the grid; were it not, nothing would be written)
    set_status(g.status, DFLASH_STATUS_TIMEOUT);
    return;
  }
  uint64_t* bar = reinterpret_cast<uint64_t*>(sm + L::kBar);
  uint64_t* full = bar;              // [NS] a key or value tile has landed
  uint64_t* empty = bar + NS;        // [NS] both issuing warps are done with it
  uint64_t* q_full = bar + 2 * NS;   // [2]
  uint64_t* q_empty = q_full + 2;    // [2] read by its last product, and seen by both issuing warps
  uint64_t* s_full = q_full + 4;     // [2][2] scores of the group's tile (rows as rows: half tile) in TMEM
  uint64_t* p_full = q_full + 8;     // [2][2] the buffer's weights (four warps; one may be a job ahead of another)
  uint64_t* pv_done = q_full + 12;   // [2][2] the product of weights and values of the buffer's job is done
  uint64_t* o_free = q_full + 16;    // [2] the accumulator has been read (four warps), for pieces with a tile of the
                                     // group's
  uint64_t* fix = q_full + 18;       // [3] meetings of group 0, group 1 (four warps), both (eight)
  uint64_t* x_full = q_full + 21;    // group 1's M and L are written (four warps)
  uint64_t* x_free = q_full + 22;    // and read
  uint64_t* drain = q_full + 23;     // [2] every product a warp issued is done
  uint64_t* v_ready = q_full + 25;   // [2] the values of the group's tile have landed
  uint64_t* pc_full = q_full + 27;   // [4] a piece is described
  uint64_t* pc_empty = q_full + 31;  // [4] and no role needs its description (11 warps)
  uint32_t* misc = reinterpret_cast<uint32_t*>(sm + L::kMisc);
  uint32_t* tslot = misc;
  volatile int* abort_f = reinterpret_cast<volatile int*>(misc + 1);
  volatile uint32_t* acc_first = misc + 2;  // [2] the first product of an item adds to O instead of setting it
  volatile uint32_t* bad_w = misc + 4;      // [2][4] keys of the tile with a value that is not finite
  int* red = reinterpret_cast<int*>(misc + 12);  // 32 ints
  int* gap = red;                    // [4][2] after the plan, with a window: pages of a piece whose first key lies in
                                     // the [1] keys from [0] on are seen by no row of its item
  volatile uint32_t* last_w = misc + 44;    // the CTA has finished an item's last piece
  volatile uint32_t* vote_w = misc + 46;    // [2][2][4] some reference of the tile has to move
  volatile uint32_t* o_uses = misc + 62;    // [2] pieces with a tile of the group before this one (with v_ready)
  float2* xch = reinterpret_cast<float2*>(sm + L::kXch);
  Piece* pieces = reinterpret_cast<Piece*>(sm + L::kPieces);
  auto as_columns = [](int prefix) { return prefix ? TP : TS; };
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
      mbar_init(&s_full[2 * i], 1);
      mbar_init(&s_full[2 * i + 1], 1);
      mbar_init(&p_full[2 * i], 4);
      mbar_init(&p_full[2 * i + 1], 4);
      mbar_init(&pv_done[2 * i], 1);
      mbar_init(&pv_done[2 * i + 1], 1);
      mbar_init(&o_free[i], 4);
      mbar_init(&fix[i], 4);
      mbar_init(&drain[i], 1);
      mbar_init(&v_ready[i], 1);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(&pc_full[i], 1);
      mbar_init(&pc_empty[i], 11);
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
  PlanView pv;
  if (g.batch > kPlanSmall) {  // a larger batch is planned by the whole block
    pdl_wait();
    pv = plan_view<KT, kTcThreads>(g, red);
  }
  // Order of an item's tiles in the ring: keys run `ahead` tiles ahead of values.
  auto ahead_of = [](bool cols) { return cols ? 2 : 0; };
  auto k_at = [](int t, int ahead) { return t + max(0, t - ahead); };
  auto v_at = [](int t, int ahead, int nt) { return min(nt, t + ahead + 1) + t; };
  // query buffers: an item with one tile takes the buffer after the last one's, an item with two both
  int seg = 0, qt = 0, qn0 = 0, qn1 = 0;
  int tiles = 0;  // key tiles before the current piece
  auto stop = [&](bool ok) { return __any_sync(0xffffffffu, !ok); };
  // The pieces of the run come from warp 3 through a ring of four.
  auto wait_piece = [&](int s) {
    return !stop(wait_phase(&pc_full[s & 3], (uint32_t)(s >> 2) & 1u, abort_f, g));
  };
  auto done_piece = [&](int s) {
    __syncwarp();
    if (lane == 0) mbar_arrive(&pc_empty[s & 3]);
  };

  if (warp < 4) {
    reg_dec<88>();
    if (warp == 0) {
      // ---------------------------------------------------------- pages
      const int per = KT >> g.ps_log2;  // pages a tile
      const bool mine = lane < per;
      bool ok = true;  // (`tiles` counts slots filled here)
      pdl_wait();
      for (; (ok = wait_piece(seg)); ++seg) {
        const Piece& pc = pieces[seg & 3];
        const int nt = pc.nt, hk = pc.hk, key_end = pc.key_end;
        if (nt == 0) break;
        const int gap0 = g.window > 0 ? gap[2 * (seg & 3)] : 0;
        const unsigned gap_n = g.window > 0 ? gap[2 * (seg & 3) + 1] : 0u;
        const int32_t* trow = g.table + (long long)pc.b * g.table_stride;
        // Whether some row sees a key of this lane's page of tile t: its entry may be anything otherwise.
        auto used = [&](int t) {
          const int key = pc.tile(t) * KT + (lane << g.ps_log2);
          return mine && t < nt && key < key_end && (unsigned)(key - gap0) >= gap_n;
        };
        // The page, and its pool row (a page that is none, or not used: past the pool, read as zeros).
        auto page_of = [&](int t, bool use) { return use ? trow[pc.tile(t) * per + lane] : -1; };
        auto row_of = [&](bool use, int page) {
          if ((unsigned)page < (unsigned)g.n_pages)
            return (int)(g.page_row0 + ((long long)page * g.nkv + hk) * g.ps);
          if (use) set_status(g.status, DFLASH_STATUS_BOUNDS);
          return pool_rows;
        };
        const int ahead = ahead_of(as_columns(pc.prefix));
        // the rows of the next tiles: [0] the next value tile's, [ahead] the next key tile's
        int rowq[3];
        {
          const bool use[3] = {used(0), used(1), used(2)};
#pragma unroll
          for (int a = 0; a < 3; ++a) rowq[a] = page_of(a, use[a]);
#pragma unroll
          for (int a = 0; a < 3; ++a) rowq[a] = row_of(use[a], rowq[a]);
        }
        for (int u = 0; ok && u < nt + ahead; ++u) {
          const int x = min(u, ahead), krow = x == 0 ? rowq[0] : x == 1 ? rowq[1] : rowq[2];
          const bool next_use = u >= ahead && used(u - ahead + 3);
          const int next_page = page_of(u - ahead + 3, next_use);
#pragma unroll
          for (int kv = 0; kv < 2; ++kv) {
            if (kv == 0 ? u >= nt : u < ahead) continue;
            const int s = tiles % NS;
            if (tiles >= NS && stop(wait_phase(&empty[s], (uint32_t)(tiles / NS - 1) & 1u, abort_f, g))) {
              ok = false;
              break;
            }
            uint8_t* dst = sm + s * L::kTile;
            if (elect_one()) mbar_arrive_expect_tx(&full[s], L::kTile);
#pragma unroll 1
            for (int p = 0; p < per; ++p) {
              const int y = __shfl_sync(0xffffffffu, kv == 0 ? krow : rowq[0], p);
              uint8_t* at_p = dst + ((p << g.ps_log2) << 7);
              if (elect_one()) {
#pragma unroll
                for (int dh = 0; dh < L::kHalves; ++dh)
                  tma_load_2d(at_p + dh * 16384, kv == 0 ? &tmK : &tmV, &full[s], dh * 64, y);
              }
            }
            ++tiles;
          }
          if (u >= ahead) {
            rowq[0] = rowq[1];
            rowq[1] = rowq[2];
            rowq[2] = row_of(next_use, next_page);
          }
        }
        if (!ok) break;
        done_piece(seg);
      }
      // the last copies land before the CTA leaves, whatever became of their readers
      for (int x = max(0, tiles - NS); x < tiles; ++x) mbar_wait(&full[x % NS], (uint32_t)(x / NS) & 1u, kTcDrainNs);
    } else if (warp < 3) {
      // ---------------------------------------------------------- products of group gq
      const int gq = warp - 1;
      const uint32_t idS = idesc_bf16_f32(128, 64), idO = idesc_bf16_f32(128, HD) | (1u << 16);  // values MN-major
      const uint32_t idSt = idesc_bf16_f32(128, NR > 0 ? NR : 16);
      const uint32_t idOt = idesc_bf16_f32(128, 64) | (3u << 15);  // values and weights both MN-major
      const uint32_t tS = tmem + gq * 128, tO = tmem + 256 + gq * 128;
      auto wait = [&](uint64_t* b, uint32_t parity) { return !stop(wait_phase(b, parity & 1u, abort_f, g)); };
      int job = 0, on = 0;  // on: pieces with a tile of this group
      bool ok = true;
      pdl_wait();
      // No wait may be lapped: a barrier's next phase needs every warp that waits for this one.  So both warps let go
      // of a query tile, also of one that only the other reads; and o_free has no phase for a piece without a tile
      // of the group, which ends without this warp.
      // Both issuing warps see every tile land and release it: a slot is refilled only after both have
      // been past it, so a wait never looks at a phase two fills away.
      while (ok && (ok = wait_piece(seg))) {
        const int nt = pieces[seg & 3].nt;
        if (nt == 0) break;
        const bool cols = as_columns(pieces[seg & 3].prefix), two = pieces[seg & 3].two;
        done_piece(seg);
        const int ahead = ahead_of(cols);
        const int buf = two ? gq : qt;
        if (two || qt == 0) ok = wait(&q_full[0], qn0);
        if (ok && (two || qt == 1)) ok = wait(&q_full[1], qn1);
        const bool has = two || gq < nt;  // some tile for this group
        if (ok && (two || !has) && elect_one()) mbar_arrive(&q_empty[two ? gq ^ 1 : buf]);
        const uint8_t* qs = sm + L::kQ + buf * L::kQBuf;
        if (cols) {
          int kjob = job;  // keys run ahead
          for (int u = 0; ok && u < nt + ahead; ++u) {
            if (u < nt) {
              const int x = 2 * tiles + k_at(u, ahead), sk = x % NS;
              ok = wait(&full[sk], x / NS);
              if (!ok) break;
              if ((u & 1) != gq) {  // the other group's tile
                if (elect_one()) mbar_arrive(&empty[sk]);
              } else {
                // (after the other layout: its last P lies where these scores go)
                if (!TP && kjob == job && kjob > 0) ok = wait(&pv_done[2 * gq + (kjob - 1 & 1)], kjob - 1 >> 1);
                if (!ok) break;
                tc_fence_after();
                const uint8_t* kt = sm + sk * L::kTile;
                const uint32_t d = tS + (kjob & 1) * 64;
                if (elect_one()) {
#pragma unroll
                  for (int kk = 0; kk < HD / 16; ++kk) {
                    const uint64_t off = (uint64_t)(((kk & 3) * 32) >> 4);
                    tc_mma_f16(d, smem_desc_sw128(kt + (kk >> 2) * 16384) + off,
                               smem_desc_sw128(qs + (kk >> 2) * 8192) + off, idSt, kk > 0 ? 1u : 0u);
                  }
                  tc_commit(&s_full[2 * gq + (kjob & 1)]);
                  tc_commit(&empty[sk]);
                  // The last scores of the piece: the query tile is free after them.  (Where the other layout comes
                  // first, it is free after the last product: the hand-over below counts on it.)
                  if (TP && u + 2 >= nt) tc_commit(&q_empty[buf]);
                }
                __syncwarp();
                ++kjob;
              }
            }
            if (u >= ahead) {
              const int t = u - ahead, x = 2 * tiles + v_at(t, ahead, nt), sv = x % NS;
              ok = wait(&full[sv], x / NS);
              if (!ok) break;
              if ((t & 1) != gq) {
                if (elect_one()) mbar_arrive(&empty[sv]);
              } else {
                const bool first = t == gq;
                if (elect_one()) {
                  o_uses[gq] = on;
                  mbar_arrive(&v_ready[gq]);
                }
                ok = wait(&p_full[2 * gq + (job & 1)], job >> 1);
                if (ok && first && on > 0) ok = wait(&o_free[gq], on - 1);
                if (!ok) break;
                tc_fence_after();
                const uint32_t acc0 = first ? acc_first[gq] : 1u;
                const uint32_t vt = smem_u32(sm + sv * L::kTile);
                if (elect_one()) {
                  // (head_dim 64: the upper 64 lanes take what lies behind the tile, and nothing reads them)
                  const uint32_t ps = smem_u32(sm + L::kQ + gq * L::kQBuf + L::kP);
#pragma unroll
                  for (int kk = 0; kk < 8; ++kk)
                    tc_mma_f16(tO, smem_desc_mn(vt + kk * 2048, 16384), smem_desc_mn(ps + kk * 2048, 16384), idOt,
                               kk > 0 ? 1u : acc0);
                  tc_commit(&pv_done[2 * gq + (job & 1)]);
                  tc_commit(&empty[sv]);
                  if (!TP && t + 2 >= nt) tc_commit(&q_empty[buf]);
                }
                __syncwarp();
                ++job;
              }
            }
          }
        } else {
          // Half a tile is a job: scores of 64 keys in one of two buffers, P over them.  The first half's product
          // and the next tile's first scores run while the group is at the second half, and the other way round.
          int vp = -1;  // slot of the value tile whose second half is still to be multiplied
          auto half_pv = [&](int j, int sv, uint32_t acc0) {  // P V of job j
            const int hf = j & 1;
            const uint32_t vt = smem_u32(sm + sv * L::kTile) + hf * 8192;
            if (elect_one()) {
#pragma unroll
              for (int kk = 0; kk < 4; ++kk)
                tc_mma_f16_tmem_a(tO, tS + hf * 64 + kk * 8, smem_desc_mn(vt + kk * 2048, 16384), idO,
                                  kk > 0 ? 1u : acc0);
              tc_commit(&pv_done[2 * gq + hf]);
              if (hf) tc_commit(&empty[sv]);
            }
            __syncwarp();
          };
          auto half_s = [&](int hf, const uint8_t* kt) {  // scores of a half
            if (elect_one()) {
#pragma unroll
              for (int kk = 0; kk < HD / 16; ++kk) {
                const uint64_t off = (uint64_t)(((kk & 3) * 32) >> 4);
                tc_mma_f16(tS + hf * 64, smem_desc_sw128(qs + (kk >> 2) * 16384) + off,
                           smem_desc_sw128(kt + (kk >> 2) * 16384 + hf * 8192) + off, idS, kk > 0 ? 1u : 0u);
              }
              tc_commit(&s_full[2 * gq + hf]);
            }
            __syncwarp();
          };
          for (int u = 0; ok && u < nt; ++u) {
            const int xk = 2 * (tiles + u), sk = xk % NS, sv = (xk + 1) % NS;
            ok = wait(&full[sk], xk / NS);
            if (!ok) break;
            if (!two && (u & 1) != gq) {  // the other group's tile
              if (elect_one()) mbar_arrive(&empty[sk]);
              ok = wait(&full[sv], (xk + 1) / NS);
              if (ok && elect_one()) mbar_arrive(&empty[sv]);
              continue;
            }
            const uint8_t* kt = sm + sk * L::kTile;
            const bool first = u == (two ? 0 : gq);
            // P lies over the last scores of a buffer until its product is done
            if (job > 1) ok = wait(&pv_done[2 * gq + (job - 2 & 1)], job - 2 >> 1);
            if (!ok) break;
            tc_fence_after();
            half_s(0, kt);
            if (vp >= 0) {
              ok = wait(&p_full[2 * gq + 1], job - 1 >> 1);
              if (!ok) break;
              tc_fence_after();
              half_pv(job - 1, vp, 1u);
            }
            if (job > 0) ok = wait(&pv_done[2 * gq + (job - 1 & 1)], job - 1 >> 1);
            if (!ok) break;
            tc_fence_after();
            half_s(1, kt);
            if (elect_one()) {
              tc_commit(&empty[sk]);
              if (u + (two ? 1 : 2) >= nt) {  // the last scores of the piece: the query tile is free after them
                tc_commit(&q_empty[buf]);
              }
            }
            __syncwarp();
            ok = wait(&full[sv], (xk + 1) / NS);
            if (ok && elect_one()) {
              o_uses[gq] = on;
              mbar_arrive(&v_ready[gq]);
            }
            ok = ok && wait(&p_full[2 * gq], job >> 1);
            if (ok && first && on > 0) ok = wait(&o_free[gq], on - 1);
            if (!ok) break;
            tc_fence_after();
            half_pv(job, sv, first ? acc_first[gq] : 1u);
            vp = sv;
            job += 2;
          }
          if (ok && vp >= 0) {
            ok = wait(&p_full[2 * gq + 1], job - 1 >> 1);
            if (ok) {
              tc_fence_after();
              half_pv(job - 1, vp, 1u);
            }
          }
        }
        tiles += nt;
        on += has;
        ++seg;
        if (two || qt == 0) ++qn0;
        if (two || qt == 1) ++qn1;
        if (!two) qt ^= 1;
      }
      if (elect_one()) tc_commit(&drain[gq]);
      mbar_wait(&drain[gq], 0, kTcDrainNs);
      __syncwarp();
    } else {
      // ---------------------------------------------------------- pieces, query rows
      bool ok = true;
      SegmentWalk<KT> walk(g, pv);
      Segment sg;
      const bool small = g.batch <= kPlanSmall;
      // One pass ahead (seg -1) runs the plan and the first piece on assumed lengths while the previous kernel
      // ends, and leaves nothing: no role can start before these few hundred instructions, and fetching them
      // takes three to four times as long as running them once they are there.  The lengths are the previous
      // kernels' to write until pdl_wait: before it they are only asked into L2, not read.
      if (small) {
        if (lane * 32 < g.batch) {
          l2_prefetch(g.len + lane * 32);
          if (g.n_rows) l2_prefetch(g.n_rows + lane * 32);
        }
        if (g.shared && lane == 0) l2_prefetch(g.shared);
      }
      for (seg = small ? -1 : 0; ok; ++seg) {
        walk.early = seg < 0;
        if (seg <= 0) {
          if (seg == 0) pdl_wait();
          if (small) pv = plan_small<KT>(g, seg == 0, seg < 0);
          walk.start();
        }
        const bool more = walk.next(sg);
        Piece pc = {};
        if (more) {
          pc.nt = sg.nt;
          pc.prefix = sg.prefix;
          pc.whole = walk.whole(sg);
          pc.b = sg.b;
          pc.hk = sg.hk;
          pc.rt = sg.rt;
          pc.ordinal = sg.ordinal;
          pc.n = paged_rows(g, sg.b, seg < 0);
          pc.P = min(paged_len(g, sg.b, seg < 0), g.cap);
          pc.x0 = sg.rt * (sg.prefix ? g.rp : g.ri);
          pc.rows = sg.prefix ? min(g.rp, g.batch * g.n * g.G - pc.x0) : min(g.ri, pc.n * g.G - pc.x0);
          pc.two = pc.rows > 128;  // (rows as columns: never)
          pc.s0 = sg.span.s0;
          pc.sn = sg.span.s1 - sg.span.s0;
          pc.w0 = sg.span.w0;
          pc.t0 = sg.t0;
          pc.key_lo = sg.prefix ? 0 : pv.sh_tiles * KT;
          pc.key_end = sg.prefix ? pv.sh_tiles * KT : min(pc.P + pc.n, g.cap);
          pc.all_lo = pc.key_lo;
          pc.all_hi = pc.key_end;
          if (!sg.prefix) {
            int a, b, lo, hi;
            row_span(g, pc.P, pc.n, div_g(g, pc.x0 + pc.rows - 1), a, lo, b);
            row_span(g, pc.P, pc.n, div_g(g, pc.x0), a, b, hi);
            pc.all_lo = max(lo, pc.key_lo);
            pc.all_hi = min(hi, pc.key_end);
          } else if (g.window > 0) {
            pc.all_hi = 0;
          }
          if (NR == 16 && pv.pre_tiles == 0 && !pc.whole) pc.nc = walk.pieces(sg, pc.c0);  // (who joins here)
          pc.slot_row = sg.slot_row;
        }
        if (seg < 0) {
          asm volatile("" ::"r"(pc.nt), "r"(pc.rows), "r"(pc.all_lo), "r"(pc.all_hi), "r"(pc.key_end), "r"(pc.nc),
                       "r"(pc.whole));  // (computed here too)
          continue;
        }
        if (seg >= 4) ok = !stop(wait_phase(&pc_empty[seg & 3], (uint32_t)((seg >> 2) - 1) & 1u, abort_f, g));
        if (!ok) break;
        if (lane == 0) {
          pieces[seg & 3] = pc;
          if (g.window > 0) {
            // between the first row's first tokens and its window (other rows' first tokens end later only where
            // they meet it)
            int sink, lo, hi;
            row_span(g, pc.prefix ? pv.min_len : pc.P, pc.n, pc.prefix ? 0 : div_g(g, pc.x0), sink, lo, hi);
            gap[2 * (seg & 3)] = sink;
            gap[2 * (seg & 3) + 1] = max(lo - g.ps + 1 - sink, 0);
          }
          mbar_arrive(&pc_full[seg & 3]);
        }
        __syncwarp();
        if (NR != 16 && seg == 0 && !g.shared) {
          // the item that this CTA's run begins inside of, when it is the second to hold a piece of it
          int c0 = 0, nc = 0;
          if (more && sg.t0 > 0) nc = walk.pieces(sg, c0);
          if (c0 + 1 != blockIdx.x) nc = 0;
          int4* rec = reinterpret_cast<int4*>(g.records) + 2 * blockIdx.x;
          if (lane == 0) {
            rec[0] = make_int4(nc, sg.b, sg.rt, sg.hk);
            rec[1].x = c0;
          }
        }
        if (!more) break;
        if (g.wait_ns == 0) {  // (a limit of 0 has expired before the first poll)
          give_up(abort_f, g);
          break;
        }
        const int rows = pc.rows;
        const bool cols = as_columns(pc.prefix), two = pc.two;
        for (int w = 0; ok && w < (two ? 2 : 1); ++w) {
          const int buf = two ? w : qt;
          int& used = buf ? qn1 : qn0;
          if (used > 0) ok = !stop(wait_phase(&q_empty[buf], (uint32_t)(used - 1) & 1u, abort_f, g));
          if (!ok) break;
          constexpr int kChunks = HD / 8, kLanes = 32 / kChunks;  // 16-byte chunks a row, rows an iteration
          const int c = lane % kChunks;
          const int r = lane / kChunks;
          const int x = pc.x0 + w * 128 + r;
          const int row = div_g(g, x);
          int h = x - row * g.G;
          const bf16* src = q + ((long long)(row + (pc.prefix ? 0 : pc.b * g.n)) * g.nq + pc.hk * g.G + h) * HD + c * 8;
          // the next row of this lane is kLanes stacked rows on
          const int dq = div_g(g, kLanes), dh = kLanes - dq * g.G;
          const long long step = ((long long)dq * g.nq + dh) * HD, wrap = (long long)(g.nq - g.G) * HD;
          // four steps at a time: their swizzled places repeat every 8 rows
          uint8_t* dst = sm + L::kQ + buf * L::kQBuf + (c >> 3) * (cols ? 8192 : 16384) + r * 128;
          uint32_t at[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) at[k] = k * kLanes * 128 + (((c & 7) ^ ((r + k * kLanes) & 7)) << 4);
          const int lim = min(128, rows - w * 128) - r;
#pragma unroll 1
          for (int x4 = 0; x4 < lim; x4 += 4 * kLanes) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
              if (x4 + k * kLanes < lim) {
                cp_async16(dst + at[k], src);
                src += step;
                h += dh;
                if (h >= g.G) {
                  h -= g.G;
                  src += wrap;
                }
              }
            dst += 4 * kLanes * 128;
          }
          // (rows past the item's: scores of 0, which nothing reads)
          if (cols) {
            dst = sm + L::kQ + buf * L::kQBuf + (c >> 3) * 8192;
            for (int y = rows / kLanes * kLanes + r; y < NR; y += kLanes)
              if (y >= rows) *reinterpret_cast<uint4*>(dst + y * 128 + (((c & 7) ^ (y & 7)) << 4)) = make_uint4(0u, 0u, 0u, 0u);
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
    reg_inc<208>();
    const int gq = (warp - 4) >> 2, qr = warp & 3;  // TMEM lane quarter
    const int r = qr * 32 + lane;
    const uint32_t lanes = (uint32_t)(qr * 32) << 16;
    const uint32_t tS = tmem + lanes + gq * 128, tO = tmem + lanes + 256 + gq * 128;
    int vjob = 0;                         // tiles done
    int job = 0, xn = 0, fn = 0, fb = 0;  // score buffers done (half tiles of rows as rows); joins; phases of the group's meetings and of both groups'
    uint32_t sn0 = 0, sn1 = 0;            // uses of the score buffers
    bool handover = false;                // a query tile of the rows-as-rows layout may still lie where P goes
    const float sl = scale_log2;
    bool ok = true;
    // a barrier of the group (or of both); false: the CTA stops
    auto meet = [&](uint64_t* b, int& ph) {
      __syncwarp();
      if (lane == 0) mbar_arrive(b);
      const bool good = !stop(wait_phase(b, (uint32_t)ph & 1u, abort_f, g));
      ++ph;
      return good;
    };
    // 16-byte chunk c of key `key` in a value tile
    auto chunk = [&](uint8_t* vt, int key, int c) {
      return reinterpret_cast<uint4*>(vt + (c >> 3) * 16384 + key * 128 + (((c & 7) ^ (key & 7)) << 4));
    };
    // x 0 is NaN for an x that is not finite, and so is a sum that has met it (n chunks of a key from c0 on)
    auto row_is_bad = [&](uint8_t* vt, int key, int c0, const int n) {
      const __nv_bfloat162 zero = __floats2bfloat162_rn(0.f, 0.f);
      __nv_bfloat162 acc[4] = {zero, zero, zero, zero};
#pragma unroll
      for (int c = 0; c < n; ++c) {
        const uint4 w = *chunk(vt, key, c0 + c);
        const __nv_bfloat162* x = reinterpret_cast<const __nv_bfloat162*>(&w);
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[e] = __hfma2(x[e], zero, acc[e]);
      }
      const float2 f = __bfloat1622float2(__hadd2(__hadd2(acc[0], acc[1]), __hadd2(acc[2], acc[3])));
      return f.x != 0.f || f.y != 0.f;
    };
    auto clean_row = [&](uint8_t* vt, int key, int c0, int n) {
#pragma unroll 1
      for (int c = c0; c < c0 + n; ++c) {
        uint4 w = *chunk(vt, key, c);
        uint32_t* x = reinterpret_cast<uint32_t*>(&w);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if ((x[e] & 0x7f800000u) == 0x7f800000u) x[e] &= 0xffffu;
          if ((x[e] & 0x7f80u) == 0x7f80u) x[e] &= 0xffff0000u;
        }
        *chunk(vt, key, c) = w;
      }
    };
    // an item's first product comes after this when its accumulator starts here
    auto zero_o = [&](int cols) {
      uint32_t z[16];
#pragma unroll
      for (int e = 0; e < 16; ++e) z[e] = 0u;
      for (int c = 0; c < cols; c += 16) tmem_st16(tO + c, z);
      tmem_st_wait();
    };
    // After a partial result: the CTA that finishes the item's last piece joins them all.
    auto join = [&](const Piece& pc) {
      if (!meet(&fix[gq], fn)) return false;
      if (r == 0) {
        __threadfence();
        const bool last = atomicAdd(g.tickets + pc.ordinal, 1) == pc.nc - 1;
        if (last) g.tickets[pc.ordinal] = 0;
        *last_w = last;
      }
      if (!meet(&fix[gq], fn)) return false;
      if (*last_w) {
        __threadfence();
        merge_item<bf16, HD>(g, pc.b, pc.rt, pc.hk, 0, pc.rows, pc.nc, pc.c0, qr, 4, out);
      }
      return true;
    };
    // While the first piece is planned and brought, the code of a first tile in the rows-as-columns layout is run
    // once on whatever TMEM holds: fetching its instructions costs several times what running them does.  Nothing
    // of it stays: the waits, the arrivals and the global reads are left out, and the first tile sets what it uses.
    // 8 blocks of 16 rows over 2K..6K keys 65.7 -> 61.4 us, 15 rows in windows of 4K 85.1 -> 82.6, single tokens
    // the same.
    int dry = 0;  // (where no item of the other layout comes first)
    if constexpr (NR > 0 && TP) {
      dry = 1;
      asm volatile("" : "+r"(dry));  // (one copy of the code)
    }
    if (!dry) {
      pdl_wait();
      ok = wait_piece(0);
    }
    // Prefix items come before suffix items, so those in the rows-as-rows layout (if any) come first.
    if constexpr (!TS || !TP) {
      while (ok && !dry && pieces[seg & 3].nt > 0 && !as_columns(pieces[seg & 3].prefix)) {
        // ------------------------------------------------ rows as rows: thread = stacked row
        const Piece& pc = pieces[seg & 3];
        const int nt = pc.nt, rows = pc.rows, key_lo = pc.key_lo, key_end = pc.key_end;
        const bool two = pc.two, whole = pc.whole;
        const int step = two ? 1 : 2, t0 = two ? 0 : gq;
        const bool has = t0 < nt, both = !two && nt > 1;
        const int rr = r + (two ? gq * 128 : 0);  // of the item
        const ItemRow me = item_row(g, pc.prefix, pc.b, pc.hk, pc.x0, rr);
        const bool warp_live = (rr - lane) < rows;  // some row of the warp belongs to the item
        int sink = 0, lo = 0, hi = 0;
        if (me.live) row_span(g, paged_len(g, me.b), paged_rows(g, me.b), me.i, sink, lo, hi);
        lo = max(lo, key_lo);
        hi = min(hi, key_end);
        sink = min(sink, key_end);
        float M = -INFINITY, Ls = 0.f;
        int own = 0;  // tiles of this group in the piece
        for (int x = 2 * t0; ok && x < 2 * nt; x += (x & 1) ? 2 * step - 1 : 1) {  // half tiles
          const int t = x >> 1, hf = x & 1;
          const bool first = x == 2 * t0;
          const int k0 = pc.tile(t) * KT + hf * 64;
          const bool inner = k0 >= pc.all_lo && k0 + 64 <= pc.all_hi;  // the same for all warps of the item
          const uint32_t tH = tS + hf * 64;
          uint32_t& sn = hf ? sn1 : sn0;
          if (stop(wait_phase(&s_full[2 * gq + hf], sn & 1u, abort_f, g))) {
            ok = false;
            break;
          }
          ++sn;
          // O may be changed once the last product is done (the one before it is: these scores came after it)
          auto wait_pv = [&]() {
            if (!first) {
              ok = !stop(wait_phase(&pv_done[2 * gq + (job - 1 & 1)], (uint32_t)(job - 1 >> 1) & 1u, abort_f, g));
              tc_fence_after();
            }
            return ok;
          };
          tc_fence_after();
          float v[64];
          uint32_t vw[2] = {0u, 0u};  // visible keys of the half
          float Mn = M, f = 1.f;
          bool wfull = true;
          if (!inner) {
            const bool row_full = k0 >= key_lo && ((lo <= k0 && hi >= k0 + 64) || sink >= k0 + 64);
            wfull = __all_sync(0xffffffffu, !me.live || row_full);
            if (me.live) {
#pragma unroll
              for (int w = 0; w < 2; ++w)
                vw[w] = bits_of(lo - k0 - 32 * w, hi - k0 - 32 * w) | bits_of(key_lo - k0 - 32 * w, sink - k0 - 32 * w);
            }
          }
          if (warp_live) {
#pragma unroll
            for (int c = 0; c < 2; ++c) tmem_ld32(tH + c * 32, *reinterpret_cast<uint32_t(*)[32]>(&v[c * 32]));
            tmem_ld_wait();
            if (!wfull) {
#pragma unroll
              for (int e = 0; e < 64; ++e)
                if (!((vw[e >> 5] >> (e & 31)) & 1u)) v[e] = -INFINITY;
            }
            float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int e = 0; e < 64; e += 8)
#pragma unroll
              for (int w = 0; w < 4; ++w) mx[w] = max3(mx[w], v[e + w], v[e + w + 4]);
            const float m = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
            bool raise = false;
            if (m != -INFINITY) {
              const float mt = m * sl;
              if (M == -INFINITY) {
                Mn = mt;
              } else if (mt > M + 8.f) {
                Mn = mt;
                raise = true;
              }
            }
            if (__any_sync(0xffffffffu, raise)) {
              if (!wait_pv()) break;
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
            // values that are not finite, two threads a key
            uint8_t* vt = sm + (2 * (tiles + t) + 1) % NS * L::kTile;
            uint64_t* fx = two ? &fix[2] : &fix[gq];
            int& ph = two ? fb : fn;
            ok = !stop(wait_phase(&v_ready[gq], (uint32_t)(vjob + own) & 1u, abort_f, g));
            if (!ok) break;
            const int vkey = hf * 64 + (r & 63), c0 = (r >> 6) * (HD / 16);
            const bool bad = row_is_bad(vt, vkey, c0, HD / 16);
            const uint32_t word = __ballot_sync(0xffffffffu, bad);
            volatile uint32_t* words = vote_w + (hf * 2 + gq) * 4;  // (two sets: a warp may be a half ahead)
            if (lane == 0) words[qr] = word;
            ok = meet(fx, ph);
            if (!ok) break;
            const uint32_t bw[2] = {words[0] | words[2], words[1] | words[3]};
            if (bw[0] | bw[1]) {  // uniform over the item's groups
              if (warp_live) {
                if (!wait_pv()) break;
                if (first) {
                  // O starts here instead of in the first product, which must not overtake its last reader
                  const uint32_t on = o_uses[gq];
                  if (on > 0) ok = !stop(wait_phase(&o_free[gq], (on - 1) & 1u, abort_f, g));
                  if (!ok) break;
                  tc_fence_after();
                  zero_o(HD);
                }
#pragma unroll 1
                for (int key = 0; key < 64; ++key) {
                  if (!(((key < 32 ? bw[0] : bw[1]) >> (key & 31)) & 1u)) continue;
                  const float s = __uint_as_float(tmem_ld1(tH + key));
                  tmem_ld_wait();
                  const bool see = ((key < 32 ? vw[0] : vw[1]) >> (key & 31)) & 1u;
                  const float p = ex2f(fmaf(s, sl, negm));
#pragma unroll 1
                  for (int c = 0; c < HD; c += 16) {
                    uint32_t o[16];
                    tmem_ld16u(tO + c, o);
                    tmem_ld_wait();
                    const uint4 w[2] = {*chunk(vt, hf * 64 + key, c >> 3), *chunk(vt, hf * 64 + key, (c >> 3) + 1)};
                    const uint32_t* y = reinterpret_cast<const uint32_t*>(w);
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                      const uint32_t hbits = (e & 1) ? y[e >> 1] & 0xffff0000u : y[e >> 1] << 16;
                      if (see && (hbits & 0x7f800000u) == 0x7f800000u)
                        o[e] = __float_as_uint(fmaf(p, __uint_as_float(hbits), __uint_as_float(o[e])));
                    }
                    tmem_st16(tO + c, o);
                    tmem_st_wait();
                  }
                }
              }
              first_acc = 1u;
              ok = meet(fx, ph);  // every row has taken what it sees
              if (!ok) break;
              if (bad) clean_row(vt, vkey, c0, HD / 16);
              fence_proxy_async_smem();
            }
          }
          if (warp_live) {
            float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
            const float2 sl2 = make_float2(sl, sl), nm2 = make_float2(negm, negm);
#pragma unroll
            for (int c = 0; c < 2; ++c) {  // 32 keys
              uint32_t p16[16];
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                float2 p = fma2(make_float2(v[c * 32 + 2 * e], v[c * 32 + 2 * e + 1]), sl2, nm2);
                p.x = ex2f(p.x);
                p.y = ex2f(p.y);
                sum[e & 1] = add2(sum[e & 1], p);
                const __nv_bfloat162 h2 = __floats2bfloat162_rn(p.x, p.y);
                p16[e] = *reinterpret_cast<const uint32_t*>(&h2);
              }
              tmem_st16(tH + c * 16, p16);
            }
            Ls = fmaf(Ls, f, (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y));
            M = Mn;
            tmem_st_wait();
          }
          if (first && r == 0) acc_first[gq] = first_acc;
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&p_full[2 * gq + (job & 1)]);
          ++job;
          own += hf;
        }
        vjob += own;
        if (!ok) break;
        if (has && stop(wait_phase(&pv_done[2 * gq + (job - 1 & 1)], (uint32_t)(job - 1 >> 1) & 1u, abort_f, g))) break;
        // ---- the piece's end: group 0 joins both groups' parts of a single query tile, else each has its own
        float2 other = make_float2(-INFINITY, 0.f);
        if (!two) {
          if (gq == 1) {
            if (xn > 0 && stop(wait_phase(x_free, (uint32_t)(xn - 1) & 1u, abort_f, g))) break;
            xch[r] = make_float2(M, Ls);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(x_full);
          } else {
            if (stop(wait_phase(x_full, (uint32_t)xn & 1u, abort_f, g))) break;
            other = xch[r];
            __syncwarp();
            if (lane == 0) mbar_arrive(x_free);
          }
          ++xn;
        }
        if (two || gq == 0) {
          tc_fence_after();
          const float Mx = fmaxf(M, other.x);
          const float ref = Mx == -INFINITY ? 0.f : Mx;
          const float wa = M == -INFINITY ? (both ? 0.f : 1.f) : ex2f(M - ref);
          const float wb = other.x == -INFINITY ? 0.f : ex2f(other.x - ref);
          const float Lt = fmaf(wb, other.y, wa * Ls);
          const float inv = whole ? 1.f / Lt : 1.f;
          if (warp_live) {
            bf16* dst = out + (((long long)me.b * g.n + me.i) * g.nq + me.head) * HD;
            float* pdst = g.part_o + (pc.slot_row + rr) * HD;
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
                  for (int e = 0; e < 32; e += 8) store32(pdst + c + e, *reinterpret_cast<const uint32_t(*)[8]>(&x[e]));
                }
              }
            }
            if (me.live && !whole) g.part_ml[pc.slot_row + rr] = make_float2(both ? Mx : M, both ? Lt : Ls);
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&o_free[gq]);
            if (both) mbar_arrive(&o_free[1]);
          }
        }
        handover = true;
        if (two || qt == 0) ++qn0;
        if (two || qt == 1) ++qn1;
        if (!two) qt ^= 1;
        tiles += nt;
        done_piece(seg);
        ++seg;
        ok = wait_piece(seg);
      }
    }
    if constexpr (NR > 0) {
      while (ok && (dry || pieces[seg & 3].nt > 0)) {
        // ------------------------------------------------ rows as columns: thread = key r of the tile
        const Piece& pc = pieces[seg & 3];
        const int nt = dry ? 2 : pc.nt;
        const bool whole = pc.whole;
        const int rows = pc.rows, x0 = pc.x0, ahead = ahead_of(true);
        const bool has = gq < nt, both = nt > 1;
        float* ref = reinterpret_cast<float*>(sm + L::kRef) + gq * 64;
        uint8_t* pbuf = sm + L::kQ + gq * L::kQBuf + L::kP;
        float* scr = reinterpret_cast<float*>(pbuf);  // scratch wherever no product reads P
        auto to_scratch = [&](float (&x)[NR]) {  // a warp's results of warp_scatter, by row
          const int at = scatter_row<NR>(lane);
          if (NR >= 32) {
#pragma unroll
            for (int e = 0; e < NR / 32; ++e) scr[qr * NR + at + e] = x[e];
          } else if (!(lane & 1)) {
            scr[qr * NR + at] = x[0];
          }
        };
        constexpr bool kPair = NR <= 32;
        constexpr bool kRegRef = NR <= 32;      // (registers for the references too)
        float Ls[NR], nm[kRegRef ? NR : 2];     // row sums of this thread's keys; -M
#pragma unroll
        for (int c = 0; c < NR; ++c) Ls[c] = 0.f;
        if (!meet(&fix[gq], fn)) break;  // the scratch's last readers are past it
        for (int t = gq; ok && t < nt; t += 2) {  // (once when dry)
          const bool first = t == gq;
          const int k0 = pc.tile(t) * KT, key = k0 + r;
          const bool inner = dry || (k0 >= pc.all_lo && k0 + KT <= pc.all_hi);
          const int sb = job & 1;  // score buffer
          uint32_t& sn = sb ? sn1 : sn0;
          if (!dry && stop(wait_phase(&s_full[2 * gq + sb], sn & 1u, abort_f, g))) {
            ok = false;
            break;
          }
          sn += !dry;
          // the last product has read P and left O to be changed
          bool pv_waited = first;
          auto wait_pv = [&]() {
            if (!pv_waited) ok = !stop(wait_phase(&pv_done[2 * gq + (job - 1 & 1)], (uint32_t)(job - 1 >> 1) & 1u, abort_f, g));
            if (!pv_waited) tc_fence_after();
            pv_waited = true;
            return ok;
          };
          if (handover) {
            ok = (qn0 == 0 || !stop(wait_phase(&q_empty[0], (uint32_t)(qn0 - 1) & 1u, abort_f, g))) &&
                 (qn1 == 0 || !stop(wait_phase(&q_empty[1], (uint32_t)(qn1 - 1) & 1u, abort_f, g)));
            if (!ok) break;
            handover = false;
          }
          tc_fence_after();
          float v[NR];      // scores, then exponents s - M
          uint64_t hid = 0; // rows that do not see the key
          auto load_scores = [&]() {
#pragma unroll
            for (int c = 0; c < NR; c += 16) tmem_ld16u(tS + sb * 64 + c, *reinterpret_cast<uint32_t(*)[16]>(&v[c]));
            tmem_ld_wait();
            if (!inner) {
#pragma unroll
              for (int c = 0; c < NR; ++c)
                if ((hid >> c) & 1) v[c] = -INFINITY;
            }
          };
          auto exponents = [&]() {
#pragma unroll
            for (int c = 0; c < NR; c += 4) {
              float4 m;
              if constexpr (kRegRef)
                m = make_float4(nm[c], nm[c + 1], nm[c + 2], nm[c + 3]);
              else
                m = *reinterpret_cast<const float4*>(ref + c);
              const float2 x = fma2(make_float2(v[c], v[c + 1]), make_float2(sl, sl), make_float2(m.x, m.y));
              const float2 y = fma2(make_float2(v[c + 2], v[c + 3]), make_float2(sl, sl), make_float2(m.z, m.w));
              v[c] = x.x, v[c + 1] = x.y, v[c + 2] = y.x, v[c + 3] = y.y;
            }
          };
          if (!inner) {
            uint64_t see = 0u;
            if (key >= pc.key_lo && key < pc.key_end) {
              if (pc.prefix) {  // (a window over a prefix: the rows' sequences differ)
#pragma unroll 1
                for (int c = 0; c < rows; ++c) {
                  const ItemRow w = item_row(g, true, 0, pc.hk, x0, c);
                  int sink, lo, hi;
                  row_span(g, paged_len(g, w.b), paged_rows(g, w.b), w.i, sink, lo, hi);
                  if (key < sink || (key >= lo && key < hi)) see |= 1ull << c;
                }
              } else {
                // block row i sees the key from i = key - P on, until the window has moved past it
                const int d = key - pc.P;
                const bool out_of = g.window > 0 && key >= g.sinks;
                if (g.causal) {
                  const long long from = (long long)max(d, 0) * g.G - x0;
                  const long long to = out_of ? ((long long)d + g.window) * g.G - x0 : 64;
                  const int a = (int)min(from, 64ll), b = (int)max(min(to, 64ll), 0ll);
                  see = bits_of(a, b) | (uint64_t)bits_of(a - 32, b - 32) << 32;
                } else if (!out_of || d >= -g.window) {
                  see = ~0ull;
                }
              }
            }
            hid = ~see;
          }
          load_scores();
          // Whether a reference has to move is the group's vote.  Its answer is nearly always no, so with up to
          // 32 rows the weights are computed while the votes come in (with 64 their sums would need registers
          // that are not there).
          volatile uint32_t* votes = vote_w + (sb * 2 + gq) * 4;  // (two sets: a warp may be a tile ahead)
          uint32_t hi[NR / 2], lo[NR == 16 ? NR / 2 : 1];
          auto add_sum = [&](int c) {
            const float2 l = add2(make_float2(Ls[c], Ls[c + 1]), make_float2(v[c], v[c + 1]));
            Ls[c] = l.x;
            Ls[c + 1] = l.y;
          };
          auto weights = [&]() {
#pragma unroll
            for (int c = 0; c < NR; c += 2) {
              v[c] = ex2f(v[c]);
              v[c + 1] = ex2f(v[c + 1]);
              if constexpr (!kRegRef) add_sum(c);
              if constexpr (NR == 16) {
                pack_bf16_hilo(v[c], v[c + 1], hi[c / 2], lo[c / 2]);
              } else if constexpr (!kPair) {
                const __nv_bfloat162 h2 = __floats2bfloat162_rn(v[c], v[c + 1]);
                hi[c / 2] = *reinterpret_cast<const uint32_t*>(&h2);
              }
            }
          };
          bool move = first;
          if (!first) {
            exponents();
            float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
            for (int c = 0; c < NR; c += 4) {
              top[0] = max3(top[0], v[c], v[c + 1]);
              top[1] = max3(top[1], v[c + 2], v[c + 3]);
            }
            const uint32_t over = __any_sync(0xffffffffu, fmaxf(top[0], top[1]) > 8.f);
            if (lane == 0) {
              votes[qr] = over;
              mbar_arrive(&fix[gq]);
            }
            if constexpr (kRegRef) weights();
            ok = !stop(wait_phase(&fix[gq], (uint32_t)fn & 1u, abort_f, g));
            ++fn;
            if (!ok) break;
            move = votes[0] | votes[1] | votes[2] | votes[3];
          }
          if (move) {
            // each row's largest score of the tile (a NaN sets no reference)
            if (!wait_pv()) break;
            if (!first) load_scores();  // (v holds weights)
            warp_scatter<NR, true>(v, lane);
            to_scratch(v);
            ok = meet(&fix[gq], fn);
            if (!ok) break;
            if (r < NR) {
              const float mx = fmaxf(fmaxf(scr[r], scr[NR + r]), fmaxf(scr[2 * NR + r], scr[3 * NR + r]));
              const float old = first ? kNoRef : ref[r];
              float nm = old, f = 1.f;
              if (mx != -INFINITY) {
                const float mt = mx * sl;
                if (old == kNoRef) {
                  nm = -mt;
                } else if (mt + old > 8.f) {
                  nm = -mt;
                  f = ex2f(-old - mt);
                }
              }
              ref[r] = nm;
              scr[4 * NR + r] = f;
            }
            ok = meet(&fix[gq], fn);
            if (!ok) break;
            if (!first) {
#pragma unroll
              for (int c = 0; c < NR; ++c) Ls[c] *= scr[4 * NR + c];
#pragma unroll 1
              for (int c = 0; c < (kPair ? 2 * NR : NR); c += 16) {
                uint32_t o[16];
                tmem_ld16u(tO + c, o);
                tmem_ld_wait();
#pragma unroll
                for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * scr[4 * NR + (c + e) % NR]);
                tmem_st16(tO + c, o);
              }
              tmem_st_wait();
              ok = meet(&fix[gq], fn);  // P overwrites the factors
              if (!ok) break;
            }
            if constexpr (kRegRef) {
#pragma unroll
              for (int c = 0; c < NR; c += 4) {
                const float4 m = *reinterpret_cast<const float4*>(ref + c);
                nm[c] = m.x, nm[c + 1] = m.y, nm[c + 2] = m.z, nm[c + 3] = m.w;
              }
            }
            load_scores();
            exponents();
            if constexpr (kRegRef) weights();
          }
          uint32_t first_acc = 0u;
          if (!inner) {
            uint8_t* vt = sm + (2 * tiles + v_at(t, ahead, nt)) % NS * L::kTile;
            // (the last product's values had landed: this wait cannot take their phase for its own)
            if (!wait_pv()) break;
            ok = !stop(wait_phase(&v_ready[gq], (uint32_t)vjob & 1u, abort_f, g));
            if (!ok) break;
            const bool bad = row_is_bad(vt, r, 0, HD / 8);
            const uint32_t word = __ballot_sync(0xffffffffu, bad);
            if (lane == 0) bad_w[gq * 4 + qr] = word;
            ok = meet(&fix[gq], fn);
            if (!ok) break;
            const uint32_t bw[4] = {bad_w[gq * 4], bad_w[gq * 4 + 1], bad_w[gq * 4 + 2], bad_w[gq * 4 + 3]};
            if (bw[0] | bw[1] | bw[2] | bw[3]) {
              if (first) {
                const uint32_t on = o_uses[gq];
                if (on > 0) ok = !stop(wait_phase(&o_free[gq], (on - 1) & 1u, abort_f, g));
                if (!ok) break;
                tc_fence_after();
                zero_o(64);
              }
              first_acc = 1u;
#pragma unroll 1
              for (int k = 0; ok && k < KT; ++k) {
                const uint32_t w = k < 64 ? (k < 32 ? bw[0] : bw[1]) : (k < 96 ? bw[2] : bw[3]);
                if (!((w >> (k & 31)) & 1u)) continue;
                if (k == r) {
#pragma unroll
                  for (int c = 0; c < NR; ++c) scr[c] = (hid >> c) & 1 ? -1.f : kRegRef ? v[c] : ex2f(v[c]);
                }
                ok = meet(&fix[gq], fn);
                if (!ok) break;
                const int d = r < HD ? r : 0;  // this lane's dimension
                const uint32_t raw = reinterpret_cast<const uint16_t*>(chunk(vt, k, d >> 3))[d & 7];
                const float val = __uint_as_float(raw << 16);
                const bool add = (raw & 0x7f80u) == 0x7f80u;
#pragma unroll 1
                for (int c = 0; c < NR; c += 16) {
                  uint32_t o[16];
                  tmem_ld16u(tO + c, o);
                  tmem_ld_wait();
#pragma unroll
                  for (int e = 0; e < 16; ++e) {
                    const float p = scr[c + e];
                    if (add && !(p < 0.f)) o[e] = __float_as_uint(fmaf(p, val, __uint_as_float(o[e])));
                  }
                  tmem_st16(tO + c, o);
                  tmem_st_wait();
                }
                ok = meet(&fix[gq], fn);
              }
              if (!ok) break;
              if (bad) clean_row(vt, r, 0, HD / 8);
            }
          }
          // this key's row of P: a bf16 a row of the item (pairs: the low parts behind the high ones)
          if constexpr (kRegRef) {
#pragma unroll
            for (int c = 0; c < NR; c += 2) add_sum(c);
          } else {
            weights();
          }
          if (!wait_pv()) break;
          {
            uint8_t* prow = pbuf + r * 128;
#pragma unroll
            for (int c = 0; c < NR / 8; ++c) {
              if constexpr (NR == 32) {  // (both parts only here: registers)
                uint32_t h[4], l[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) pack_bf16_hilo(v[8 * c + 2 * e], v[8 * c + 2 * e + 1], h[e], l[e]);
                *reinterpret_cast<uint4*>(prow + ((c ^ (r & 7)) << 4)) = make_uint4(h[0], h[1], h[2], h[3]);
                *reinterpret_cast<uint4*>(prow + ((c + 4 ^ (r & 7)) << 4)) = make_uint4(l[0], l[1], l[2], l[3]);
                continue;
              }
              *reinterpret_cast<uint4*>(prow + ((c ^ (r & 7)) << 4)) =
                  make_uint4(hi[4 * c], hi[4 * c + 1], hi[4 * c + 2], hi[4 * c + 3]);
              if constexpr (NR == 16)
                *reinterpret_cast<uint4*>(prow + ((c + NR / 8 ^ (r & 7)) << 4)) =
                    make_uint4(lo[4 * c], lo[4 * c + 1], lo[4 * c + 2], lo[4 * c + 3]);
            }
          }
          fence_proxy_async_smem();
          if (first && !dry && r == 0) acc_first[gq] = first_acc;
          tc_fence_before();
          __syncwarp();
          if (dry) break;
          if (lane == 0) mbar_arrive(&p_full[2 * gq + (job & 1)]);
          ++job;
          ++vjob;
        }
        if (!ok) break;
        if (dry) {
          dry = 0;
          pdl_wait();
          ok = wait_piece(0);
          continue;
        }
        // ---- the piece's end: row sums over the group, then group 0 joins both groups' parts
        float M = -INFINITY, Lr = 0.f;  // of row r (threads below NR)
        if (has) {
          if (stop(wait_phase(&pv_done[2 * gq + (job - 1 & 1)], (uint32_t)(job - 1 >> 1) & 1u, abort_f, g))) break;
          warp_scatter<NR, false>(Ls, lane);
          to_scratch(Ls);
          if (!meet(&fix[gq], fn)) break;
          if (r < NR) {
            M = ref[r] == kNoRef ? -INFINITY : -ref[r];
            Lr = (scr[r] + scr[NR + r]) + (scr[2 * NR + r] + scr[3 * NR + r]);
          }
        }
        float2 other = make_float2(-INFINITY, 0.f);
        if (gq == 1) {
          if (xn > 0 && stop(wait_phase(x_free, (uint32_t)(xn - 1) & 1u, abort_f, g))) break;
          if (r < NR) xch[r] = make_float2(M, Lr);
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(x_full);
        } else {
          if (stop(wait_phase(x_full, (uint32_t)xn & 1u, abort_f, g))) break;
          if (r < NR) other = xch[r];
          __syncwarp();
          if (lane == 0) mbar_arrive(x_free);
        }
        ++xn;
        if (gq == 0) {
          float2* coef = reinterpret_cast<float2*>(scr + 8 * NR);
          const long long prow = pc.slot_row;
          if (r < NR) {
            const float Mx = fmaxf(M, other.x), ref0 = Mx == -INFINITY ? 0.f : Mx;
            const float wa = M == -INFINITY ? (both ? 0.f : 1.f) : ex2f(M - ref0);
            const float wb = other.x == -INFINITY ? 0.f : ex2f(other.x - ref0);
            const float Lt = fmaf(wb, other.y, wa * Lr);
            const float inv = whole ? 1.f / Lt : 1.f;
            coef[r] = make_float2(wa * inv, wb * inv);
            if (!whole && r < rows) g.part_ml[prow + r] = make_float2(Mx, Lt);
          }
          if (!meet(&fix[gq], fn)) break;
          tc_fence_after();
          if (qr * 32 < HD) {  // this lane's dimension is r
            const int f = div_g(g, x0);  // block row (of the sequence or of the batch)
            int h = x0 - f * g.G;
            bf16* dst = out + ((long long)((pc.prefix ? 0 : pc.b * g.n) + f) * g.nq + pc.hk * g.G + h) * HD + r;
            float* pdst = g.part_o + prow * HD + r;
            const long long skip = (long long)(g.nq - g.G) * HD;  // to the next block row's heads
#pragma unroll 1
            for (int c0 = 0; c0 < rows; c0 += 16) {
              uint32_t a[16], a2[16], b[16], b2[16];
              tmem_ld16u(tO + c0, a);
              if (kPair) tmem_ld16u(tO + NR + c0, a2);
              if (both) {
                tmem_ld16u(tO + 128 + c0, b);
                if (kPair) tmem_ld16u(tO + 128 + NR + c0, b2);
              }
              tmem_ld_wait();
#pragma unroll
              for (int c = 0; c < 16; ++c) {
                const float2 w = coef[c0 + c];
                float x = __uint_as_float(a[c]), xb = both ? __uint_as_float(b[c]) : 0.f;
                if (kPair) {
                  // (the high parts' sum is infinite where an infinite value is seen; its product with a low part
                  // of 0 or below would be NaN)
                  if (!isinf(x)) x += __uint_as_float(a2[c]);
                  if (both && !isinf(xb)) xb += __uint_as_float(b2[c]);
                }
                x *= w.x;
                if (both) x = fmaf(w.y, xb, x);
                if (c0 + c < rows) {
                  if (whole)
                    *dst = __float2bfloat16_rn(x);
                  else
                    *pdst = x;
                }
                dst += HD;
                pdst += HD;
                if (++h == g.G) {
                  h = 0;
                  dst += skip;
                }
              }
            }
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&o_free[0]);
            if (both) mbar_arrive(&o_free[1]);
          }
          if (NR == 16 && !whole && pc.nc > 0 && !join(pc)) break;  // (few rows; else a kernel does)
        }
        if (qt == 0)
          ++qn0;
        else
          ++qn1;
        qt ^= 1;
        tiles += nt;
        done_piece(seg);
        ++seg;
        ok = wait_piece(seg);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 3) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

PagedRule paged_rule_tc(const PagedGeom& g) {
  // Items of two query tiles where there are rows for them.
  const int ri = g.n * g.G > 128 ? 256 : 128, rp = g.batch * g.n * g.G > 128 ? 256 : 128;
  // A tile takes two positions of the line, an item's start and end the time of two tiles more: with 0 instead,
  // 8 prompts' first 128 rows take 36.0 us (28.0 so), 64 tokens behind a common 12K 119 (107), 128 rows behind
  // 36K 130 (126); only a window's pieces (15 rows, 34 tiles an item) lose, 80.7 (82.9).
  return PagedRule{ri, rp, kPagedTcKeys, 2, 4};
}

template <int HD, int NR, bool TS, bool TP>
static cudaError_t tc_launch(PagedGeom g, const CUtensorMap& tk, const CUtensorMap& tv, long long pool_rows,
                             const void* q, void* out, long long part_rows, cudaStream_t s) {
  typedef TcLayout<HD> L;
  static PerDevice smem;
  DFL_RET(smem.once([] {
    return cudaFuncSetAttribute(paged_attn_tc_kernel<HD, NR, TS, TP>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                L::kSmem);
  }));
  if (paged_split(g, paged_rule_tc(g), num_sms(), 2) > part_rows) return cudaErrorInvalidValue;
  const float scale_log2 = 1.4426950408889634f / sqrtf((float)HD);
  DFL_RET(launch_pdl(paged_attn_tc_kernel<HD, NR, TS, TP>, dim3(g.grid), dim3(kTcThreads), L::kSmem, s, tk, tv, g,
                     (int)pool_rows, (const bf16*)q, (bf16*)out, scale_log2));
  count_launch();
  if (g.shared) return paged_merge_bf16(HD, g, out, s);
  // The CTAs join their pieces where an item has up to 16 rows; beyond, one CTA's threads would take longer than a
  // kernel over all items (8 blocks of 16 rows over 2K..6K keys: 75 us instead of 61).
  return NR == 16 ? cudaSuccess : paged_join_bf16(HD, g, out, s);
}

template <int HD>
static cudaError_t tc_pick(const PagedGeom& g, const CUtensorMap& tk, const CUtensorMap& tv, long long pool_rows,
                           const void* q, void* out, long long part_rows, cudaStream_t s) {
  const int ns = g.n * g.G, np = g.shared ? g.batch * ns : ns;  // stacked rows of a sequence, of a shared prefix
#define DFL_TC(NR, TS, TP) return tc_launch<HD, NR, TS, TP>(g, tk, tv, pool_rows, q, out, part_rows, s)
  if (ns > 64) DFL_TC(0, false, false);
  if (ns > 32) {
    if (np > 64) DFL_TC(64, true, false);
    DFL_TC(64, true, true);
  }
  if (ns > 16) {
    if (np > 32) DFL_TC(32, true, false);
    DFL_TC(32, true, true);
  }
  if (np > 16) DFL_TC(16, true, false);
  DFL_TC(16, true, true);
#undef DFL_TC
}

cudaError_t paged_attention_tc(int hd, const PagedGeom& g, const CUtensorMap& tk, const CUtensorMap& tv,
                               long long pool_rows, const void* q, void* out, long long part_rows, cudaStream_t s) {
  return hd == 64 ? tc_pick<64>(g, tk, tv, pool_rows, q, out, part_rows, s)
                  : tc_pick<128>(g, tk, tv, pool_rows, q, out, part_rows, s);
}

}  // namespace dfl
