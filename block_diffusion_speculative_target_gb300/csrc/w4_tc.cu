// Products with 4-bit weights on the 5th-generation tensor cores.
//
// y[n][m] = sum over groups of s[m][g] * sum_{k in g} (code[m][k] - zero[m][g]) x[n][k]
//
// Codes less zero points are integers of at most 15, exact in bf16, and so are
// their products with x in float32.  A group's sum is taken by the tensor cores in
// an accumulator of its own, D; then acc += s D in float32.  Weights are the
// products' 128 rows, read from TMEM; rows of x their columns, in shared memory.
//
// A code pair becomes two bf16 in one register without a conversion.  Eight bits
// v at the low end of a bf16 are the number v 2^-133, below the normal numbers and
// just into them; so the low or the high half of a byte, masked out and multiplied
// by 2^127 or 2^123, less zero / 64, is (code - zero) / 64 exactly: one mask and
// one packed multiply-add a pair, one shift for every other byte.  (The integer
// pipe has half the lanes of the others: with a shift for every pair it was the
// bound.)  The results take the factor of 64 back.  The codes lie in memory in the
// order in which a warp's 16 by 16 matrix fragments hold them, which is also the
// order of a TMEM store of 128-bit rows: a lane reads 32 of its own codes with one
// 16-byte load and nothing is shuffled.
//
// Split: the blocks of 128 by 128 of the whole matrix form a line (row blocks
// one after another), cut into equal runs, one to a CTA and a CTA to an SM, whatever
// M and K are.  A row block that lies in several runs leaves a partial sum in each;
// who ends the last one adds them in order of the columns.  The cut depends on M, K
// and the GPU only, and no sum on the other rows of x: a row has the same bits alone
// and in a block.
//
// Warps: 0 streams the blocks (codes with their scales and zero points, one bulk
// copy each) through a ring; 1 issues the products; 2 brings the columns of x that a
// block meets by TMA, or, where rows of x do not lie on 16-byte boundaries, 2 and 3 do
// by hand; 4..7 read the sums back, scale, add, join and write; 8..11 and
// 12..15 expand every other block's codes into one of four TMEM buffers.
//
// Measured: 128 rows of 4096 x 12288, groups of 64, zero points, a residual added,
// 48 us (266 TFLOP/s; 33 MB at 0.7 TB/s); without zero points in groups of 128 and
// without the residual 33. Bound by latency, tensor pipe 15% and issue slots 27%
// taken: a CTA's 21 blocks go one after another from codes to TMEM to products
// to sums, and the CTA that ends a row block joins up to 6 pieces of 128 x 128 alone.
//
// Every wait is bounded (dflash_debug_set_wait_limit); one that runs out sets
// DFLASH_STATUS_TIMEOUT, the CTA stops, drains its copies and products, whatever the
// limit, and leaves without a result.
#include <algorithm>

#include "common.cuh"
#include "internal.h"
#include "w4.cuh"
#include "w4_ops.cuh"

namespace dfl {

namespace {
constexpr int kThreads = 512;
constexpr int kXWarps = 2;
constexpr int kABufs = 4;        // buffers of expanded weights, 64 TMEM columns each
constexpr int kDColumns = 256;   // TMEM columns of sums: at least two buffers
constexpr int kMaxD = 16;

// N: columns of a product (rows of x, padded).
template <int N>
struct TcLayout {
  static constexpr int kX = N * 256;  // two halves of 64 columns: rows of 128 bytes, 16-byte chunks swizzled by row
  static constexpr int kXSlots = N <= 64 ? 6 : 3;
  static constexpr int kCodeSlots = 10;
  static constexpr int kBars = 2 * kCodeSlots + 2 * kXSlots + 2 * kABufs + 2 * kMaxD + 1;
};

// Two float32 lanes at once.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(reinterpret_cast<uint64_t&>(d))
      : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)), "l"(reinterpret_cast<uint64_t&>(c)));
  return d;
}
// 16 lanes of 64 columns: registers 4 s + {0, 1, 2, 3} of lane 4 g + t are, of columns 8 s .. 8 s + 7, (row g, column
// t), (row g + 8, t), (g, 4 + t), (g + 8, 4 + t).
__device__ __forceinline__ void tmem_st_16x128b_x16(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x128b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
      "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
}  // namespace

// How TMEM holds the sums.
struct W4Sums {
  int group_shift;        // log2(group / 32)
  int part_shift;         // log2 of the parts of a block whose sums are read back together
  int buffers;            // of a part's sums in TMEM
};

// One CTA: run blockIdx.x.
template <int N>
__global__ void __launch_bounds__(kThreads, 1)
    w4_tc_kernel(const __grid_constant__ W4View w, const __grid_constant__ W4Run run,
                 const __grid_constant__ W4Sums sums, const __grid_constant__ CUtensorMap tmx,
                 const bf16* __restrict__ x, long long ldx, int vec, int rows, const __grid_constant__ W4Epi epi) {
  typedef TcLayout<N> L;
  constexpr int V = N / 4;  // float4 of sums a thread
  constexpr int CS = L::kCodeSlots, XS = L::kXSlots;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t bars[L::kBars];
  __shared__ uint32_t tmem_slot;
  __shared__ volatile int abort_s;
  __shared__ float sums_s[4][16 * kW4SumRow];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* code_full = bars;              // [CS] a block has landed
  uint64_t* code_empty = bars + CS;        // [CS] its four expanding and its four adding warps are done with it
  uint64_t* x_full = code_empty + CS;      // [XS] both warps' columns of x are there
  uint64_t* x_empty = x_full + XS;         // [XS] read by the block's products
  uint64_t* a_full = x_empty + XS;         // [4] four warps have expanded a block
  uint64_t* a_empty = a_full + kABufs;     // [4] read by its products
  uint64_t* d_full = a_empty + kABufs;     // [nd] sums are there
  uint64_t* d_empty = d_full + kMaxD;      // [nd] and have been read (four warps)
  uint64_t* drain = d_empty + kMaxD;       // every product is done
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int b0 = blockIdx.x * run.per, b1 = min(b0 + run.per, run.blocks);
  uint8_t* codes = smem + XS * L::kX;
  // groups of a part, its columns, and how many parts' sums TMEM holds
  const int gs = sums.group_shift, groups = 4 >> gs, part_groups = groups >> sums.part_shift;
  const int part_columns = N * part_groups, nd = sums.buffers, parts = 1 << sums.part_shift;
  const int fresh = (1 << gs) - 1;  // 32-column steps q with (q & fresh) == 0 begin a group
  if (tid == 0) {
    for (int i = 0; i < CS; ++i) {
      mbar_init(&code_full[i], 1);
      mbar_init(&code_empty[i], 8);
    }
    for (int i = 0; i < XS; ++i) {
      mbar_init(&x_full[i], vec ? 1 : kXWarps);
      mbar_init(&x_empty[i], 1);
    }
    for (int i = 0; i < kABufs; ++i) {
      mbar_init(&a_full[i], 4);
      mbar_init(&a_empty[i], 1);
    }
    for (int i = 0; i < kMaxD; ++i) {
      mbar_init(&d_full[i], 1);
      mbar_init(&d_empty[i], 4);
    }
    mbar_init(drain, 1);
    abort_s = 0;
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(&tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot, tD = tmem + 64 * kABufs;
  pdl_launch();
  // Waits for a phase, giving up on the CTA's abort flag or after the limit (then raising the flag).  A warp's lanes
  // wait together and agree.
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    if (run.wait_ns > 0 && __all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
    bool ok = false;
    if (run.wait_ns > 0) {
      const uint64_t t0 = global_ns();
      while (true) {
#pragma unroll 1
        for (int i = 0; i < 64 && !ok; ++i) ok = mbar_try_wait(bar, parity);
        if (ok || abort_s || global_ns() - t0 > run.wait_ns) break;
      }
    }
    if (__any_sync(0xffffffffu, !ok)) {
      if (lane == 0) {
        if (!abort_s) set_status(run.status, DFLASH_STATUS_TIMEOUT);
        abort_s = 1;
      }
      return false;
    }
    return true;
  };

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    if (warp == 0) {
      // ---------------------------------------------------------- blocks
      // The weights do not depend on the kernels before this one (packing lets no successor start early, and has
      // published its stores by its end): they are asked for without waiting for them.
      const uint8_t* src = w.packed + (long long)b0 * w.block_bytes;
      int slot = 0;
      uint32_t phase = 0;
      int i = b0;
      for (; i < b1; ++i) {
        if (i - b0 >= CS && !wait(&code_empty[slot], phase ^ 1u)) break;
        if (elect_one()) {
          mbar_arrive_expect_tx(&code_full[slot], w.block_bytes);
          bulk_load(codes + (size_t)slot * w.block_bytes, src, w.block_bytes, &code_full[slot]);
        }
        __syncwarp();
        src += w.block_bytes;
        if (++slot == CS) {
          slot = 0;
          phase ^= 1u;
        }
      }
      // every copy asked for lands before the CTA ends, whichever warp gives up, and when
      const int asked = i - b0;
      for (int u = max(0, asked - CS); u < asked; ++u) mbar_wait(&code_full[u % CS], (uint32_t)(u / CS) & 1u, kW4DrainNs);
    } else if (warp == 1) {
      // ---------------------------------------------------------- products
      constexpr uint32_t idesc = idesc_bf16_f32(128, N);
      const int quarters = 4 >> sums.part_shift;  // steps of 32 columns in a part
      int xs = 0, ab = 0, db = 0;
      uint32_t xp = 0, ap = 0, dp = 0;
      bool ok = true, first_d = true;
      for (int i = b0; i < b1 && ok; ++i) {
        ok = wait(&x_full[xs], xp) && wait(&a_full[ab], ap);
        const uint64_t xd = smem_desc_sw128(smem + xs * L::kX);
        for (int p = 0; p < parts && ok; ++p) {
          if (!first_d && !(ok = wait(&d_empty[db], dp ^ 1u))) break;
          tc_fence_after();
          if (elect_one()) {
            const uint32_t d = tD + db * part_columns;
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              if (u >= quarters) break;
              const int q = p * quarters + u;
              const uint32_t to = d + (u >> gs) * N, from = tmem + 64 * ab + 16 * q;
              const uint64_t b = xd + (uint64_t)((q >> 1) * (N * 128 / 16) + 4 * (q & 1));
              tc_mma_f16_tmem_a(to, from, b, idesc, (q & fresh) != 0);
              tc_mma_f16_tmem_a(to, from + 8, b + 2, idesc, 1u);
            }
            tc_commit(&d_full[db]);
            if (p == parts - 1) {
              tc_commit(&a_empty[ab]);
              tc_commit(&x_empty[xs]);
            }
          }
          __syncwarp();
          if (++db == nd) {
            db = 0;
            dp ^= 1u;
            first_d = false;
          }
        }
        if (++xs == XS) {
          xs = 0;
          xp ^= 1u;
        }
        if (++ab == kABufs) {
          ab = 0;
          ap ^= 1u;
        }
      }
      if (elect_one()) tc_commit(drain);
      __syncwarp();
      mbar_wait(drain, 0, kW4DrainNs);
    } else if (vec) {
      // ---------------------------------------------------------- x in wide rows: two boxes of 64 columns a block
      // (columns past K and rows past the last one arrive as zeros)
      if (warp == 2) {
        int kb = b0 % w.kt, slot = 0, i = b0;
        uint32_t phase = 0;
        if (elect_one()) tma_prefetch_desc(&tmx);
        __syncwarp();
        pdl_wait();
        for (; i < b1; ++i) {
          if (i - b0 >= XS && !wait(&x_empty[slot], phase ^ 1u)) break;
          if (elect_one()) {
            uint8_t* to = smem + slot * L::kX;
            mbar_arrive_expect_tx(&x_full[slot], L::kX);
            tma_load_2d(to, &tmx, &x_full[slot], kb * kW4Tile, 0);
            tma_load_2d(to + L::kX / 2, &tmx, &x_full[slot], kb * kW4Tile + 64, 0);
          }
          __syncwarp();
          if (++slot == XS) {
            slot = 0;
            phase ^= 1u;
          }
          if (++kb == w.kt) kb = 0;
        }
        const int asked = i - b0;
        for (int u = max(0, asked - XS); u < asked; ++u) mbar_wait(&x_full[u % XS], (uint32_t)(u / XS) & 1u, kW4DrainNs);
      }
    } else {
      // ---------------------------------------------------------- x anywhere
      // Lane l of warp 2 + v brings chunk l % 16 (8 columns) of the rows 2 v + l / 16 + 4 u.  Rows past the last one
      // are not filled: their columns of the products are not read.
      const int xc = lane & 15, xr = 2 * (warp - 2) + (lane >> 4);
      int kb = b0 % w.kt, slot = 0;
      uint32_t phase = 0;
      pdl_wait();
      const bf16* src0 = x + (long long)xr * ldx + 8 * xc;
      const uint32_t at0 = (uint32_t)((xc >> 3) * (N * 128) + xr * 128);
      for (int i = b0; i < b1; ++i) {
        if (i - b0 >= XS && !wait(&x_empty[slot], phase ^ 1u)) break;
        const bool in_k = kb * kW4Tile + 8 * xc < w.K;
        const bf16* src = src0 + kb * kW4Tile;
        const uint32_t at = slot * L::kX + at0;
#pragma unroll 4
        for (int u = 0; u < N / 4; ++u) {
          if (xr + 4 * u >= rows) break;
          const uint32_t dst = at + u * 512 + 16 * ((xc & 7) ^ ((xr + 4 * u) & 7));
          const bf16* p = in_k ? src + (long long)(4 * u) * ldx : x;
          *reinterpret_cast<uint4*>(smem + dst) = gather8(p, in_k);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&x_full[slot]);
        if (++slot == XS) {
          slot = 0;
          phase ^= 1u;
        }
        if (++kb == w.kt) kb = 0;
      }
    }
  } else if (warp < 8) {
    // ------------------------------------------------------------ sums
    asm volatile("setmaxnreg.inc.sync.aligned.u32 224;");
    const int r = tid - 128;  // this thread's row of the block
    const uint32_t lanes = (uint32_t)(32 * (warp - 4)) << 16;
    alignas(8) float acc[V][4];
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[v][e] = 0.f;
    int mt = b0 / w.kt, kb = b0 - mt * w.kt, cs = 0, db = 0;
    uint32_t cp = 0, dp = 0;
    pdl_wait();
    for (int i = b0; i < b1; ++i) {
      bool ok = wait(&code_full[cs], cp);  // (the scales are there)
      const uint8_t* scales = codes + (size_t)cs * w.block_bytes + kW4Codes;
      for (int p = 0; p < parts && ok; ++p) {
        if (!(ok = wait(&d_full[db], dp))) break;
        tc_fence_after();
        for (int gp = 0; gp < part_groups; ++gp) {
          const int at = (p * part_groups + gp) * kW4Tile + r;
          const float s = w.scale_f32 ? reinterpret_cast<const float*>(scales)[at]
                                      : to_f<bf16>(reinterpret_cast<const bf16*>(scales)[at]);
          const uint32_t src = tD + db * part_columns + gp * N + lanes;
          constexpr int kRead = N < 64 ? 32 : 64;  // columns read at once
#pragma unroll
          for (int c = 0; c < N; c += kRead) {
            uint32_t d[kRead / 32][32];
#pragma unroll
            for (int h = 0; h < kRead / 32; ++h) tmem_ld32(src + c + 32 * h, d[h]);
            tmem_ld_wait();
#pragma unroll
            for (int n = 0; n < kRead; n += 2) {
              float2& y = *reinterpret_cast<float2*>(&acc[(c + n) / 4][n % 4]);
              y = fma2(make_float2(s, s),
                       make_float2(__uint_as_float(d[n / 32][n % 32]), __uint_as_float(d[n / 32][n % 32 + 1])), y);
            }
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&d_empty[db]);
        if (++db == nd) {
          db = 0;
          dp ^= 1u;
        }
      }
      if (!ok) break;
      __syncwarp();
      if (lane == 0) mbar_arrive(&code_empty[cs]);
      if (++cs == CS) {
        cs = 0;
        cp ^= 1u;
      }
      const int tile = mt;
      const bool tile_end = ++kb == w.kt;
      if (tile_end) {
        kb = 0;
        ++mt;
      }
      if (!tile_end && i + 1 < b1) continue;
      // The row block ends here, or the run does.  A warp deals with its 32 rows by itself.
      w4_join<V, 4>(w, run, tile, r, acc, [&](int v0, const float (&sum)[4][4]) {
        if (4 * v0 >= rows) return;
        // what is added to the later rows comes closer meanwhile
        if (epi.add && v0 == 0 && tile * kW4Tile + r - lane < w.M)
          for (int n = 16 + lane; n < rows; n += 32) l2_prefetch(epi.add + (long long)n * w.M + tile * kW4Tile + r - lane);
        float* sums = sums_s[warp - 4];  // 16 columns at a time
#pragma unroll
        for (int n = 0; n < 16; ++n) sums[n * kW4SumRow + lane] = sum[n / 4][n % 4];
        __syncwarp();
        w4_results(w, epi, tile * kW4Tile + r - lane, sums, 4 * v0, min(16, rows - 4 * v0));
        __syncwarp();
      });
#pragma unroll
      for (int v = 0; v < V; ++v)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[v][e] = 0.f;
    }
  } else {
    // ------------------------------------------------------------ codes to bf16
    asm volatile("setmaxnreg.dec.sync.aligned.u32 104;");
    const int wg = (warp - 8) >> 2, wq = warp & 3, g = lane >> 2;
    const int zero_at = kW4Codes + groups * kW4Tile * (w.scale_f32 ? 4 : 2);
    int cs = wg, ab = wg;
    uint32_t cp = 0, ap = 0;
    for (int i = b0 + wg; i < b1; i += 2) {
      if (!wait(&code_full[cs], cp)) break;
      const uint8_t* blk = codes + (size_t)cs * w.block_bytes;
      uint4 word[2][2];
#pragma unroll
      for (int y = 0; y < 4; ++y)
        word[y >> 1][y & 1] = *reinterpret_cast<const uint4*>(blk + w4_word_at(2 * wq + (y >> 1), y & 1, lane));
      if (i - b0 >= kABufs && !wait(&a_empty[ab], ap ^ 1u)) break;
      tc_fence_after();
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        uint32_t a[32];
        uint32_t off0 = offset_of(kW4Zero), off1 = off0;
#pragma unroll
        for (int q = 0; q < 4; ++q) {  // 32 columns: steps 2 q and 2 q + 1
          if (w.zeros && (q & fresh) == 0) {
            const uint8_t* z = blk + zero_at + (q >> gs) * kW4Tile + 32 * wq + 16 * y + g;
            off0 = offset_of(z[0]);
            off1 = offset_of(z[8]);
          }
          const uint4 v = word[y][q >> 1];
          const uint32_t lo = q & 1 ? v.y : v.x, hi = q & 1 ? v.w : v.z;
          a[8 * q] = pair_of<0>(lo, off0);
          a[8 * q + 1] = pair_of<0>(hi, off1);
          a[8 * q + 2] = pair_of<1>(lo, off0);
          a[8 * q + 3] = pair_of<1>(hi, off1);
          a[8 * q + 4] = pair_of<0>(lo >> 8, off0);
          a[8 * q + 5] = pair_of<0>(hi >> 8, off1);
          a[8 * q + 6] = pair_of<1>(lo >> 8, off0);
          a[8 * q + 7] = pair_of<1>(hi >> 8, off1);
        }
        tmem_st_16x128b_x16(tmem + 64 * ab + ((uint32_t)(32 * wq + 16 * y) << 16), a);
      }
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&a_full[ab]);
        mbar_arrive(&code_empty[cs]);
      }
      cs += 2;
      if (cs >= CS) {
        cs -= CS;
        cp ^= 1u;
      }
      ab += 2;
      if (ab >= kABufs) {
        ab -= kABufs;
        ap ^= 1u;
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

namespace {
template <int N>
cudaError_t tc_launch(const W4View& w, const bf16* x, long long ldx, int rows, const W4Epi& epi, const W4Scratch& sc,
                      cudaStream_t s) {
  typedef TcLayout<N> L;
  static PerDevice attr;
  // (the widest block: groups of 32, float32 scales and zero points)
  constexpr int kMost = 1024 + L::kCodeSlots * (kW4Codes + 4 * kW4Tile * 5) + L::kXSlots * L::kX;
  static_assert(kMost <= 232448 - 12288, "shared memory per block");
  static_assert(L::kCodeSlots % 2 == 0, "two groups take every other block");
  DFL_RET(attr.once([] {
    return cudaFuncSetAttribute(w4_tc_kernel<N>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMost);
  }));
  const int vec = (reinterpret_cast<uintptr_t>(x) & 15) == 0 && ldx % 8 == 0;
  CUtensorMap tmx = {};
  if (vec && !make_rows_map(x, rows, w.K, ldx, N, &tmx)) return cudaErrorInvalidValue;
  const W4Run run = w4_run(w, sc, rows);
  W4Sums sums;
  sums.group_shift = w.group == 32 ? 0 : w.group == 64 ? 1 : 2;
  sums.part_shift = 0;
  while (N * w.groups() >> sums.part_shift > kDColumns / 2) ++sums.part_shift;
  sums.buffers = std::min(kDColumns / (N * w.groups() >> sums.part_shift), kMaxD);
  DFL_RET(launch_pdl(w4_tc_kernel<N>, dim3(run.runs), dim3(kThreads),
                     1024 + L::kCodeSlots * w.block_bytes + L::kXSlots * L::kX, s, w, run, sums, tmx, x, ldx, vec,
                     rows, epi));
  count_launch();
  return cudaSuccess;
}
}  // namespace

cudaError_t w4_linear_tc(const W4View& w, const void* x, long long ldx, int rows, const W4Epi& epi, const W4Scratch& sc,
                         cudaStream_t s) {
  return rows <= 32   ? tc_launch<32>(w, (const bf16*)x, ldx, rows, epi, sc, s)
         : rows <= 64 ? tc_launch<64>(w, (const bf16*)x, ldx, rows, epi, sc, s)
                      : tc_launch<128>(w, (const bf16*)x, ldx, rows, epi, sc, s);
}

}  // namespace dfl
