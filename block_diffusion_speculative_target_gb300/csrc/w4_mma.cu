// Products of few rows with 4-bit weights, tensor cores fed from registers.
//
// y[n][m] = sum over groups of s[m][g] * sum_{k in g} (code[m][k] - zero[m][g]) x[n][k]
//
// Codes less zero points are integers of at most 15, exact in bf16, and so are
// their products with x in float32.  A group's sum c is taken in float32 by the
// products' accumulator, then acc += s c.  Weights are the products' rows (m16),
// rows of x their columns (n8), so a token costs one column of eight.
//
// A code pair becomes two bf16 in one register without a conversion.  Eight bits
// v at the low end of a bf16 are the number v 2^-133, below the normal numbers and
// just into them; so the low or the high half of a byte, masked out and multiplied
// by 2^127 or 2^123, less zero / 64, is (code - zero) / 64 exactly: one mask and
// one packed multiply-add a pair, one shift for every other byte.  (The integer
// pipe has half the lanes of the others: with a shift for every pair it was the
// bound.)  The results take the factor of 64 back.  The codes lie in memory in the
// order of the products' fragments, so a lane reads 32 of its own codes with one
// 16-byte load and nothing is shuffled.
//
// Split: the blocks of 128 by 128 of the whole matrix form a line (row blocks
// one after another), cut into equal runs, one to a CTA, whatever M and K are.
// A CTA streams its run through shared memory, a block (one bulk copy) and the 128
// columns of x that it meets (asynchronous copies, swizzled by hand, so that rows
// of x may lie anywhere) a stage; 4 warps take 32 weight rows each.  A row block
// that lies in several runs leaves a partial sum in each; the warp that ends the
// last one of its 32 rows adds them in order of the columns.  The cut depends on M,
// K and the GPU only, and no sum on the other rows of x: a row has the same bits
// alone and in a block.
//
// Measured: 15 rows of 151936 x 5120 100 us (4.1 TB/s, the floor 60), 16 rows of
// 24576 x 4096 with the activation 22.7 us (2.4 TB/s), one row of 4096 x 4096 7.8 us.
// On large matrices neither issue (59% of the slots) nor memory (50%) is at its limit:
// four warps in step at a barrier a block, 16 warps a multiprocessor.  Small ones are a
// chain of trips to memory: first block, x, partial sums, ticket, join.
// 17 rows and more go to the kernel that expands codes once for 128 columns: with 32 rows
// of 4096 x 12288 that took 21 us, a form of four column tiles of this one 30.
//
// The waits for copies are bounded (dflash_debug_set_wait_limit); a CTA whose wait
// runs out sets DFLASH_STATUS_TIMEOUT, waits for what it has in flight and leaves
// without a result.
#include <algorithm>

#include "common.cuh"
#include "internal.h"
#include "w4.cuh"
#include "w4_ops.cuh"

namespace dfl {

namespace {
constexpr int kThreads = 128;
// Rows of x in one pass, as tiles of eight.
template <int NT>
struct MmaLayout {
  static constexpr int kRows = 8 * NT;
  static constexpr int kX = kRows * 256;  // 128 columns of bf16, 16-byte chunks swizzled by row
  static constexpr int kStages = NT == 1 ? 4 : 3;
  static constexpr int kSums = 4 * kRows * kW4SumRow * 4;  // the warps' sums at a row block's end
};

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, "
      "%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// c = a b
__device__ __forceinline__ void mma16816_first(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, "
      "%10, %10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}
}  // namespace

// One CTA: run blockIdx.x.  NT: tiles of eight rows of x; GS: log2(group / 32).
template <int NT, int GS>
__global__ void __launch_bounds__(kThreads, 4)
    w4_mma_kernel(const __grid_constant__ W4View w, const __grid_constant__ W4Run run, const bf16* __restrict__ x,
                  long long ldx, int vec, int rows, const __grid_constant__ W4Epi epi) {
  typedef MmaLayout<NT> L;
  constexpr int S = L::kStages, V = 2 * NT;  // V: float4 of sums a thread
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ __align__(8) uint64_t code_full[S];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, t = lane & 3;
  const int b0 = blockIdx.x * run.per, b1 = min(b0 + run.per, run.blocks);
  const int stage_bytes = L::kX + w.block_bytes;
  const uint32_t base = smem_u32(smem);

  // One thread: codes, scales and zeros of the block at `src` into a stage.
  auto load_codes = [&](const uint8_t* src, int slot) {
    mbar_arrive_expect_tx(&code_full[slot], w.block_bytes);
    bulk_load(smem + slot * stage_bytes + L::kX, src, w.block_bytes, &code_full[slot]);
  };
  // The columns k0 .. of x: row r's chunk c (8 columns) at r * 256 + 16 (c ^ (r & 7)); this thread brings chunk
  // tid % 16 of the rows tid / 16 + 8 u.  Rows past the last one are not filled: their columns of the products are
  // not used.
  const int xr = tid >> 4, xc = tid & 15;
  const uint32_t x_at = (uint32_t)(xr * 256 + 16 * (xc ^ xr));
  const bf16* x_row = x + (long long)xr * ldx + 8 * xc;
  auto load_x = [&](int k0, int slot) {
    const bool in_k = k0 + 8 * xc < w.K;
    const uint32_t at = slot * stage_bytes + x_at;
#pragma unroll
    for (int u = 0; u < NT; ++u) {
      if (xr + 8 * u >= rows) break;
      const bf16* src = in_k ? x_row + (long long)(8 * u) * ldx + k0 : x;
      if (vec)
        cp16z(base + at + u * 2048, src, in_k ? 16 : 0);
      else
        *reinterpret_cast<uint4*>(smem + at + u * 2048) = gather8(src, in_k);
    }
  };

  const uint8_t* next_block = w.packed + (long long)b0 * w.block_bytes;
  int mt = b0 / w.kt, kb = b0 - mt * w.kt;  // the block at hand
  int next_kb = kb;                         // the next one to be asked for
  if (tid == 0) {
    for (int u = 0; u < S; ++u) mbar_init(&code_full[u], 1);
    fence_barrier_init();
    // The weights do not depend on the kernels before this one (packing lets no successor start early, and has
    // published its stores by its end): the first blocks are asked for before the wait.
#pragma unroll
    for (int u = 0; u < S - 1; ++u)
      if (b0 + u < b1) load_codes(next_block + (long long)u * w.block_bytes, u);
  }
  next_block += (long long)(S - 1) * w.block_bytes;
  __syncthreads();
  pdl_launch();
  pdl_wait();
#pragma unroll
  for (int u = 0; u < S - 1; ++u) {
    if (b0 + u < b1) load_x(next_kb * kW4Tile, u);
    cp_commit();
    if (++next_kb == w.kt) next_kb = 0;
  }

  float acc[V][4];
#pragma unroll
  for (int v = 0; v < V; ++v)
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[v][e] = 0.f;
  const int zero_at = kW4Codes + (4 >> GS) * kW4Tile * (w.scale_f32 ? 4 : 2);
  uint32_t off[2][2];
#pragma unroll
  for (int y = 0; y < 2; ++y) off[y][0] = off[y][1] = offset_of(kW4Zero);
  // chunk 4 q + lane / 8 of row 8 j + lane % 8 of x lies at x_lane + 2048 j + 128 (q / 2) + x_q[q % 2]
  const uint32_t x_lane = base + (lane & 7) * 256 + 16 * ((lane >> 3) ^ (lane & 3));
  const uint32_t x_q[2] = {16u * (lane & 4), 16u * ((lane & 4) ^ 4)};

  int slot = 0;
  uint32_t phase = 0;
  for (int i = b0; i < b1; ++i) {
    cp_wait<S - 2>();
    const bool ok = landed(&code_full[slot], phase, run.wait_ns);
    if (__syncthreads_or(!ok)) {
      // (what was asked for lands before the CTA ends)
      cp_wait<0>();
      if (tid == 0) {
        set_status(run.status, DFLASH_STATUS_TIMEOUT);
        for (int u = i; u < min(i + S - 1, b1); ++u)
          mbar_wait(&code_full[(u - b0) % S], (uint32_t)((u - b0) / S) & 1u, kW4DrainNs);
      }
      return;
    }
    if (i + S - 1 < b1) {
      const int to = slot == 0 ? S - 1 : slot - 1;
      if (tid == 0) load_codes(next_block, to);
      load_x(next_kb * kW4Tile, to);
      next_block += w.block_bytes;
      if (++next_kb == w.kt) next_kb = 0;
    }
    cp_commit();
    const uint8_t* blk = smem + slot * stage_bytes + L::kX;
    const uint32_t xs = x_lane + slot * stage_bytes;
    if (++slot == S) {
      slot = 0;
      phase ^= 1u;
    }
    float c[V][4];
    uint4 word[2][2];
#pragma unroll
    for (int y = 0; y < 4; ++y)
      word[y >> 1][y & 1] = *reinterpret_cast<const uint4*>(blk + w4_word_at(2 * warp + (y >> 1), y & 1, lane));
#pragma unroll
    for (int q = 0; q < 4; ++q) {  // 32 columns: steps 2 q and 2 q + 1
      constexpr int kMask = (1 << GS) - 1;
      const bool first = (q & kMask) == 0, last = (q & kMask) == kMask;
      if (first && w.zeros) {
        const uint8_t* z = blk + zero_at + (q >> GS) * kW4Tile + 32 * warp + g;
#pragma unroll
        for (int y = 0; y < 2; ++y)
#pragma unroll
          for (int r = 0; r < 2; ++r) off[y][r] = offset_of(z[16 * y + 8 * r]);
      }
      uint32_t a[2][2][4];  // [m tile][step]
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const uint4 v = word[y][q >> 1];
        const uint32_t lo = q & 1 ? v.y : v.x, hi = q & 1 ? v.w : v.z;
        a[y][0][0] = pair_of<0>(lo, off[y][0]);
        a[y][0][1] = pair_of<0>(hi, off[y][1]);
        a[y][0][2] = pair_of<1>(lo, off[y][0]);
        a[y][0][3] = pair_of<1>(hi, off[y][1]);
        a[y][1][0] = pair_of<0>(lo >> 8, off[y][0]);
        a[y][1][1] = pair_of<0>(hi >> 8, off[y][1]);
        a[y][1][2] = pair_of<1>(lo >> 8, off[y][0]);
        a[y][1][3] = pair_of<1>(hi >> 8, off[y][1]);
      }
      // four chunks of 8 rows of x: (b0, b1) of the first step, then of the second
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        uint32_t b[4];
        ldsm4(b, xs + j * 2048 + (q >> 1) * 128 + x_q[q & 1]);
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          if (first)
            mma16816_first(c[y * NT + j], a[y][0], b[0], b[1]);
          else
            mma16816(c[y * NT + j], a[y][0], b[0], b[1]);
          mma16816(c[y * NT + j], a[y][1], b[2], b[3]);
        }
      }
      if (last) {
        const int at = (q >> GS) * kW4Tile + 32 * warp + g;
        float s[4];
        if (w.scale_f32) {
#pragma unroll
          for (int r = 0; r < 4; ++r) s[r] = reinterpret_cast<const float*>(blk + kW4Codes)[at + 8 * r];
        } else {
#pragma unroll
          for (int r = 0; r < 4; ++r) s[r] = to_f<bf16>(reinterpret_cast<const bf16*>(blk + kW4Codes)[at + 8 * r]);
        }
#pragma unroll
        for (int v = 0; v < V; ++v)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[v][e] = fmaf(s[2 * (v / NT) + (e >> 1)], c[v][e], acc[v][e]);
      }
    }
    const int tile = mt;
    const bool tile_end = ++kb == w.kt;
    if (tile_end) {
      kb = 0;
      ++mt;
    } else if (i + 1 < b1) {
      continue;
    }
    // The row block ends here, or the run does.  A warp deals with its 32 rows by itself.
    w4_join<V, V>(w, run, tile, tid, acc, [&](int, const float (&sum)[V][4]) {
      float* sums = reinterpret_cast<float*>(smem + S * stage_bytes) + warp * (L::kRows * kW4SumRow);
#pragma unroll
      for (int v = 0; v < V; ++v)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          sums[(8 * (v % NT) + 2 * t + (e & 1)) * kW4SumRow + 16 * (v / NT) + g + 8 * (e >> 1)] = sum[v][e];
      __syncwarp();
      w4_results(w, epi, tile * kW4Tile + 32 * warp, sums, 0, rows);
      __syncwarp();
    });
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[v][e] = 0.f;
  }
}

namespace {
template <int NT, int GS>
cudaError_t mma_launch(const W4View& w, const bf16* x, long long ldx, int rows, const W4Epi& epi, const W4Scratch& sc,
                       cudaStream_t s) {
  typedef MmaLayout<NT> L;
  static PerDevice attr;
  // (the widest block: float32 scales and zero points)
  constexpr int kMost = L::kStages * (kW4Codes + (4 >> GS) * kW4Tile * 5 + L::kX) + L::kSums;
  static_assert(kMost <= 232448 - 1024, "shared memory per block");
  DFL_RET(attr.once([] {
    return cudaFuncSetAttribute(w4_mma_kernel<NT, GS>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMost);
  }));
  const int vec = (reinterpret_cast<uintptr_t>(x) & 15) == 0 && ldx % 8 == 0;
  const W4Run run = w4_run(w, sc, rows);
  DFL_RET(launch_pdl(w4_mma_kernel<NT, GS>, dim3(run.runs), dim3(kThreads), L::kStages * (w.block_bytes + L::kX) + L::kSums,
                     s, w, run, x, ldx, vec, rows, epi));
  count_launch();
  return cudaSuccess;
}
template <int NT>
cudaError_t mma_group(const W4View& w, const bf16* x, long long ldx, int rows, const W4Epi& epi, const W4Scratch& sc,
                      cudaStream_t s) {
  return w.group == 32   ? mma_launch<NT, 0>(w, x, ldx, rows, epi, sc, s)
         : w.group == 64 ? mma_launch<NT, 1>(w, x, ldx, rows, epi, sc, s)
                         : mma_launch<NT, 2>(w, x, ldx, rows, epi, sc, s);
}
}  // namespace

cudaError_t w4_linear_mma(const W4View& w, const void* x, long long ldx, int rows, const W4Epi& epi,
                          const W4Scratch& sc, cudaStream_t s) {
  const bf16* b = (const bf16*)x;
  return rows <= 8 ? mma_group<1>(w, b, ldx, rows, epi, sc, s) : mma_group<2>(w, b, ldx, rows, epi, sc, s);
}

}  // namespace dfl
