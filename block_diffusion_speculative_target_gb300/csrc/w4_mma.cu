// Products with 4-bit weights, tensor cores fed from registers.
//
// y[n][m] = sum over groups of s[m][g] * sum_{k in g} (code[m][k] - zero[m][g]) x[n][k]
//
// Codes less zero points are integers of at most 15, exact in bf16, and so are
// their products with x in float32; a group's sum c is taken in float32 by the
// products' accumulator, then acc += s c.  Weights are the products' rows (m16),
// rows of x their columns (n8), so a token costs one column of eight and not one
// row of sixteen.
//
// A code pair becomes two bf16 in one register without a conversion: the bits
// 0x4300 | code are the bf16 128 + code, and 128 + zero taken off it leaves
// code - zero exactly: for 8 codes 3 shifts, 4 masks and 4 packed subtractions.
// The codes lie in memory in the order of the products' fragments, so a lane
// reads 32 of its own codes with one 16-byte load and nothing is shuffled.
//
// Split: the blocks of 128 by 128 of the whole matrix form a line (row blocks
// one after another), cut into equal runs, one to a CTA, whatever M and K are.
// A CTA streams its run through shared memory (asynchronous copies, one block
// and the 128 columns of x that it meets a stage); 4 warps take 32 weight rows
// each.  A row block that lies in several runs leaves a partial sum in each; the
// CTA that ends the last one adds them in order of the columns.  The cut depends
// on M, K and the GPU only, and no sum on the other rows of x: a row has the same
// bits alone and in a block.
#include <algorithm>

#include "common.cuh"
#include "internal.h"
#include "w4.cuh"

namespace dfl {

namespace {
constexpr int kThreads = 128;
// Rows of x in one pass, as tiles of eight.
template <int NT>
struct MmaLayout {
  static constexpr int kRows = 8 * NT;
  static constexpr int kX = kRows * 256;  // 128 columns of bf16, 16-byte chunks swizzled by row
  static constexpr int kStages = NT == 1 ? 5 : NT == 2 ? 4 : NT == 4 ? 3 : 4;
  static constexpr int kCtas = NT <= 4 ? 4 : 2;
};

__device__ __forceinline__ void cp16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
// `bytes` of 16 (0: none is read), the rest zeros
__device__ __forceinline__ void cp16z(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
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
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, "
      "%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Pair p of a word of codes, less the zero point: off = bf16 pair of 128 + zero.
template <int P>
__device__ __forceinline__ uint32_t pair_of(uint32_t word, uint32_t off) {
  const uint32_t v = ((word >> (4 * P)) & 0x000F000Fu) | 0x43004300u;
  uint32_t d;
  asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(v), "r"(off));
  return d;
}
__device__ __forceinline__ uint32_t offset_of(int zero) {
  return 0x43004300u + (uint32_t)zero * 0x00010001u;  // (128 + zero needs 8 bits)
}
}  // namespace

struct W4Run {
  int blocks, per;    // blocks of the matrix, blocks a run
  float* part;        // [passes][runs][2][values][threads][4]
  int* tickets;       // [passes][runs]
  int runs;
};

// One CTA: run blockIdx.x, rows 8 NT blockIdx.y .. of x.
template <int NT>
__global__ void __launch_bounds__(kThreads, MmaLayout<NT>::kCtas)
    w4_mma_kernel(const __grid_constant__ W4View w, const __grid_constant__ W4Run run, const bf16* __restrict__ x,
                  long long ldx, int vec, int rows, const __grid_constant__ W4Epi epi) {
  typedef MmaLayout<NT> L;
  constexpr int S = L::kStages;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int last_s;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, t = lane & 3;
  const int stage_bytes = w.block_bytes + L::kX;
  const int n0 = blockIdx.y * L::kRows;
  const int b0 = blockIdx.x * run.per, b1 = min(b0 + run.per, run.blocks);
  const uint32_t base = smem_u32(smem);

  auto load_codes = [&](int i) {  // block i of the line
    const uint32_t dst = base + (uint32_t)((i - b0) % S) * stage_bytes;
    const uint8_t* src = w.packed + (long long)i * w.block_bytes;
    for (int c = tid * 16; c < w.block_bytes; c += kThreads * 16) cp16(dst + c, src + c);
  };
  // the columns of x that block i meets: row r's chunk c (8 columns) at r * 256 + 16 (c ^ (r & 7))
  auto load_x = [&](int i, bool async) {
    const int slot = (i - b0) % S, k0 = i % w.kt * kW4Tile;
    const uint32_t dst = base + (uint32_t)slot * stage_bytes + w.block_bytes;
    uint8_t* sx = smem + (size_t)slot * stage_bytes + w.block_bytes;
#pragma unroll
    for (int u = 0; u < NT; ++u) {
      const int r = u * 8 + (tid >> 4), c = tid & 15, k = k0 + 8 * c;
      const uint32_t at = (uint32_t)(r * 256 + 16 * (c ^ (r & 7)));
      const bool in = n0 + r < rows && k < w.K;
      const bf16* src = x + (in ? (long long)(n0 + r) * ldx + k : 0);
      if (vec && async) {
        cp16z(dst + at, src, in ? 16 : 0);
      } else if (vec) {
        uint4 v = make_uint4(0u, 0u, 0u, 0u);
        if (in) v = *reinterpret_cast<const uint4*>(src);
        *reinterpret_cast<uint4*>(sx + at) = v;
      } else {
        uint32_t v[4] = {0u, 0u, 0u, 0u};
        if (in) {
          const uint16_t* h = reinterpret_cast<const uint16_t*>(src);
#pragma unroll
          for (int e = 0; e < 4; ++e) v[e] = h[2 * e] | (uint32_t)h[2 * e + 1] << 16;
        }
        *reinterpret_cast<uint4*>(sx + at) = make_uint4(v[0], v[1], v[2], v[3]);
      }
    }
  };

  // The weights do not depend on the kernels before this one (packing lets no successor start early): the first
  // stages are asked for before the wait.
#pragma unroll
  for (int u = 0; u < S - 1; ++u) {
    if (b0 + u < b1) load_codes(b0 + u);
    cp_commit();
  }
  pdl_launch();
  pdl_wait();
#pragma unroll
  for (int u = 0; u < S - 1; ++u)
    if (b0 + u < b1) load_x(b0 + u, false);

  float acc[2][NT][4];
#pragma unroll
  for (int y = 0; y < 2; ++y)
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[y][j][e] = 0.f;
  const int groups32 = w.group / 32, zero_at = kW4Codes + w.groups() * kW4Tile * (w.scale_f32 ? 4 : 2);
  uint32_t off[2][2];
#pragma unroll
  for (int y = 0; y < 2; ++y) off[y][0] = off[y][1] = offset_of(kW4Zero);

  for (int i = b0; i < b1; ++i) {
    cp_wait<S - 2>();
    __syncthreads();
    if (i + S - 1 < b1) {
      load_codes(i + S - 1);
      load_x(i + S - 1, true);
    }
    cp_commit();
    const uint8_t* blk = smem + (size_t)((i - b0) % S) * stage_bytes;
    const uint32_t xs = base + (uint32_t)((i - b0) % S) * stage_bytes + w.block_bytes;
    float c[2][NT][4];
    uint4 word[2];
#pragma unroll
    for (int q = 0; q < 4; ++q) {  // 32 columns: steps 2 q and 2 q + 1
      if ((q & 1) == 0) {
#pragma unroll
        for (int y = 0; y < 2; ++y)
          word[y] = *reinterpret_cast<const uint4*>(blk + w4_word_at(2 * warp + y, q >> 1, lane));
      }
      const bool first = q % groups32 == 0;
      if (first) {
#pragma unroll
        for (int y = 0; y < 2; ++y)
#pragma unroll
          for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) c[y][j][e] = 0.f;
        if (w.zeros) {
          const uint8_t* z = blk + zero_at + q / groups32 * kW4Tile + 32 * warp + g;
#pragma unroll
          for (int y = 0; y < 2; ++y)
#pragma unroll
            for (int r = 0; r < 2; ++r) off[y][r] = offset_of(z[16 * y + 8 * r]);
        }
      }
      uint32_t a[2][2][4];  // [m tile][step]
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const uint32_t lo = q & 1 ? word[y].y : word[y].x, hi = q & 1 ? word[y].w : word[y].z;
        a[y][0][0] = pair_of<0>(lo, off[y][0]);
        a[y][0][1] = pair_of<0>(hi, off[y][1]);
        a[y][0][2] = pair_of<1>(lo, off[y][0]);
        a[y][0][3] = pair_of<1>(hi, off[y][1]);
        a[y][1][0] = pair_of<2>(lo, off[y][0]);
        a[y][1][1] = pair_of<2>(hi, off[y][1]);
        a[y][1][2] = pair_of<3>(lo, off[y][0]);
        a[y][1][3] = pair_of<3>(hi, off[y][1]);
      }
      // chunks 4 q .. 4 q + 3 of 8 rows of x: (b0, b1) of the first step, then of the second
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        uint32_t b[4];
        const int r = 8 * j + (lane & 7), ch = 4 * q + (lane >> 3);
        ldsm4(b, xs + (uint32_t)(r * 256 + 16 * (ch ^ (r & 7))));
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          mma16816(c[y][j], a[y][0], b[0], b[1]);
          mma16816(c[y][j], a[y][1], b[2], b[3]);
        }
      }
      if ((q + 1) % groups32 == 0) {
        const int at = q / groups32 * kW4Tile + 32 * warp + g;
        const float* sf = reinterpret_cast<const float*>(blk + kW4Codes) + at;
        const bf16* sb = reinterpret_cast<const bf16*>(blk + kW4Codes) + at;
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          const float s0 = w.scale_f32 ? sf[16 * y] : to_f<bf16>(sb[16 * y]);
          const float s1 = w.scale_f32 ? sf[16 * y + 8] : to_f<bf16>(sb[16 * y + 8]);
#pragma unroll
          for (int j = 0; j < NT; ++j) {
            acc[y][j][0] = fmaf(s0, c[y][j][0], acc[y][j][0]);
            acc[y][j][1] = fmaf(s0, c[y][j][1], acc[y][j][1]);
            acc[y][j][2] = fmaf(s1, c[y][j][2], acc[y][j][2]);
            acc[y][j][3] = fmaf(s1, c[y][j][3], acc[y][j][3]);
          }
        }
      }
    }
    const int mt = i / w.kt;
    const bool tile_end = i - mt * w.kt == w.kt - 1;
    if (!tile_end && i + 1 < b1) continue;
    // The row block ends here, or the run does.
    const int t0 = mt * w.kt, first_run = t0 / run.per, last_run = (t0 + w.kt - 1) / run.per, pieces = last_run - first_run + 1;
    bool done = true;
    if (pieces > 1) {
      // run r's piece of the row block: its first slot if the run begins in the block, else its second
      auto slot = [&](int r) {
        return run.part +
               (((long long)blockIdx.y * run.runs + r) * 2 + (r * run.per < t0)) * (kW4Tile * L::kRows);
      };
      float4* own = reinterpret_cast<float4*>(slot(blockIdx.x));
#pragma unroll
      for (int y = 0; y < 2; ++y)
#pragma unroll
        for (int j = 0; j < NT; ++j)
          own[(y * NT + j) * kThreads + tid] = make_float4(acc[y][j][0], acc[y][j][1], acc[y][j][2], acc[y][j][3]);
      __threadfence();
      __syncthreads();
      int* ticket = run.tickets + blockIdx.y * run.runs + first_run;
      if (tid == 0) {
        const int was = atomicAdd(ticket, 1);
        last_s = was == pieces - 1;
        if (was == pieces - 1) *ticket = 0;
      }
      __syncthreads();
      done = last_s;
      if (done) {
        __threadfence();
#pragma unroll
        for (int y = 0; y < 2; ++y)
#pragma unroll
          for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[y][j][e] = 0.f;
        for (int r = first_run; r <= last_run; ++r) {
          const float4* p = reinterpret_cast<const float4*>(slot(r));
#pragma unroll
          for (int y = 0; y < 2; ++y)
#pragma unroll
            for (int j = 0; j < NT; ++j) {
              const float4 v = __ldcg(p + (y * NT + j) * kThreads + tid);
              acc[y][j][0] += v.x;
              acc[y][j][1] += v.y;
              acc[y][j][2] += v.z;
              acc[y][j][3] += v.w;
            }
        }
      }
    }
    if (done) {
#pragma unroll
      for (int y = 0; y < 2; ++y)
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int m = mt * kW4Tile + 32 * warp + 16 * y + g + 8 * (e >> 1);
            const int n = n0 + 8 * j + 2 * t + (e & 1);
            const bool live = m < w.M && n < rows;
            float v = acc[y][j][e];
            if (epi.add && live) v += epi.add[(long long)n * w.M + m];
            if (epi.swiglu) {  // the lane of row m + 1 is 4 further
              const float up = __shfl_down_sync(0xffffffffu, v, 4);
              if (live && !(m & 1)) {
                const float o = v / (1.f + expf(-v)) * up;
                reinterpret_cast<bf16*>(epi.out)[(long long)n * (w.M / 2) + m / 2] = from_f<bf16>(o);
              }
            } else if (live) {
              reinterpret_cast<float*>(epi.out)[(long long)n * w.M + m] = v;
            }
          }
    }
#pragma unroll
    for (int y = 0; y < 2; ++y)
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[y][j][e] = 0.f;
  }
}

namespace {
constexpr int kRunsPerSm = 4;
constexpr int kMinRun = 4;  // blocks of a run at least

template <int NT>
cudaError_t mma_launch(const W4View& w, const bf16* x, long long ldx, int rows, const W4Epi& epi, float* part,
                       int* tickets, cudaStream_t s) {
  typedef MmaLayout<NT> L;
  static PerDevice attr;
  // (the widest block: groups of 32, float32 scales and zero points)
  constexpr int kMost = L::kStages * (kW4Codes + 4 * kW4Tile * 5 + L::kX);
  static_assert(kMost <= 232448 - 1024, "shared memory per block");
  DFL_RET(attr.once([] {
    return cudaFuncSetAttribute(w4_mma_kernel<NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMost);
  }));
  const int vec = (reinterpret_cast<uintptr_t>(x) & 15) == 0 && ldx % 8 == 0;
  W4Run run;
  run.blocks = (w.M + kW4Tile - 1) / kW4Tile * w.kt;
  run.per = w4_run_blocks(w);
  run.runs = (run.blocks + run.per - 1) / run.per;
  run.part = part;
  run.tickets = tickets;
  const dim3 grid(run.runs, (rows + L::kRows - 1) / L::kRows);
  DFL_RET(launch_pdl(w4_mma_kernel<NT>, grid, dim3(kThreads), L::kStages * (w.block_bytes + L::kX), s, w, run, x, ldx,
                     vec, rows, epi));
  count_launch();
  return cudaSuccess;
}
}  // namespace

int w4_run_blocks(const W4View& w) {
  const int blocks = (w.M + kW4Tile - 1) / kW4Tile * w.kt, most = num_sms() * kRunsPerSm;
  return std::max(kMinRun, (blocks + most - 1) / most);
}
int w4_max_runs() { return num_sms() * kRunsPerSm; }

cudaError_t w4_linear_mma(const W4View& w, const void* x, long long ldx, int rows, const W4Epi& epi, float* part,
                          int* tickets, cudaStream_t s) {
  const bf16* b = (const bf16*)x;
  if (rows <= 8) return mma_launch<1>(w, b, ldx, rows, epi, part, tickets, s);
  if (rows <= 16) return mma_launch<2>(w, b, ldx, rows, epi, part, tickets, s);
  if (rows <= 32) return mma_launch<4>(w, b, ldx, rows, epi, part, tickets, s);
  return mma_launch<8>(w, b, ldx, rows, epi, part, tickets, s);
}

}  // namespace dfl
