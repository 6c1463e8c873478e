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
__device__ __forceinline__ void mma16816_first(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, "
      "%10, %10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}
// Pair p (0, 1: of the low bytes) of a word of codes as (code - zero) / 64; off holds -zero / 64 twice.
template <int P>
__device__ __forceinline__ uint32_t pair_of(uint32_t word, uint32_t off) {
  uint32_t d;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;"
      : "=r"(d)
      : "r"(word & (P ? 0x00F000F0u : 0x000F000Fu)), "r"(P ? 0x7D007D00u : 0x7F007F00u), "r"(off));
  return d;
}
constexpr float kW4Unit = 64.f;
__device__ __forceinline__ uint32_t offset_of(int zero) {
  const __nv_bfloat162 v = __float2bfloat162_rn((float)zero * (-1.f / kW4Unit));
  return *reinterpret_cast<const uint32_t*>(&v);
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

  // Codes, scales and zeros of the block at `src` into the stage at `at`.
  auto load_codes = [&](const uint8_t* src, uint32_t at) {
    const uint32_t dst = base + at + 16 * tid;
    src += 16 * tid;
#pragma unroll
    for (int c = 0; c < kW4Codes; c += kThreads * 16) cp16(dst + c, src + c);
    for (int c = kW4Codes; c + 16 * tid < w.block_bytes; c += kThreads * 16) cp16(dst + c, src + c);
  };
  // The columns k0 .. of x: row r's chunk c (8 columns) at r * 256 + 16 (c ^ (r & 7)); this thread brings chunk
  // tid % 16 of the rows tid / 16 + 8 u.
  const int xr = tid >> 4, xc = tid & 15;
  const uint32_t x_at = (uint32_t)(w.block_bytes + xr * 256 + 16 * (xc ^ xr));
  const bf16* x_row = x + (long long)(n0 + xr) * ldx + 8 * xc;
  auto load_x = [&](int k0, uint32_t at, bool async) {
    const bool in_k = k0 + 8 * xc < w.K;
    at += x_at;
#pragma unroll
    for (int u = 0; u < NT; ++u) {
      const bool in = in_k && n0 + xr + 8 * u < rows;
      const bf16* src = in ? x_row + (long long)(8 * u) * ldx + k0 : x;
      uint4* dst = reinterpret_cast<uint4*>(smem + at + u * 2048);
      if (vec && async) {
        cp16z(base + at + u * 2048, src, in ? 16 : 0);
      } else if (vec) {
        *dst = in ? *reinterpret_cast<const uint4*>(src) : make_uint4(0u, 0u, 0u, 0u);
      } else {
        uint32_t v[4] = {0u, 0u, 0u, 0u};
        if (in) {
          const uint16_t* h = reinterpret_cast<const uint16_t*>(src);
#pragma unroll
          for (int e = 0; e < 4; ++e) v[e] = h[2 * e] | (uint32_t)h[2 * e + 1] << 16;
        }
        *dst = make_uint4(v[0], v[1], v[2], v[3]);
      }
    }
  };

  // The weights do not depend on the kernels before this one (packing lets no successor start early): the first
  // stages are asked for before the wait.
  const uint8_t* next_block = w.packed + (long long)b0 * w.block_bytes;
  int mt = b0 / w.kt, kb = b0 - mt * w.kt;  // the block at hand
  int next_kb = kb;                         // the next one to be asked for
#pragma unroll
  for (int u = 0; u < S - 1; ++u) {
    if (b0 + u < b1) load_codes(next_block, u * stage_bytes);
    next_block += w.block_bytes;
    cp_commit();
  }
  pdl_launch();
  pdl_wait();
#pragma unroll
  for (int u = 0; u < S - 1; ++u) {
    if (b0 + u < b1) load_x(next_kb * kW4Tile, u * stage_bytes, false);
    if (++next_kb == w.kt) next_kb = 0;
  }

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

  uint32_t at = 0, next_at = (S - 1) * stage_bytes;  // the stage at hand and the one to fill
  for (int i = b0; i < b1; ++i) {
    cp_wait<S - 2>();
    __syncthreads();
    if (i + S - 1 < b1) {
      load_codes(next_block, next_at);
      load_x(next_kb * kW4Tile, next_at, true);
      next_block += w.block_bytes;
      if (++next_kb == w.kt) next_kb = 0;
    }
    cp_commit();
    const uint8_t* blk = smem + at;
    // chunk 4 q + lane / 8 of row 8 j + lane % 8
    const uint32_t xs = base + at + w.block_bytes + (lane & 7) * 256 + 16 * ((lane >> 3) ^ (lane & 3));
    next_at = at;
    at += stage_bytes;
    if (at == S * stage_bytes) at = 0;
    float c[2][NT][4];
    uint4 word[2];
#pragma unroll
    for (int q = 0; q < 4; ++q) {  // 32 columns: steps 2 q and 2 q + 1
      if ((q & 1) == 0) {
#pragma unroll
        for (int y = 0; y < 2; ++y)
          word[y] = *reinterpret_cast<const uint4*>(blk + w4_word_at(2 * warp + y, q >> 1, lane));
      }
      if (w.zeros && (q & (groups32 - 1)) == 0) {
        const uint8_t* z = blk + zero_at + q / groups32 * kW4Tile + 32 * warp + g;
#pragma unroll
        for (int y = 0; y < 2; ++y)
#pragma unroll
          for (int r = 0; r < 2; ++r) off[y][r] = offset_of(z[16 * y + 8 * r]);
      }
      uint32_t a[2][2][4];  // [m tile][step]
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const uint32_t lo = q & 1 ? word[y].y : word[y].x, hi = q & 1 ? word[y].w : word[y].z;
        a[y][0][0] = pair_of<0>(lo, off[y][0]);
        a[y][0][1] = pair_of<0>(hi, off[y][1]);
        a[y][0][2] = pair_of<1>(lo, off[y][0]);
        a[y][0][3] = pair_of<1>(hi, off[y][1]);
        a[y][1][0] = pair_of<0>(lo >> 8, off[y][0]);
        a[y][1][1] = pair_of<0>(hi >> 8, off[y][1]);
        a[y][1][2] = pair_of<1>(lo >> 8, off[y][0]);
        a[y][1][3] = pair_of<1>(hi >> 8, off[y][1]);
      }
      // four chunks of 8 rows of x: (b0, b1) of the first step, then of the second.  (4 q ^ bit 2 of the row: the
      // rest of the swizzle is in xs)
      const bool fresh = (q & (groups32 - 1)) == 0;
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        uint32_t b[4];
        ldsm4(b, xs + j * 2048 + 16 * ((4 * q) ^ (lane & 4)));
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          if (q == 0 || fresh)
            mma16816_first(c[y][j], a[y][0], b[0], b[1]);
          else
            mma16816(c[y][j], a[y][0], b[0], b[1]);
          mma16816(c[y][j], a[y][1], b[2], b[3]);
        }
      }
      if (((q + 1) & (groups32 - 1)) == 0) {
        const int sat = q / groups32 * kW4Tile + 32 * warp + g;
        const float* sf = reinterpret_cast<const float*>(blk + kW4Codes) + sat;
        const bf16* sb = reinterpret_cast<const bf16*>(blk + kW4Codes) + sat;
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
    const int tile = mt;
    const bool tile_end = ++kb == w.kt;
    if (tile_end) {
      kb = 0;
      ++mt;
    } else if (i + 1 < b1) {
      continue;
    }
    // The row block ends here, or the run does.
    const int t0 = tile * w.kt, first_run = t0 / run.per, last_run = (t0 + w.kt - 1) / run.per;
    bool done = true;
    if (last_run > first_run) {
      // run r's piece of the row block: its first slot if the run begins in the block, else its second
      auto slot = [&](int r) {
        return reinterpret_cast<float4*>(run.part + (((long long)blockIdx.y * run.runs + r) * 2 + (r * run.per < t0)) *
                                                        (kW4Tile * L::kRows)) + tid;
      };
      float4* own = slot(blockIdx.x);
#pragma unroll
      for (int v = 0; v < 2 * NT; ++v) {
        const float* p = acc[v / NT][v % NT];
        __stcg(own + v * kThreads, make_float4(p[0], p[1], p[2], p[3]));
      }
      __threadfence();
      __syncthreads();
      if (tid == 0) {
        int* ticket = run.tickets + blockIdx.y * run.runs + first_run;
        last_s = atomicAdd(ticket, 1) == last_run - first_run;
        if (last_s) *ticket = 0;
      }
      __syncthreads();
      done = last_s;
      if (done) {
        __threadfence();
        // the pieces' sums in order, the loads of several in flight
        constexpr int kAhead = NT <= 2 ? 4 : NT == 4 ? 2 : 1;
#pragma unroll
        for (int v = 0; v < 2 * NT; ++v)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[v / NT][v % NT][e] = 0.f;
        for (int r = first_run; r <= last_run; r += kAhead) {
          float4 p[kAhead][2 * NT];
#pragma unroll
          for (int u = 0; u < kAhead; ++u) {
            const float4* src = slot(min(r + u, last_run));
#pragma unroll
            for (int v = 0; v < 2 * NT; ++v) p[u][v] = __ldcg(src + v * kThreads);
          }
#pragma unroll
          for (int u = 0; u < kAhead; ++u)
            if (r + u <= last_run) {
#pragma unroll
              for (int v = 0; v < 2 * NT; ++v) {
                float* d = acc[v / NT][v % NT];
                d[0] += p[u][v].x;
                d[1] += p[u][v].y;
                d[2] += p[u][v].z;
                d[3] += p[u][v].w;
              }
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
            const int m = tile * kW4Tile + 32 * warp + 16 * y + g + 8 * (e >> 1);
            const int n = n0 + 8 * j + 2 * t + (e & 1);
            const bool live = m < w.M && n < rows;
            float v = acc[y][j][e] * kW4Unit;
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
    for (int v = 0; v < 2 * NT; ++v)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[v / NT][v % NT][e] = 0.f;
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
