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
// one after another), cut into equal runs, one to a CTA, whatever M and K are.
// A CTA streams its run through shared memory (asynchronous copies, a block and
// the 128 columns of x that it meets a stage).  Several CTAs share an SM: while
// one waits for its products another one expands codes.  A row block that lies in
// several runs leaves a partial sum in each; the CTA that ends the last one adds
// them in order of the columns.  The cut depends on M, K and the GPU only, and no
// sum on the other rows of x: a row has the same bits alone and in a block.
//
// The waits for products are bounded (dflash_debug_set_wait_limit); a CTA whose
// wait runs out sets DFLASH_STATUS_TIMEOUT, waits for what it has in flight and
// leaves without a result.
#include <algorithm>

#include "common.cuh"
#include "internal.h"
#include "w4.cuh"

namespace dfl {

namespace {
constexpr int kThreads = 128;
constexpr uint64_t kDrainNs = 125000000ull;

// N: columns of a product (rows of x in one pass, padded); NR: those that are read back.
template <int N, int NR>
struct TcLayout {
  static constexpr int kX = N * 256;  // two halves of 64 columns: rows of 128 bytes, 16-byte chunks swizzled by row
  static constexpr int kStages = N <= 16 ? 4 : N == 32 ? 3 : N == 64 ? 4 : 2;
  static constexpr int kCtas = N <= 32 ? 4 : 2;
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
__device__ __forceinline__ void tmem_ld8u(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr)
               : "memory");
}
// Pair P (0, 1: of the low bytes) of a word of codes as (code - zero) / 64; off holds -zero / 64 twice.
template <int P>
__device__ __forceinline__ uint32_t pair_of(uint32_t word, uint32_t off) {
  uint32_t d;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;"
      : "=r"(d)
      : "r"(word & (P ? 0x00F000F0u : 0x000F000Fu)), "r"(P ? 0x7D007D00u : 0x7F007F00u), "r"(off));
  return d;
}
constexpr float kUnit = 64.f;
__device__ __forceinline__ uint32_t offset_of(int zero) {
  const __nv_bfloat162 v = __float2bfloat162_rn((float)zero * (-1.f / kUnit));
  return *reinterpret_cast<const uint32_t*>(&v);
}
}  // namespace

struct W4Run {
  int blocks, per, runs;  // blocks of the matrix, blocks a run, runs
  float* part;            // [passes][runs][2][NR / 4][threads][4]
  int* tickets;           // [passes][runs]
  int* status;
  unsigned long long wait_ns;
  uint32_t columns;       // TMEM columns: 64 of weights, N for each group of a block
};

// One CTA: run blockIdx.x, rows N blockIdx.y .. of x.
template <int N, int NR>
__global__ void __launch_bounds__(kThreads, (TcLayout<N, NR>::kCtas))
    w4_tc_kernel(const __grid_constant__ W4View w, const __grid_constant__ W4Run run, const bf16* __restrict__ x,
                 long long ldx, int vec, int rows, const __grid_constant__ W4Epi epi) {
  typedef TcLayout<N, NR> L;
  constexpr int S = L::kStages;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t mma_done;
  __shared__ uint32_t tmem_slot;
  __shared__ int last_s;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2;
  const int n0 = blockIdx.y * N;
  const int b0 = blockIdx.x * run.per, b1 = min(b0 + run.per, run.blocks);
  const uint32_t base = smem_u32(smem), codes_base = S * L::kX;

  // Codes, scales and zeros of the block at `src` into a stage.
  auto load_codes = [&](const uint8_t* src, int slot) {
    const uint32_t dst = base + codes_base + slot * w.block_bytes + 16 * tid;
    src += 16 * tid;
#pragma unroll
    for (int c = 0; c < kW4Codes; c += kThreads * 16) cp16(dst + c, src + c);
    for (int c = kW4Codes; c + 16 * tid < w.block_bytes; c += kThreads * 16) cp16(dst + c, src + c);
  };
  // The columns k0 .. of x: this thread brings chunk tid % 16 (8 columns) of the rows tid / 16 + 8 u.  Rows past the
  // last one are not filled: their columns of the products are not read.
  const int xr = tid >> 4, xc = tid & 15;
  const uint32_t x_at = (uint32_t)((xc >> 3) * (N * 128) + xr * 128 + 16 * ((xc & 7) ^ xr));
  const bf16* x_row = x + (long long)(n0 + xr) * ldx + 8 * xc;
  auto load_x = [&](int k0, int slot, bool async) {
    const bool in_k = k0 + 8 * xc < w.K;
    const uint32_t at = slot * L::kX + x_at;
#pragma unroll
    for (int u = 0; u < N / 8; ++u) {
      if (n0 + xr + 8 * u >= rows) break;
      const bf16* src = in_k ? x_row + (long long)(8 * u) * ldx + k0 : x;
      uint4* dst = reinterpret_cast<uint4*>(smem + at + u * 1024);
      if (vec && async) {
        cp16z(base + at + u * 1024, src, in_k ? 16 : 0);
      } else if (vec) {
        *dst = in_k ? *reinterpret_cast<const uint4*>(src) : make_uint4(0u, 0u, 0u, 0u);
      } else {
        uint32_t v[4] = {0u, 0u, 0u, 0u};
        if (in_k) {
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
  int mt = b0 / w.kt, kb = b0 - mt * w.kt;  // of the block whose products are to be read next
  int next_kb = kb;                         // of the block to be asked for next
#pragma unroll
  for (int u = 0; u < S - 1; ++u) {
    if (b0 + u < b1) load_codes(next_block, u);
    next_block += w.block_bytes;
    cp_commit();
  }
  if (tid == 0) {
    mbar_init(&mma_done, 1);
    fence_barrier_init();
  }
  if (warp == 0) {
    tmem_alloc(&tmem_slot, run.columns);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot, tA = tmem, tD = tmem + 64;
  pdl_launch();
  pdl_wait();
#pragma unroll
  for (int u = 0; u < S - 1; ++u) {
    if (b0 + u < b1) load_x(next_kb * kW4Tile, u, false);
    if (++next_kb == w.kt) next_kb = 0;
  }

  float acc[NR];
#pragma unroll
  for (int n = 0; n < NR; ++n) acc[n] = 0.f;
  const int groups = w.groups(), groups32 = w.group / 32;
  const int zero_at = kW4Codes + groups * kW4Tile * (w.scale_f32 ? 4 : 2);
  constexpr uint32_t idesc = idesc_bf16_f32(128, N);
  bool timed_out = false;
  uint32_t drain_parity = 0;

  int slot = 0, before = S - 1;  // stages of block i and of block i - 1 (the one to fill)
  for (int i = b0; i <= b1; ++i) {
    cp_wait<S - 2>();
    fence_proxy_async_smem();
    if (i > b0) {
      // The products of block i - 1: this thread's row of each group's sums.
      drain_parity = (uint32_t)(i - 1 - b0) & 1u;
      const bool ok = mbar_wait(&mma_done, drain_parity, run.wait_ns);
      if (__syncthreads_or(!ok)) {
        timed_out = true;
        break;
      }
      tc_fence_after();
      const uint8_t* blk = smem + codes_base + before * w.block_bytes + kW4Codes;
      const uint32_t row = tD + ((uint32_t)(32 * warp) << 16);
      for (int gi = 0; gi < groups; ++gi) {
        const float s = w.scale_f32 ? reinterpret_cast<const float*>(blk)[gi * kW4Tile + tid]
                                    : to_f<bf16>(reinterpret_cast<const bf16*>(blk)[gi * kW4Tile + tid]);
        if constexpr (NR == 8) {
          uint32_t d[8];
          tmem_ld8u(row + gi * N, d);
          tmem_ld_wait();
#pragma unroll
          for (int n = 0; n < 8; ++n) acc[n] = fmaf(s, __uint_as_float(d[n]), acc[n]);
        } else if constexpr (NR <= 32) {
#pragma unroll
          for (int c = 0; c < NR; c += 16) {
            uint32_t d[16];
            tmem_ld16u(row + gi * N + c, d);
            tmem_ld_wait();
#pragma unroll
            for (int n = 0; n < 16; ++n) acc[c + n] = fmaf(s, __uint_as_float(d[n]), acc[c + n]);
          }
        } else {
#pragma unroll
          for (int c = 0; c < NR; c += 32) {
            uint32_t d[32];
            tmem_ld32(row + gi * N + c, d);
            tmem_ld_wait();
#pragma unroll
            for (int n = 0; n < 32; ++n) acc[c + n] = fmaf(s, __uint_as_float(d[n]), acc[c + n]);
          }
        }
      }
      tc_fence_before();
      const int tile = mt;
      const bool tile_end = ++kb == w.kt;
      if (tile_end) {
        kb = 0;
        ++mt;
      }
      if (tile_end || i == b1) {
        // The row block ends here, or the run does.
        const int t0 = tile * w.kt, first_run = t0 / run.per, last_run = (t0 + w.kt - 1) / run.per;
        bool done = true;
        if (last_run > first_run) {
          // run r's piece of the row block: its first slot if the run begins in the block, else its second
          auto piece = [&](int r) {
            return reinterpret_cast<float4*>(run.part + (((long long)blockIdx.y * run.runs + r) * 2 + (r * run.per < t0)) *
                                                            (kW4Tile * NR)) + tid;
          };
          float4* own = piece(blockIdx.x);
#pragma unroll
          for (int v = 0; v < NR / 4; ++v)
            __stcg(own + v * kThreads, make_float4(acc[4 * v], acc[4 * v + 1], acc[4 * v + 2], acc[4 * v + 3]));
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
            constexpr int kV = NR == 8 ? 2 : 4, kAhead = 4;
#pragma unroll
            for (int v0 = 0; v0 < NR / 4; v0 += kV) {
              float sum[4 * kV];
#pragma unroll
              for (int e = 0; e < 4 * kV; ++e) sum[e] = 0.f;
              for (int r = first_run; r <= last_run; r += kAhead) {
                float4 p[kAhead][kV];
#pragma unroll
                for (int u = 0; u < kAhead; ++u) {
                  const float4* src = piece(min(r + u, last_run)) + v0 * kThreads;
#pragma unroll
                  for (int v = 0; v < kV; ++v) p[u][v] = __ldcg(src + v * kThreads);
                }
#pragma unroll
                for (int u = 0; u < kAhead; ++u)
                  if (r + u <= last_run) {
#pragma unroll
                    for (int v = 0; v < kV; ++v) {
                      sum[4 * v] += p[u][v].x;
                      sum[4 * v + 1] += p[u][v].y;
                      sum[4 * v + 2] += p[u][v].z;
                      sum[4 * v + 3] += p[u][v].w;
                    }
                  }
              }
#pragma unroll
              for (int e = 0; e < 4 * kV; ++e) acc[4 * v0 + e] = sum[e];
            }
          }
        }
        if (done) {
          const int m = tile * kW4Tile + tid;
          const bool live = m < w.M;
#pragma unroll
          for (int c = 0; c < NR; c += 8) {
            float add[8];
#pragma unroll
            for (int n = 0; n < 8; ++n)
              add[n] = epi.add && live && n0 + c + n < rows ? epi.add[(long long)(n0 + c + n) * w.M + m] : 0.f;
#pragma unroll
            for (int n = 0; n < 8; ++n) {
              const long long at = n0 + c + n;
              const float v = fmaf(acc[c + n], kUnit, add[n]);
              if (epi.swiglu) {
                const float up = __shfl_down_sync(0xffffffffu, v, 1);
                if (live && !(m & 1) && at < rows)
                  reinterpret_cast<bf16*>(epi.out)[at * (w.M / 2) + m / 2] = from_f<bf16>(v / (1.f + expf(-v)) * up);
              } else if (live && at < rows) {
                reinterpret_cast<float*>(epi.out)[at * w.M + m] = v;
              }
            }
          }
        }
#pragma unroll
        for (int n = 0; n < NR; ++n) acc[n] = 0.f;
      }
    }
    if (i == b1) break;
    __syncthreads();  // block i is there for all, and nobody needs block i - 1 any more
    if (i + S - 1 < b1) {
      load_codes(next_block, before);
      load_x(next_kb * kW4Tile, before, true);
      next_block += w.block_bytes;
      if (++next_kb == w.kt) next_kb = 0;
    }
    cp_commit();
    // Codes to bf16, into TMEM: 32 rows a warp.
    const uint8_t* blk = smem + codes_base + slot * w.block_bytes;
#pragma unroll
    for (int y = 0; y < 2; ++y) {
      uint32_t a[32];
      uint32_t off0 = offset_of(kW4Zero), off1 = off0;
      const uint4 w0 = *reinterpret_cast<const uint4*>(blk + w4_word_at(2 * warp + y, 0, lane));
      const uint4 w1 = *reinterpret_cast<const uint4*>(blk + w4_word_at(2 * warp + y, 1, lane));
#pragma unroll
      for (int q = 0; q < 4; ++q) {  // 32 columns: steps 2 q and 2 q + 1
        if (w.zeros && (q & (groups32 - 1)) == 0) {
          const uint8_t* z = blk + zero_at + q / groups32 * kW4Tile + 32 * warp + 16 * y + g;
          off0 = offset_of(z[0]);
          off1 = offset_of(z[8]);
        }
        const uint32_t lo = q == 0 ? w0.x : q == 1 ? w0.y : q == 2 ? w1.x : w1.y;
        const uint32_t hi = q == 0 ? w0.z : q == 1 ? w0.w : q == 2 ? w1.z : w1.w;
        a[8 * q] = pair_of<0>(lo, off0);
        a[8 * q + 1] = pair_of<0>(hi, off1);
        a[8 * q + 2] = pair_of<1>(lo, off0);
        a[8 * q + 3] = pair_of<1>(hi, off1);
        a[8 * q + 4] = pair_of<0>(lo >> 8, off0);
        a[8 * q + 5] = pair_of<0>(hi >> 8, off1);
        a[8 * q + 6] = pair_of<1>(lo >> 8, off0);
        a[8 * q + 7] = pair_of<1>(hi >> 8, off1);
      }
      tmem_st_16x128b_x16(tA + ((uint32_t)(32 * warp + 16 * y) << 16), a);
    }
    tmem_st_wait();
    tc_fence_before();
    __syncthreads();
    if (warp == 0 && elect_one()) {
      tc_fence_after();
      const uint64_t xd = smem_desc_sw128(smem + slot * L::kX);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int q = k >> 1;
        tc_mma_f16_tmem_a(tD + q / groups32 * N, tA + 8 * k, xd + (uint64_t)((k >> 2) * (N * 128 / 16) + 2 * (k & 3)), idesc,
                          (k & 1) != 0 || (q & (groups32 - 1)) != 0);
      }
      tc_commit(&mma_done);
    }
    __syncwarp();
    before = slot;
    if (++slot == S) slot = 0;
  }
  cp_wait<0>();
  if (timed_out) {  // (the same for all threads)
    if (tid == 0) set_status(run.status, DFLASH_STATUS_TIMEOUT);
    mbar_wait(&mma_done, drain_parity, kDrainNs);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, run.columns);
  }
}

namespace {
constexpr int kRunsPerSm = 4;
constexpr int kMinRun = 4;  // blocks of a run at least

template <int N, int NR>
cudaError_t tc_launch(const W4View& w, const bf16* x, long long ldx, int rows, const W4Epi& epi, const W4Scratch& sc,
                      cudaStream_t s) {
  typedef TcLayout<N, NR> L;
  static PerDevice attr;
  // (the widest block: groups of 32, float32 scales and zero points)
  constexpr int kMost = 1024 + L::kStages * (kW4Codes + 4 * kW4Tile * 5 + L::kX);
  static_assert(kMost <= 232448 - 1024, "shared memory per block");
  DFL_RET(attr.once([] {
    return cudaFuncSetAttribute(w4_tc_kernel<N, NR>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMost);
  }));
  const int vec = (reinterpret_cast<uintptr_t>(x) & 15) == 0 && ldx % 8 == 0;
  W4Run run;
  run.blocks = (w.M + kW4Tile - 1) / kW4Tile * w.kt;
  run.per = w4_run_blocks(w);
  run.runs = (run.blocks + run.per - 1) / run.per;
  run.part = sc.part;
  run.tickets = sc.tickets;
  run.status = sc.status;
  run.wait_ns = wait_limit_ns();
  run.columns = 128;
  while (run.columns < 64u + N * w.groups()) run.columns *= 2;
  const dim3 grid(run.runs, (rows + N - 1) / N);
  DFL_RET(launch_pdl(w4_tc_kernel<N, NR>, grid, dim3(kThreads), 1024 + L::kStages * (w.block_bytes + L::kX), s, w, run, x,
                     ldx, vec, rows, epi));
  count_launch();
  return cudaSuccess;
}
}  // namespace

int w4_run_blocks(const W4View& w) {
  const int blocks = (w.M + kW4Tile - 1) / kW4Tile * w.kt, most = num_sms() * kRunsPerSm;
  return std::max(kMinRun, (blocks + most - 1) / most);
}
int w4_max_runs() { return num_sms() * kRunsPerSm; }

cudaError_t w4_linear_tc(const W4View& w, const void* x, long long ldx, int rows, const W4Epi& epi, const W4Scratch& sc,
                         cudaStream_t s) {
  const bf16* b = (const bf16*)x;
  if (rows <= 8) return tc_launch<16, 8>(w, b, ldx, rows, epi, sc, s);
  if (rows <= 16) return tc_launch<16, 16>(w, b, ldx, rows, epi, sc, s);
  if (rows <= 32) return tc_launch<32, 32>(w, b, ldx, rows, epi, sc, s);
  // (128 columns for each of four groups do not fit TMEM beside the weights: two passes)
  if (rows <= 64 || w.groups() == 4) return tc_launch<64, 64>(w, b, ldx, rows, epi, sc, s);
  return tc_launch<128, 128>(w, b, ldx, rows, epi, sc, s);
}

}  // namespace dfl
