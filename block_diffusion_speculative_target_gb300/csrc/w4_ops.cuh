// What the tensor-core products with 4-bit weights share: copies, codes to bf16,
// and the end of a row block (joining its pieces, writing its results).
#pragma once
#include "common.cuh"
#include "w4.cuh"

namespace dfl {

constexpr uint64_t kW4DrainNs = 125000000ull;  // for copies and products in flight after a wait that ran out

// `bytes` of 16 (0: none is read), the rest zeros
__device__ __forceinline__ void cp16z(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
// 8 values of x at any alignment, or zeros.
__device__ __forceinline__ uint4 gather8(const bf16* src, bool in) {
  uint32_t v[4] = {0u, 0u, 0u, 0u};
  if (in) {
    const uint16_t* h = reinterpret_cast<const uint16_t*>(src);
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = h[2 * e] | (uint32_t)h[2 * e + 1] << 16;
  }
  return make_uint4(v[0], v[1], v[2], v[3]);
}
// A phase is complete, waited for up to the limit (0: it has expired).  Asked once by itself first: 50 cycles
// where the phase is over, and 100 to 290 through the loop.
__device__ __forceinline__ bool landed(uint64_t* bar, uint32_t parity, uint64_t limit_ns) {
  if (limit_ns != 0 && mbar_try_wait(bar, parity)) return true;
  return mbar_wait(bar, parity, limit_ns);
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
constexpr float kW4Unit = 64.f;
__device__ __forceinline__ uint32_t offset_of(int zero) {
  const __nv_bfloat162 v = __float2bfloat162_rn((float)zero * (-1.f / kW4Unit));
  return *reinterpret_cast<const uint32_t*>(&v);
}

// One warp's share of the row block `tile`, whose last column that this run holds has been added: V float4 of sums a
// thread.  Where other runs hold some of its columns, the sums are left for whoever comes last, who adds the pieces in
// order of the columns.  That warp, or the only one, has `emit(v0, sums)` called with kV float4 of whole sums at a time.
template <int V, int kV, typename F>
__device__ __forceinline__ void w4_join(const W4View& w, const W4Run& run, int tile, int tid, const float (&acc)[V][4],
                                        F emit) {
  const int t0 = tile * w.kt, first = t0 / run.per, last = (t0 + w.kt - 1) / run.per;
  if (first == last) {
#pragma unroll
    for (int v0 = 0; v0 < V; v0 += kV) {
      float sum[kV][4];
#pragma unroll
      for (int v = 0; v < kV; ++v)
#pragma unroll
        for (int e = 0; e < 4; ++e) sum[v][e] = acc[v0 + v][e];
      emit(v0, sum);
    }
    return;
  }
  // run r's piece of the row block: its first slot if the run begins in the block, else its second
  auto piece = [&](int r) {
    return reinterpret_cast<float4*>(run.part) + ((long long)r * 2 + (r * run.per < t0)) * (V * kW4Tile) + tid;
  };
  float4* own = piece(blockIdx.x);
#pragma unroll
  for (int v = 0; v < V; ++v) __stcg(own + v * kW4Tile, make_float4(acc[v][0], acc[v][1], acc[v][2], acc[v][3]));
  __threadfence();
  __syncwarp();
  int ends = 0;
  if ((tid & 31) == 0) {
    int* ticket = run.tickets + first * 4 + (tid >> 5);
    ends = atomicAdd(ticket, 1) == last - first;
    if (ends) *ticket = 0;
  }
  if (!__shfl_sync(0xffffffffu, ends, 0)) return;
  __threadfence();
  constexpr int kAhead = V <= 4 ? 4 : 6;  // pieces in flight
#pragma unroll 1
  for (int v0 = 0; v0 < V; v0 += kV) {
    float sum[kV][4];
#pragma unroll
    for (int v = 0; v < kV; ++v)
#pragma unroll
      for (int e = 0; e < 4; ++e) sum[v][e] = 0.f;
#pragma unroll 1
    for (int r = first; r <= last; r += kAhead) {
      float4 p[kAhead][kV];
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const float4* src = piece(min(r + u, last)) + v0 * kW4Tile;
#pragma unroll
        for (int v = 0; v < kV; ++v) p[u][v] = __ldcg(src + v * kW4Tile);
      }
#pragma unroll
      for (int u = 0; u < kAhead; ++u)
        if (r + u <= last) {
#pragma unroll
          for (int v = 0; v < kV; ++v) {
            sum[v][0] += p[u][v].x;
            sum[v][1] += p[u][v].y;
            sum[v][2] += p[u][v].z;
            sum[v][3] += p[u][v].w;
          }
        }
    }
    emit(v0, sum);
  }
}

// A warp's results: the whole sums of row `lane` of its 32 rows (of the matrix's from m0 on) and row n of x at
// sums[n * kW4SumRow + lane] in shared memory, n < count <= 16, for the rows n0 + n of x.  Rolled: the code is run once
// a row block, and fetching it unrolled takes as long as running it.  But what is added is asked for all at once: in
// fours, 128 rows waited 32 times for memory (4096 x 12288: 61 us instead of 52).
constexpr int kW4SumRow = 36;  // (a fragment's 8 rows by 4 column pairs fall into 32 banks)
__device__ __forceinline__ void w4_results(const W4View& w, const W4Epi& epi, int m0, float* sums, int n0,
                                           int count) {
  const int lane = threadIdx.x & 31, m = m0 + lane;
  const bool live = m < w.M;
  float unit = kW4Unit;
  if (epi.add) {
    const float* src = epi.add + (long long)n0 * w.M + m;
    float a[16];
#pragma unroll
    for (int n = 0; n < 16; ++n) a[n] = live && n < count ? src[(long long)n * w.M] : 0.f;
#pragma unroll
    for (int n = 0; n < 16; ++n)
      if (n < count) sums[n * kW4SumRow + lane] = fmaf(sums[n * kW4SumRow + lane], kW4Unit, a[n]);
    unit = 1.f;
  }
  constexpr int U = 4;
#pragma unroll 1
  for (int c = 0; c < count; c += U) {
    float v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      v[u] = sums[(c + u) * kW4SumRow + lane] * unit;
      const long long n = n0 + c + u;
      if (epi.swiglu) {  // (row m + 1 is the next lane's)
        const float up = __shfl_down_sync(0xffffffffu, v[u], 1);
        // (both sides of the quotient by 1/4: the fast division is 0 where the divisor is past 2^126, v below -87.3)
        if (live && !(m & 1) && c + u < count)
          reinterpret_cast<bf16*>(epi.out)[n * (w.M / 2) + m / 2] =
              from_f<bf16>(__fdividef(0.25f * v[u], fmaf(0.25f, __expf(-v[u]), 0.25f)) * up);
      } else if (live && c + u < count) {
        reinterpret_cast<float*>(epi.out)[n * w.M + m] = v[u];
      }
    }
  }
}

}  // namespace dfl
