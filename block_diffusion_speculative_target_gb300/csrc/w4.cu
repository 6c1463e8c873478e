// Weights in 4 bits: packing, quantising, reading back, and the product on the
// CUDA cores.
#include "w4.cuh"

#include <algorithm>

#include "internal.h"

namespace dfl {

namespace {
constexpr int kPackWarps = 8;

template <typename S>
__device__ __forceinline__ void put_scale(const W4View& w, uint8_t* block, int gi, int r, S s) {
  if (w.scale_f32)
    reinterpret_cast<float*>(block + kW4Codes)[gi * kW4Tile + r] = to_f<S>(s);
  else
    reinterpret_cast<bf16*>(block + kW4Codes)[gi * kW4Tile + r] = from_f<bf16>(to_f<S>(s));
}
__device__ __forceinline__ void put_zero(const W4View& w, uint8_t* block, int gi, int r, int z) {
  if (w.zeros)
    block[kW4Codes + w.groups() * kW4Tile * (w.scale_f32 ? 4 : 2) + gi * kW4Tile + r] = (uint8_t)z;
}
// Whether this lane keeps the scale and zero point of group gi of its two rows: one of a row's four lanes does.
__device__ __forceinline__ bool keeps(int lane, int gi) { return (lane & 3) == (gi & 3); }

// The warp's place: a block and 16 of its rows.
struct WarpTile {
  int mt, k, mi;
  bool live;
};
__device__ __forceinline__ WarpTile warp_tile(const W4View& w) {
  const long long i = (long long)blockIdx.x * kPackWarps + (threadIdx.x >> 5);
  WarpTile t;
  t.mi = (int)(i & 7);
  const long long b = i >> 3;
  t.mt = (int)(b / w.kt);
  t.k = (int)(b - (long long)t.mt * w.kt);
  t.live = t.mt < (w.M + kW4Tile - 1) / kW4Tile;
  return t;
}
unsigned warp_tiles(const W4View& w) {
  return (unsigned)(((long long)((w.M + kW4Tile - 1) / kW4Tile) * w.kt * 8 + kPackWarps - 1) / kPackWarps);
}
}  // namespace

// Products read weights ahead of their own wait for the kernels before them, by bulk copies.  So packing and quantising
// do not let the next kernel start before their end, and each thread makes its stores visible to such copies before
// its own: a kernel that starts behind the trigger which the end raises has, before its wait, no other promise of that.
__device__ __forceinline__ void publish() {
  __threadfence();
  asm volatile("fence.proxy.async;" ::: "memory");
}
// Codes [M][K / 2] (even column in the low half of a byte), scales and zeros [M][K / group].
template <typename S>
__global__ void __launch_bounds__(kPackWarps * 32)
    w4_pack_kernel(const __grid_constant__ W4View w, const uint8_t* __restrict__ codes, const S* __restrict__ scales,
                   const uint8_t* __restrict__ zeros) {
  pdl_wait();
  const WarpTile t = warp_tile(w);
  if (!t.live) return;
  const int lane = threadIdx.x & 31;
  uint8_t* block = const_cast<uint8_t*>(w.block(t.mt, t.k));
  for (int h = 0; h < 2; ++h) {
    uint4 v;
    uint32_t* word = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const long long m = (long long)t.mt * kW4Tile + w4_row(t.mi, lane, x);
      word[x] = 0x11111111u * kW4Zero;
      if (m < w.M) {
#pragma unroll
        for (int p = 0; p < 4; ++p) {
          const int k = t.k * kW4Tile + w4_col(h, lane, x, p);
          if (k < w.K) {
            const uint32_t c = codes[m * (w.K / 2) + k / 2];
            word[x] &= ~(0x000F000Fu << (4 * p));
            word[x] |= ((c & 15u) | (c >> 4) << 16) << (4 * p);
          }
        }
      }
    }
    *reinterpret_cast<uint4*>(block + w4_word_at(t.mi, h, lane)) = v;
  }
  const int groups = w.K / w.group;
  for (int gi = 0; gi < w.groups(); ++gi) {
    if (!keeps(lane, gi)) continue;
    for (int y = 0; y < 2; ++y) {
      const int r = w4_row(t.mi, lane, 2 * y);
      const long long m = (long long)t.mt * kW4Tile + r, g = (long long)t.k * w.groups() + gi;
      const bool in = m < w.M && g < groups;
      put_scale<S>(w, block, gi, r, in ? scales[m * groups + g] : from_f<S>(0.f));
      put_zero(w, block, gi, r, in && zeros ? min((int)zeros[m * groups + g], 15) : kW4Zero);
    }
  }
  publish();
}

cudaError_t w4_pack(const W4View& w, const uint8_t* codes, const void* scales, const uint8_t* zeros, cudaStream_t s) {
  const dim3 grid(warp_tiles(w)), block(kPackWarps * 32);
  if (w.scale_f32)
    DFL_RET(launch_pdl(w4_pack_kernel<float>, grid, block, 0, s, w, codes, (const float*)scales, zeros));
  else
    DFL_RET(launch_pdl(w4_pack_kernel<bf16>, grid, block, 0, s, w, codes, (const bf16*)scales, zeros));
  count_launch();
  return cudaSuccess;
}

// Nearest codes of a matrix.  Without zeros s = max|w| / 7 and code = rhe(w / s) + 8, with them, the range
// stretched to hold 0, s = (max - min) / 15, z = rhe(-min / s), code = rhe(w / s) + z; s is rounded to the scale
// type before it divides, and codes are clamped to 0..15.  A lane holds 8 columns of a row in a step of 32.
template <typename T>
__global__ void __launch_bounds__(kPackWarps * 32)
    w4_quantize_kernel(const __grid_constant__ W4View w, const T* __restrict__ src, long long ld) {
  pdl_wait();
  const WarpTile t = warp_tile(w);
  if (!t.live) return;
  const int lane = threadIdx.x & 31, steps = w.group / 32;
  uint8_t* block = const_cast<uint8_t*>(w.block(t.mt, t.k));
  for (int y = 0; y < 2; ++y) {
    const int r = w4_row(t.mi, lane, 2 * y);
    const long long m = (long long)t.mt * kW4Tile + r;
    for (int gi = 0; gi < w.groups(); ++gi) {
      float x[4][8], hi = 0.f, lo = 0.f;
#pragma unroll
      for (int st = 0; st < 4; ++st) {
        if (st >= steps) break;
        const int step = gi * steps + st;  // of 32 columns: word step % 2 of half step / 2
#pragma unroll
        for (int p = 0; p < 4; ++p) {
          const int k = t.k * kW4Tile + w4_col(step >> 1, lane, step & 1, p);
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float v = m < w.M && k < w.K ? to_f<T>(src[m * ld + k + e]) : 0.f;
            x[st][2 * p + e] = v;
            hi = fmaxf(hi, v);
            lo = fminf(lo, v);
          }
        }
      }
#pragma unroll
      for (int o = 1; o < 4; o <<= 1) {
        hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
        lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
      }
      float s = w.zeros ? __fdiv_rn(hi - lo, 15.f) : __fdiv_rn(fmaxf(hi, -lo), 7.f);
      // (a range past float32: its fifteenth is not)
      if (w.zeros && hi - lo == INFINITY) s = (float)(((double)hi - (double)lo) / 15.0);
      if (!w.scale_f32) s = to_f<bf16>(from_f<bf16>(s));
      const int z = w.zeros && s > 0.f ? (int)fminf(fmaxf(rintf(__fdiv_rn(-lo, s)), 0.f), 15.f) : kW4Zero;
      if (keeps(lane, gi)) {
        put_scale<float>(w, block, gi, r, s);
        put_zero(w, block, gi, r, z);
      }
#pragma unroll
      for (int st = 0; st < 4; ++st) {
        if (st >= steps) break;
        const int step = gi * steps + st;
        uint32_t word = 0;
#pragma unroll
        for (int p = 0; p < 4; ++p)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            // (a value that is no number takes the zero point)
            const float q = s > 0.f ? rintf(__fdiv_rn(x[st][2 * p + e], s)) : 0.f;
            const int c = q == q ? (int)fminf(fmaxf(q + (float)z, 0.f), 15.f) : z;
            word |= (uint32_t)c << (4 * p + 16 * e);
          }
        reinterpret_cast<uint32_t*>(block + w4_word_at(t.mi, step >> 1, lane))[2 * y + (step & 1)] = word;
      }
    }
  }
  publish();
}

cudaError_t w4_quantize(const W4View& w, int dtype, const void* src, long long ld, cudaStream_t s) {
  const dim3 grid(warp_tiles(w)), block(kPackWarps * 32);
  if (dtype == DFLASH_F32)
    DFL_RET(launch_pdl(w4_quantize_kernel<float>, grid, block, 0, s, w, (const float*)src, ld));
  else
    DFL_RET(launch_pdl(w4_quantize_kernel<bf16>, grid, block, 0, s, w, (const bf16*)src, ld));
  count_launch();
  return cudaSuccess;
}

// The values (code - zero) scale, rounded once to T.
template <typename T>
__global__ void __launch_bounds__(kPackWarps * 32)
    w4_unpack_kernel(const __grid_constant__ W4View w, T* __restrict__ dst) {
  pdl_launch();
  pdl_wait();
  const WarpTile t = warp_tile(w);
  if (!t.live) return;
  const int lane = threadIdx.x & 31;
  const uint8_t* block = w.block(t.mt, t.k);
  for (int h = 0; h < 2; ++h) {
    const uint4 v = *reinterpret_cast<const uint4*>(block + w4_word_at(t.mi, h, lane));
    const uint32_t* word = reinterpret_cast<const uint32_t*>(&v);
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const int r = w4_row(t.mi, lane, x);
      const long long m = (long long)t.mt * kW4Tile + r;
      if (m >= w.M) continue;
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        const int c = w4_col(h, lane, x, p), k = t.k * kW4Tile + c;
        if (k >= w.K) continue;
        const float s = w4_scale(w, block, c / w.group, r);
        const int z = w4_zero(w, block, c / w.group, r);
#pragma unroll
        for (int e = 0; e < 2; ++e)
          dst[m * w.K + k + e] = from_f<T>((float)((int)(word[x] >> (4 * p + 16 * e) & 15u) - z) * s);
      }
    }
  }
}

cudaError_t w4_unpack(const W4View& w, int dtype, void* dst, cudaStream_t s) {
  const dim3 grid(warp_tiles(w)), block(kPackWarps * 32);
  if (dtype == DFLASH_F32)
    DFL_RET(launch_pdl(w4_unpack_kernel<float>, grid, block, 0, s, w, (float*)dst));
  else
    DFL_RET(launch_pdl(w4_unpack_kernel<bf16>, grid, block, 0, s, w, (bf16*)dst));
  count_launch();
  return cudaSuccess;
}

// ------------------------------------------------------------------ split
constexpr int kMmaRuns = 4, kTcRuns = 1;  // runs an SM at most, up to kW4MmaRows rows and beyond
constexpr int kMinRun = 4;  // blocks of a run at least
static int runs_of(int rows) { return num_sms() * (rows <= kW4MmaRows ? kMmaRuns : kTcRuns); }
static int padded(int rows) {
  int n = 8;
  while (n < rows) n *= 2;
  return n;
}
int w4_max_runs() { return num_sms() * std::max(kMmaRuns, kTcRuns); }
size_t w4_part_floats(int max_rows) {
  const int few = std::min(max_rows, kW4MmaRows);
  const size_t rows = std::max((long long)runs_of(few) * padded(few), (long long)runs_of(max_rows) * padded(max_rows));
  return rows * 2 * kW4Tile;
}
W4Run w4_run(const W4View& w, const W4Scratch& sc, int rows) {
  const int blocks = (w.M + kW4Tile - 1) / kW4Tile * w.kt, most = runs_of(rows);
  const int per = std::max(kMinRun, (blocks + most - 1) / most);
  return W4Run{blocks, per, (blocks + per - 1) / per, sc.part, sc.tickets, sc.status, wait_limit_ns()};
}

// ------------------------------------------------------------------ product on the CUDA cores
// A block takes 64 weight rows and 16 rows of x and walks the columns 128 at a
// time: the codes become float32 values in shared memory (code - zero times
// scale: 2^-24 relative), a thread sums two weight rows (2 f, 2 f + 1: the pair
// of the activation) by two rows of x, in the order of the columns, 128 at a time
// so that rounding errors grow with the number of blocks and not of columns.
constexpr int kCoreN = 16, kCoreM = 64;

__global__ void __launch_bounds__(256)
    w4_core_kernel(const __grid_constant__ W4View w, const float* __restrict__ x, long long ldx, int rows,
                   const __grid_constant__ W4Epi epi) {
  __shared__ float ws[kCoreM][kW4Tile + 1];
  __shared__ float xs[kCoreN][kW4Tile + 1];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int mp = tid & 31, np = tid >> 5;
  const int m0 = blockIdx.x * kCoreM, n0 = blockIdx.y * kCoreN;
  const int mt = m0 / kW4Tile, mi0 = (m0 % kW4Tile) / 16;
  float acc[2][2] = {{0.f, 0.f}, {0.f, 0.f}};
  pdl_launch();
  pdl_wait();
  for (int k = 0; k < w.kt; ++k) {
    const uint8_t* block = w.block(mt, k);
    __syncthreads();
    {  // 8 warps: 4 times 16 rows by 2 halves
      const int mi = warp >> 1, h = warp & 1;
      const uint4 v = *reinterpret_cast<const uint4*>(block + w4_word_at(mi0 + mi, h, lane));
      const uint32_t* word = reinterpret_cast<const uint32_t*>(&v);
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        const int r = w4_row(mi, lane, y);
#pragma unroll
        for (int p = 0; p < 4; ++p) {
          const int c = w4_col(h, lane, y, p), gi = c / w.group;
          const float s = w4_scale(w, block, gi, mi0 * 16 + r);
          const int z = w4_zero(w, block, gi, mi0 * 16 + r);
          ws[r][c] = (float)((int)(word[y] >> (4 * p) & 15u) - z) * s;
          ws[r][c + 1] = (float)((int)(word[y] >> (4 * p + 16) & 15u) - z) * s;
        }
      }
    }
    for (int i = tid; i < kCoreN * kW4Tile; i += 256) {
      const int r = i / kW4Tile, c = i % kW4Tile, kk = k * kW4Tile + c;
      xs[r][c] = n0 + r < rows && kk < w.K ? x[(n0 + r) * ldx + kk] : 0.f;
    }
    __syncthreads();
    float part[2][2] = {{0.f, 0.f}, {0.f, 0.f}};
#pragma unroll 8
    for (int c = 0; c < kW4Tile; ++c) {
      const float w0 = ws[2 * mp][c], w1 = ws[2 * mp + 1][c];
      const float x0 = xs[2 * np][c], x1 = xs[2 * np + 1][c];
      part[0][0] = fmaf(x0, w0, part[0][0]);
      part[0][1] = fmaf(x0, w1, part[0][1]);
      part[1][0] = fmaf(x1, w0, part[1][0]);
      part[1][1] = fmaf(x1, w1, part[1][1]);
    }
#pragma unroll
    for (int a = 0; a < 4; ++a) acc[a >> 1][a & 1] += part[a >> 1][a & 1];
  }
#pragma unroll
  for (int a = 0; a < 2; ++a) {
    const long long n = n0 + 2 * np + a;
    const int m = m0 + 2 * mp;
    if (n >= rows || m >= w.M) continue;
    float y0 = acc[a][0], y1 = acc[a][1];
    if (epi.add) {
      y0 += epi.add[n * w.M + m];
      if (m + 1 < w.M) y1 += epi.add[n * w.M + m + 1];
    }
    if (epi.swiglu) {
      reinterpret_cast<float*>(epi.out)[n * (w.M / 2) + m / 2] = y0 / (1.f + expf(-y0)) * y1;
    } else {
      float* out = reinterpret_cast<float*>(epi.out) + n * w.M + m;
      out[0] = y0;
      if (m + 1 < w.M) out[1] = y1;
    }
  }
}

cudaError_t w4_linear_core(const W4View& w, const void* x, long long ldx, int rows, const W4Epi& epi, cudaStream_t s) {
  const dim3 grid((w.M + kCoreM - 1) / kCoreM, (rows + kCoreN - 1) / kCoreN);
  DFL_RET(launch_pdl(w4_core_kernel, grid, dim3(256), 0, s, w, (const float*)x, ldx, rows, epi));
  count_launch();
  return cudaSuccess;
}

}  // namespace dfl
