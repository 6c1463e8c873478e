// 8-bit KV pages: the append that quantises, and the read that brings rows back
// (8-bit pages and pages of the model's type).
#include <algorithm>

#include "common.cuh"
#include "internal.h"
#include "paged.cuh"

namespace dfl {

namespace {
// 8 entries as they lie in memory.
template <typename T>
struct Row8 {
  uint4 v[sizeof(T) / 2];
};
template <typename T>
__device__ __forceinline__ Row8<T> fetch8(const T* p, bool vec) {
  Row8<T> r;
  if (vec) {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) r.v[i] = *(reinterpret_cast<const uint4*>(p) + i);
  } else {
    T x[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = p[e];
    memcpy(&r, x, sizeof(r));
  }
  return r;
}
__device__ __forceinline__ void values8(const Row8<float>& r, float (&x)[8]) { memcpy(x, &r, sizeof(r)); }
__device__ __forceinline__ void values8(const Row8<bf16>& r, float (&x)[8]) {
  const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&r);
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float2 f = __bfloat1622float2(h[e]);
    x[2 * e] = f.x;
    x[2 * e + 1] = f.y;
  }
}
// N values of an output row, 16 bytes at a time (8 bf16 or 4 float32).
template <typename T, int N>
__device__ __forceinline__ void put(T* p, const float (&x)[N]) {
  if (sizeof(T) == 4) {
#pragma unroll
    for (int e = 0; e < N; e += 4)
      *reinterpret_cast<float4*>(p + e) = make_float4(x[e], x[e + 1], x[e + 2], x[e + 3]);
  } else {
#pragma unroll
    for (int c = 0; c < N; c += 8) {
      uint4 v;
      __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&v);
#pragma unroll
      for (int e = 0; e < 4; ++e) h[e] = __floats2bfloat162_rn(x[c + 2 * e], x[c + 2 * e + 1]);
      *reinterpret_cast<uint4*>(p + c) = v;
    }
  }
}
// The codes of 8 entries, q + 128 with q = x / s rounded half to even (a row of zeros, or one that holds a value
// that is not finite: 128 everywhere).  r = 1 / s rounded.  A quotient is at most 127 (1 + 2^-22), so x r is within
// 127 2^-22 < 4e-5 of it and of the rounded quotient: where x r lies further than 1e-4 from a tie, its integer is
// theirs.  The others, and rows whose scale is below the normal numbers, are divided.  (With 16 divisions a thread
// they, not memory, were the bound: 16384 rows took 134 us where they then took 115.)
__device__ __forceinline__ uint2 codes8(const float (&x)[8], float s, float r) {
  if (!(s > 0.f)) return make_uint2(0x80808080u, 0x80808080u);
  // added to an integer below 2^22 in size: the sum's low byte is the integer + 128
  constexpr float kAt = 12582912.f + 128.f;
  uint32_t u[8];
  float far = 0.f;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float t = fmaf(x[e], r, kAt);
    u[e] = __float_as_uint(t);
    far = fmaxf(far, fabsf(fmaf(x[e], r, kAt - t)));
  }
  if (!(far < 0.4999f) || s < 1.17549435e-38f) {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      u[e] = (uint32_t)((int)fminf(fmaxf(rintf(__fdiv_rn(x[e], s)), -127.f), 127.f) + 128);
  }
  return make_uint2(__byte_perm(__byte_perm(u[0], u[1], 0x0040), __byte_perm(u[2], u[3], 0x0040), 0x5410),
                    __byte_perm(__byte_perm(u[4], u[5], 0x0040), __byte_perm(u[6], u[7], 0x0040), 0x5410));
}
}  // namespace

// ------------------------------------------------------------------ append
// As the append into pages of the model's type, with key and value rows leaving
// as 8-bit codes and a scale: s = max|x| / 127 over the row's rotated float32
// entries.  The rotation's products are not fused, so the codes are those of
// x_lo c - x_hi s with each operation rounded.  The hd / 16 threads of a head
// exchange their maxima; a thread moves 8 entries of the lower half and the 8
// they rotate with.
//
// Bound by its bytes in and out: 16384 bf16 rows of 40 + 8 + 8 heads of 128 and the
// rows read back take 109 us for 74 us of bytes, 95 of them here (4.6 TB/s in all).
// A thread has four heads' loads in flight where there are many rows; with bf16 rows
// three blocks a multiprocessor (80 registers, a few spilled) are faster than two
// (115 us), and two heads a thread no faster.  float32 rows need the registers.
template <typename TI, typename T, int HPT>
__global__ void __launch_bounds__(256, sizeof(TI) == 2 ? 3 : 2)
    paged_append_q8_kernel(const TI* __restrict__ qkv, long long ld, int vec, int rows, int n, int nq, int nkv, int hd,
                           int rpb, const int32_t* __restrict__ n_rows, const int32_t* __restrict__ table,
                           int table_stride, const int32_t* __restrict__ len, const float2* __restrict__ tab,
                           int max_pos, int n_pages, int ps_log2, long long page0, T* __restrict__ qout,
                           uint8_t* __restrict__ kp, uint8_t* __restrict__ vp, float* __restrict__ ks,
                           float* __restrict__ vs, int* status) {
  const int half = hd / 2, lanes = half / 8, heads = nq + 2 * nkv;
  const int groups = (heads + HPT - 1) / HPT;  // group hg takes heads hg, hg + groups, ..
  const int per_row = groups * lanes;
  const int r0 = blockIdx.x * rpb, items = min(rpb, rows - r0) * per_row;
  // the threads of this one's row and heads, which take every branch below together
  const unsigned mates = ((1u << lanes) - 1u) << (threadIdx.x & 31 & ~(lanes - 1));
  pdl_launch();
  pdl_wait();
  for (int t = threadIdx.x; t < items; t += 256) {
    const int rr = t / per_row, w = t - rr * per_row, r = r0 + rr;
    const int b = r / n, j = r - b * n;
    if (n_rows && j >= n_rows[b]) continue;
    const int hg = w / lanes, e = (w - hg * lanes) * 8;
    const TI* src = qkv + (long long)r * ld + e;
    Row8<TI> lo[HPT], hi[HPT];
#pragma unroll
    for (int x = 0; x < HPT; ++x) {
      const int h = hg + x * groups;
      if (h < heads) {
        lo[x] = fetch8<TI>(src + h * hd, vec);
        hi[x] = fetch8<TI>(src + h * hd + half, vec);
      }
    }
    const long long pos = (long long)len[b] + j;
    if (pos < 0 || pos >= max_pos || (pos >> ps_log2) >= table_stride) {
      if (w == 0) set_status(status, DFLASH_STATUS_CAPACITY);
      continue;
    }
    const int page = table[(long long)b * table_stride + (pos >> ps_log2)];
    const bool good = (unsigned)page < (unsigned)n_pages;
    if (!good && w == 0) set_status(status, DFLASH_STATUS_BOUNDS);
    const float4* cs = reinterpret_cast<const float4*>(tab + pos * half + e);
    float4 c[4];  // two (cos, sin) pairs each
#pragma unroll
    for (int x = 0; x < 4; ++x) c[x] = __ldg(cs + x);
    // slot (pos mod ps) of the page's first head
    const long long slot = (((page0 + page) * nkv) << ps_log2) + (pos & ((1 << ps_log2) - 1));
#pragma unroll
    for (int x = 0; x < HPT; ++x) {
      const int h = hg + x * groups;
      if (h >= heads) break;
      float a[8], z[8];
      values8(lo[x], a);
      values8(hi[x], z);
      if (h < nq + nkv) {
#pragma unroll
        for (int y = 0; y < 8; ++y) {
          const float cc = y & 1 ? c[y >> 1].z : c[y >> 1].x, ss = y & 1 ? c[y >> 1].w : c[y >> 1].y;
          const float a0 = a[y], z0 = z[y];
          a[y] = __fsub_rn(__fmul_rn(a0, cc), __fmul_rn(z0, ss));
          z[y] = __fadd_rn(__fmul_rn(z0, cc), __fmul_rn(a0, ss));
        }
      }
      if (h < nq) {
        T* dst = qout + ((long long)r * nq + h) * hd + e;
        put<T>(dst, a);
        put<T>(dst + half, z);
        continue;
      }
      if (!good) break;  // (heads ascend: keys and values only from here on)
      float most = 0.f;
      bool fine = true;
#pragma unroll
      for (int y = 0; y < 8; ++y) {
        most = fmaxf(most, fmaxf(fabsf(a[y]), fabsf(z[y])));
        fine = fine && isfinite(a[y]) && isfinite(z[y]);
      }
      if (!fine) most = INFINITY;
      for (int o = 1; o < lanes; o <<= 1) most = fmaxf(most, __shfl_xor_sync(mates, most, o));
      // a row that holds a value that is not finite reads back as NaN
      const float s = most < INFINITY ? __fdiv_rn(most, 127.f) : __int_as_float(0x7fffffff);
      const int hk = h - nq < nkv ? h - nq : h - nq - nkv;
      const long long at = slot + ((long long)hk << ps_log2);
      uint8_t* dst = (h - nq < nkv ? kp : vp) + at * hd + e;
      const float inv = __fdiv_rn(1.f, s);
      *reinterpret_cast<uint2*>(dst) = codes8(a, s, inv);
      *reinterpret_cast<uint2*>(dst + half) = codes8(z, s, inv);
      if (e == 0) (h - nq < nkv ? ks : vs)[at] = s;
    }
  }
}

cudaError_t paged_append_q8(int in_dtype, int dtype, const void* qkv, long long ld, int batch, int n, int nq, int nkv,
                            int hd, const int32_t* n_rows, const int32_t* table, int table_stride, const int32_t* len,
                            const float2* tab, int max_pos, int n_pages, int ps, long long page0, void* qout,
                            uint8_t* kp, uint8_t* vp, float* ks, float* vs, int* status, cudaStream_t s) {
  const size_t es = in_dtype == DFLASH_BF16 ? 2 : 4;
  const int vec = (reinterpret_cast<uintptr_t>(qkv) & 15) == 0 && (ld * es) % 16 == 0;
  const int rows = batch * n, heads = nq + 2 * nkv, lanes = hd / 16, ps_log2 = 31 - __builtin_clz(ps);
  const bool many = (long long)rows * heads * lanes >= (long long)num_sms() * 2048 * 4;
  const int per_row = (heads + (many ? 3 : 0)) / (many ? 4 : 1) * lanes;
  const int rpb = many ? std::max(1, 1024 / per_row) : 1;
  const unsigned grid = (unsigned)((rows + (long long)rpb - 1) / rpb);
#define DFL_APPEND_H(TI, T, H)                                                                                         \
  DFL_RET(launch_pdl(paged_append_q8_kernel<TI, T, H>, dim3(grid), dim3(256), 0, s, (const TI*)qkv, ld, vec, rows, n,  \
                     nq, nkv, hd, rpb, n_rows, table, table_stride, len, tab, max_pos, n_pages, ps_log2, page0,        \
                     (T*)qout, kp, vp, ks, vs, status))
#define DFL_APPEND(TI, T)   \
  if (many)                 \
    DFL_APPEND_H(TI, T, 4); \
  else                      \
    DFL_APPEND_H(TI, T, 1)
  if (dtype == DFLASH_F32) {
    DFL_APPEND(float, float);
  } else if (in_dtype == DFLASH_F32) {
    DFL_APPEND(float, bf16);
  } else {
    DFL_APPEND(bf16, bf16);
  }
#undef DFL_APPEND
#undef DFL_APPEND_H
  count_launch();
  return cudaSuccess;
}

// ------------------------------------------------------------------ read
// Row (b, j), j < n_rows[b], at position start[b] + j, of head hk goes to
// out[b][hk][j].  A block takes 64 positions of one sequence and head, keys or
// values; a thread moves 16 entries.
constexpr int kReadRows = 64;

template <typename TK, typename TO>
__global__ void __launch_bounds__(256)
    paged_read_kernel(const TK* __restrict__ kp, const TK* __restrict__ vp, const float* __restrict__ ks,
                      const float* __restrict__ vs, int n, int nkv, int hd, int chunks,
                      const int32_t* __restrict__ n_rows, const int32_t* __restrict__ table, int table_stride,
                      const int32_t* __restrict__ start, int max_pos, int n_pages, int ps_log2, long long page0,
                      TO* __restrict__ k_out, TO* __restrict__ v_out, int* status) {
  const bool values = blockIdx.y || !k_out;
  const TK* pool = values ? vp : kp;
  const float* scales = values ? vs : ks;
  TO* out = values ? v_out : k_out;
  const int bh = blockIdx.x / chunks, j0 = (blockIdx.x - bh * chunks) * kReadRows;
  const int b = bh / nkv, hk = bh - b * nkv, parts = hd / 16;
  pdl_launch();
  pdl_wait();
  const int rows = min(n_rows ? min(n_rows[b], n) : n, j0 + kReadRows) - j0;
  for (int t = threadIdx.x; t < rows * parts; t += 256) {
    const int j = j0 + t / parts, e = t % parts * 16;
    const long long pos = (long long)start[b] + j;
    if (pos < 0 || pos >= max_pos || (pos >> ps_log2) >= table_stride) {
      set_status(status, DFLASH_STATUS_CAPACITY);
      continue;
    }
    const int page = table[(long long)b * table_stride + (pos >> ps_log2)];
    if ((unsigned)page >= (unsigned)n_pages) {
      set_status(status, DFLASH_STATUS_BOUNDS);
      continue;
    }
    const long long row = (((page0 + page) * nkv + hk) << ps_log2) + (pos & ((1 << ps_log2) - 1));
    float x[16];
    if constexpr (sizeof(TK) == 1) {
      const uint4 u = *reinterpret_cast<const uint4*>(pool + row * hd + e);
      const float s = scales[row];
      const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int y = 0; y < 16; ++y) x[y] = (float)((int)(w[y >> 2] >> (8 * (y & 3)) & 255u) - 128) * s;
    } else {
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float y[8];
        values8(fetch8<TK>(pool + row * hd + e + 8 * c, true), y);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[8 * c + i] = y[i];
      }
    }
    put<TO>(out + ((long long)bh * n + j) * hd + e, x);
  }
}

cudaError_t paged_read(int dtype, int out_dtype, const void* kp, const void* vp, const float* ks, const float* vs,
                       int batch, int n, int nkv, int hd, const int32_t* n_rows, const int32_t* table,
                       int table_stride, const int32_t* start, int max_pos, int n_pages, int ps, long long page0,
                       void* k_out, void* v_out, int* status, cudaStream_t s) {
  const int chunks = (n + kReadRows - 1) / kReadRows, ps_log2 = 31 - __builtin_clz(ps);
  const long long blocks = (long long)batch * nkv * chunks;
  if (blocks >= (1ll << 31)) return cudaErrorInvalidValue;
  const dim3 grid((unsigned)blocks, k_out && v_out ? 2 : 1);
#define DFL_READ(TK, TO)                                                                                             \
  DFL_RET(launch_pdl(paged_read_kernel<TK, TO>, grid, dim3(256), 0, s, (const TK*)kp, (const TK*)vp, ks, vs, n, nkv, \
                     hd, chunks, n_rows, table, table_stride, start, max_pos, n_pages, ps_log2, page0, (TO*)k_out,   \
                     (TO*)v_out, status))
  if (ks) {
    if (out_dtype == DFLASH_F32)
      DFL_READ(uint8_t, float);
    else
      DFL_READ(uint8_t, bf16);
  } else if (dtype == DFLASH_F32) {
    DFL_READ(float, float);
  } else if (out_dtype == DFLASH_F32) {
    DFL_READ(bf16, float);
  } else {
    DFL_READ(bf16, bf16);
  }
#undef DFL_READ
  count_launch();
  return cudaSuccess;
}

}  // namespace dfl
