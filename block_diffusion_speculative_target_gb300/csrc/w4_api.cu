// C ABI of the weights in 4 bits.
#include <algorithm>
#include <new>

#include "common.cuh"
#include "internal.h"
#include "w4.cuh"

using namespace dfl;

struct dflash_w4_workspace {
  int32_t max_rows;
  int device;
  size_t ticket_bytes;
  W4Scratch sc;
};

#define CK(expr)                                         \
  do {                                                   \
    cudaError_t e_ = (expr);                             \
    if (e_ != cudaSuccess) return record_cuda_error(e_); \
  } while (0)
#define REQ(cond)                               \
  do {                                          \
    if (!(cond)) return DFLASH_ERR_INVALID_ARG; \
  } while (0)

static bool aligned(const void* p, int to) { return (reinterpret_cast<uintptr_t>(p) & (uintptr_t)(to - 1)) == 0; }
static bool apart(const void* a, long long abytes, const void* b, long long bbytes) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x + (uintptr_t)abytes <= y || y + (uintptr_t)bbytes <= x;
}

// The sizes of a matrix in 4 bits, or why it is none.
static int view_of(const dflash_w4* w, W4View* v) {
  REQ(w && w->M > 0 && w->K > 0);
  REQ(w->scale_dtype == DFLASH_F32 || w->scale_dtype == DFLASH_BF16);
  if (w->group != 32 && w->group != 64 && w->group != 128) return DFLASH_ERR_UNSUPPORTED_SHAPE;
  if (w->K % w->group != 0) return DFLASH_ERR_UNSUPPORTED_SHAPE;
  // (row and column block numbers, and their product by 8, stay below 2^31)
  if ((double)w->M * w->K > 17179869184.0 || w->M > (1 << 28) || w->K > (1 << 28)) return DFLASH_ERR_TOO_LARGE;
  v->M = w->M;
  v->K = w->K;
  v->group = w->group;
  v->scale_f32 = w->scale_dtype == DFLASH_F32;
  v->zeros = w->zeros != 0;
  v->kt = (w->K + kW4Tile - 1) / kW4Tile;
  v->block_bytes = kW4Codes + kW4Tile / w->group * kW4Tile * ((v->scale_f32 ? 4 : 2) + v->zeros);
  v->packed = (const uint8_t*)w->packed;
  return DFLASH_OK;
}
static long long packed_bytes(const W4View& v) {
  return (long long)((v.M + kW4Tile - 1) / kW4Tile) * v.kt * v.block_bytes;
}
static int packed_view(const dflash_w4* w, W4View* v) {
  const int rc = view_of(w, v);
  if (rc != DFLASH_OK) return rc;
  REQ(w->packed && aligned(w->packed, 16));
  return DFLASH_OK;
}

extern "C" {

int64_t dflash_w4_bytes(const dflash_w4* w) {
  W4View v;
  const int rc = view_of(w, &v);
  return rc == DFLASH_OK ? packed_bytes(v) : rc;
}

int dflash_w4_pack(const dflash_w4* w, const void* codes, const void* scales, const void* zeros,
                   dflash_stream_t stream) {
  W4View v;
  const int rc = packed_view(w, &v);
  if (rc != DFLASH_OK) return rc;
  REQ(codes && scales && aligned(scales, v.scale_f32 ? 4 : 2) && (zeros != nullptr) == (v.zeros != 0));
  const long long groups = (long long)v.M * (v.K / v.group), pb = packed_bytes(v);
  REQ(apart(w->packed, pb, codes, (long long)v.M * v.K / 2));
  REQ(apart(w->packed, pb, scales, groups * (v.scale_f32 ? 4 : 2)));
  REQ(!zeros || apart(w->packed, pb, zeros, groups));
  CK(w4_pack(v, (const uint8_t*)codes, scales, (const uint8_t*)zeros, (cudaStream_t)stream));
  return DFLASH_OK;
}

int dflash_w4_quantize(const dflash_w4* w, int32_t dtype, const void* src, int64_t ld, dflash_stream_t stream) {
  W4View v;
  const int rc = packed_view(w, &v);
  if (rc != DFLASH_OK) return rc;
  REQ(dtype == DFLASH_F32 || dtype == DFLASH_BF16);
  const int es = dtype == DFLASH_F32 ? 4 : 2;
  REQ(src && ld >= v.K && aligned(src, es));
  REQ(apart(w->packed, packed_bytes(v), src, ((long long)(v.M - 1) * ld + v.K) * es));
  CK(w4_quantize(v, dtype, src, ld, (cudaStream_t)stream));
  return DFLASH_OK;
}

int dflash_w4_unpack(const dflash_w4* w, int32_t dtype, void* dst, dflash_stream_t stream) {
  W4View v;
  const int rc = packed_view(w, &v);
  if (rc != DFLASH_OK) return rc;
  REQ(dtype == DFLASH_F32 || dtype == DFLASH_BF16);
  const int es = dtype == DFLASH_F32 ? 4 : 2;
  REQ(dst && aligned(dst, es) && apart(w->packed, packed_bytes(v), dst, (long long)v.M * v.K * es));
  CK(w4_unpack(v, dtype, dst, (cudaStream_t)stream));
  return DFLASH_OK;
}

int dflash_w4_workspace_alloc(int32_t max_rows, dflash_w4_workspace** out) {
  REQ(out);
  *out = nullptr;
  REQ(max_rows > 0);
  if (max_rows > kMaxRows) return DFLASH_ERR_TOO_LARGE;
  dflash_w4_workspace* ws = new (std::nothrow) dflash_w4_workspace();
  if (!ws) return DFLASH_ERR_OOM;
  ws->max_rows = max_rows;
  const cudaError_t e = cudaGetDevice(&ws->device);
  if (e != cudaSuccess) {
    delete ws;
    return record_cuda_error(e);
  }
  const size_t runs = (size_t)w4_max_runs();
  ws->ticket_bytes = runs * 4 * sizeof(int);
  struct Req {
    void** p;
    size_t bytes;
  } reqs[] = {{(void**)&ws->sc.part, w4_part_floats(max_rows) * sizeof(float)},
              {(void**)&ws->sc.tickets, ws->ticket_bytes},
              {(void**)&ws->sc.status, sizeof(int)}};
  for (auto& r : reqs)
    if (cudaMalloc(r.p, r.bytes) != cudaSuccess) {
      cudaGetLastError();
      dflash_w4_workspace_free(ws);
      return DFLASH_ERR_OOM;
    }
  cudaError_t z = cudaMemset(ws->sc.tickets, 0, ws->ticket_bytes);
  if (z == cudaSuccess) z = cudaMemset(ws->sc.status, 0, sizeof(int));
  if (z == cudaSuccess) z = cudaStreamSynchronize(0);
  if (z != cudaSuccess) {
    dflash_w4_workspace_free(ws);
    return record_cuda_error(z);
  }
  *out = ws;
  return DFLASH_OK;
}

int dflash_w4_workspace_free(dflash_w4_workspace* ws) {
  if (!ws) return DFLASH_OK;
  cudaFree(ws->sc.part);
  cudaFree(ws->sc.tickets);
  cudaFree(ws->sc.status);
  delete ws;
  return DFLASH_OK;
}

int dflash_w4_status(dflash_w4_workspace* ws, dflash_stream_t stream, int32_t* status_out) {
  REQ(ws && status_out);
  int32_t v = 0;
  const cudaStream_t s = (cudaStream_t)stream;
  CK(cudaMemcpyAsync(&v, ws->sc.status, 4, cudaMemcpyDeviceToHost, s));
  CK(cudaMemsetAsync(ws->sc.status, 0, 4, s));
  CK(cudaStreamSynchronize(s));
  // a call that timed out may have left pieces counted
  if (v & DFLASH_STATUS_TIMEOUT) CK(cudaMemsetAsync(ws->sc.tickets, 0, ws->ticket_bytes, s));
  *status_out = v;
  return DFLASH_OK;
}

int dflash_linear_w4(int32_t dtype, const void* x, int64_t ldx, const dflash_w4* w, const float* add, int32_t swiglu,
                     void* y, int32_t rows, dflash_w4_workspace* ws, dflash_stream_t stream) {
  REQ(ws);
  W4View v;
  const int rc = packed_view(w, &v);
  if (rc != DFLASH_OK) return rc;
  REQ(dtype == DFLASH_F32 || dtype == DFLASH_BF16);
  REQ(x && y && rows > 0 && rows <= ws->max_rows && ldx >= v.K);
  if (swiglu && v.M % 2 != 0) return DFLASH_ERR_UNSUPPORTED_SHAPE;
  const int es = dtype == DFLASH_F32 ? 4 : 2, os = swiglu ? es : 4;
  REQ(aligned(x, es) && aligned(y, os) && aligned(add, 4));
  const long long ybytes = (long long)rows * (swiglu ? v.M / 2 : v.M) * os;
  REQ(apart(y, ybytes, x, ((long long)(rows - 1) * ldx + v.K) * es) && apart(y, ybytes, w->packed, packed_bytes(v)));
  REQ(!add || (!swiglu && add == y) || apart(y, ybytes, add, (long long)rows * v.M * 4));
  int device = -1;
  REQ(cudaGetDevice(&device) == cudaSuccess && device == ws->device);
  const W4Epi epi = {add, swiglu != 0, y};
  // 16 rows of 6144 x 4096: 11 us fed from registers, 15 through TMEM; 15 rows of 151936 x 5120: 100 and 198.  32 rows of
  // 4096 x 12288: 30 (in a form of four column tiles, since dropped) and 21.  On large matrices the 17th row costs a step:
  // 24576 x 4096 with the gate 23 -> 36 us, 151936 x 5120 100 -> 199 (217 with 64 rows).
  if (dtype == DFLASH_BF16 && rows <= kW4MmaRows)
    CK(w4_linear_mma(v, x, ldx, rows, epi, ws->sc, (cudaStream_t)stream));
  else if (dtype == DFLASH_BF16)
    CK(w4_linear_tc(v, x, ldx, rows, epi, ws->sc, (cudaStream_t)stream));
  else
    CK(w4_linear_core(v, x, ldx, rows, epi, (cudaStream_t)stream));
  return DFLASH_OK;
}

}  // extern "C"
