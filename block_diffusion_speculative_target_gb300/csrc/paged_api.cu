// C ABI of the KV pages: the handle, the workspace and the calls on them.
#include <math.h>

#include <algorithm>
#include <new>

#include "common.cuh"
#include "internal.h"
#include "paged.cuh"

using namespace dfl;

struct dflash_pages {
  int32_t n_layers, n_pages, page_size, max_pos, nq, nkv, hd, dtype;
  int device;
  void *k, *v;     // the caller's pool
  float *ks, *vs;  // 8-bit pages: the scales of its rows; else null
  float2* rope;    // [max_pos][hd / 2]
  CUtensorMap tk, tv;  // bf16: over the whole pool
};

struct dflash_paged_workspace {
  int32_t max_batch, max_rows, nq, nkv, hd;
  int device;
  long long part_rows;
  float* part_o;     // [part_rows][hd]
  float2* part_ml;   // [part_rows]
  int32_t* plan;     // [kPlanCum + max_batch]
  int32_t* tickets;  // [items]
  int32_t* records;  // [CTAs][8]
  size_t ticket_bytes;
  int* status;
};

#define CK(expr)                                           \
  do {                                                     \
    cudaError_t e_ = (expr);                               \
    if (e_ != cudaSuccess) return record_cuda_error(e_);   \
  } while (0)
#define REQ(cond)                               \
  do {                                          \
    if (!(cond)) return DFLASH_ERR_INVALID_ARG; \
  } while (0)

static long long pool_rows(const dflash_pages* p) {
  return (long long)p->n_layers * p->n_pages * p->nkv * p->page_size;
}
static bool on_device(int device) {
  int d = -1;
  return cudaGetDevice(&d) == cudaSuccess && d == device;
}
static bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
static bool apart(const void* a, long long abytes, const void* b, long long bbytes) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x + (uintptr_t)abytes <= y || y + (uintptr_t)bbytes <= x;
}
static int elem_size(int dtype) { return dtype == DFLASH_F32 ? 4 : 2; }
static long long pool_bytes(const dflash_pages* p) {
  return pool_rows(p) * p->hd * (p->ks ? 1 : elem_size(p->dtype));
}
static bool apart_from_pool(const dflash_pages* p, const void* a, long long bytes) {
  if (p->ks && !(apart(a, bytes, p->ks, pool_rows(p) * 4) && apart(a, bytes, p->vs, pool_rows(p) * 4))) return false;
  return apart(a, bytes, p->k, pool_bytes(p)) && apart(a, bytes, p->v, pool_bytes(p));
}
// The pool's own parts.
static bool pool_apart(const dflash_pages* p) {
  if (!apart(p->k, pool_bytes(p), p->v, pool_bytes(p))) return false;
  if (!p->ks) return true;
  const long long b = pool_bytes(p), s = pool_rows(p) * 4;
  return apart(p->ks, s, p->vs, s) && apart(p->k, b, p->ks, s) && apart(p->k, b, p->vs, s) && apart(p->v, b, p->ks, s) &&
         apart(p->v, b, p->vs, s);
}

static int create(const dflash_model_desc* d, int32_t n_layers, int32_t n_pages, int32_t page_size, int32_t max_pos,
                  void* k, void* v, float* ks, float* vs, dflash_pages** out) {
  REQ(out);
  *out = nullptr;
  REQ(desc_ok(d) && d->rope_theta > 0.f && isfinite(d->rope_theta));
  REQ(n_layers > 0 && n_pages > 0 && max_pos > 0 && k && v && aligned16(k) && aligned16(v));
  REQ(page_size == 16 || page_size == 32 || page_size == 64 || page_size == 128);
  if (d->n_q_heads / d->n_kv_heads > kPagedMaxG) return DFLASH_ERR_UNSUPPORTED_SHAPE;
  // pool rows are addressed by int32 coordinates
  if ((double)n_layers * n_pages * d->n_kv_heads * page_size > 2147483000.0) return DFLASH_ERR_TOO_LARGE;
  dflash_pages* p = new (std::nothrow) dflash_pages();
  if (!p) return DFLASH_ERR_OOM;
  *p = dflash_pages{n_layers, n_pages, page_size, max_pos, d->n_q_heads, d->n_kv_heads, d->head_dim, d->dtype,
                    0,        k,       v,         ks,      vs,           nullptr,       {},          {}};
  if (ks && !pool_apart(p)) {
    delete p;
    return DFLASH_ERR_INVALID_ARG;
  }
  if (p->dtype == DFLASH_BF16 && !ks && !make_page_maps(k, v, pool_rows(p), p->hd, page_size, &p->tk, &p->tv)) {
    delete p;
    return record_cuda_error(cudaErrorInvalidValue);
  }
  cudaError_t e = cudaGetDevice(&p->device);
  if (e == cudaSuccess) {
    const int half = d->head_dim / 2;
    if (cudaMalloc(&p->rope, sizeof(float2) * (size_t)max_pos * half) != cudaSuccess) {
      cudaGetLastError();
      delete p;
      return DFLASH_ERR_OOM;
    }
    e = rope_table(p->rope, max_pos, half, (double)d->rope_theta);
    // the table is there for whatever stream the first call comes on
    if (e == cudaSuccess) e = cudaStreamSynchronize(0);
  }
  if (e != cudaSuccess) {
    dflash_pages_free(p);
    return record_cuda_error(e);
  }
  *out = p;
  return DFLASH_OK;
}

extern "C" {

int dflash_pages_create(const dflash_model_desc* d, int32_t n_layers, int32_t n_pages, int32_t page_size,
                        int32_t max_pos, void* k, void* v, dflash_pages** out) {
  return create(d, n_layers, n_pages, page_size, max_pos, k, v, nullptr, nullptr, out);
}

int dflash_pages_create_q8(const dflash_model_desc* d, int32_t n_layers, int32_t n_pages, int32_t page_size,
                           int32_t max_pos, void* k, void* v, float* k_scales, float* v_scales, dflash_pages** out) {
  REQ(out);
  *out = nullptr;
  REQ(k_scales && v_scales && aligned16(k_scales) && aligned16(v_scales));
  return create(d, n_layers, n_pages, page_size, max_pos, k, v, k_scales, v_scales, out);
}

int dflash_pages_free(dflash_pages* p) {
  if (!p) return DFLASH_OK;
  cudaFree(p->rope);
  delete p;
  return DFLASH_OK;
}

int dflash_paged_workspace_alloc(const dflash_model_desc* d, int32_t max_batch, int32_t max_rows,
                                 dflash_paged_workspace** out) {
  REQ(out);
  *out = nullptr;
  REQ(desc_ok(d) && max_batch > 0 && max_rows >= max_batch);
  if (d->n_q_heads / d->n_kv_heads > kPagedMaxG) return DFLASH_ERR_UNSUPPORTED_SHAPE;
  if (max_rows > (1 << 20)) return DFLASH_ERR_TOO_LARGE;
  dflash_paged_workspace* w = new (std::nothrow) dflash_paged_workspace();
  if (!w) return DFLASH_ERR_OOM;
  w->max_batch = max_batch;
  w->max_rows = max_rows;
  w->nq = d->n_q_heads;
  w->nkv = d->n_kv_heads;
  w->hd = d->head_dim;
  cudaError_t e = cudaGetDevice(&w->device);
  if (e != cudaSuccess) {
    delete w;
    return record_cuda_error(e);
  }
  // whole row groups (at most twice the rows) and a slot per CTA, for a sequence's own pieces and the shared ones
  w->part_rows = 2 * (2ll * max_rows * d->n_q_heads + (long long)num_sms() * kPagedItemRows);
  // items of 16 stacked rows at least, or of one sequence
  w->ticket_bytes = (size_t)((long long)max_rows * d->n_q_heads / 16 + (long long)max_batch * d->n_kv_heads) * 4;
  struct Req {
    void** p;
    size_t bytes;
  } reqs[] = {{(void**)&w->part_o, (size_t)w->part_rows * d->head_dim * 4},
              {(void**)&w->part_ml, (size_t)w->part_rows * 8},
              {(void**)&w->plan, (size_t)(kPlanCum + max_batch) * 4},
              {(void**)&w->tickets, w->ticket_bytes},
              {(void**)&w->records, (size_t)num_sms() * kPagedMaxCtas * 32},
              {(void**)&w->status, 4}};
  for (auto& r : reqs)
    if (cudaMalloc(r.p, r.bytes) != cudaSuccess) {
      cudaGetLastError();
      dflash_paged_workspace_free(w);
      return DFLASH_ERR_OOM;
    }
  e = cudaMemset(w->status, 0, 4);
  if (e == cudaSuccess) e = cudaMemset(w->tickets, 0, w->ticket_bytes);
  if (e == cudaSuccess) e = cudaStreamSynchronize(0);
  if (e != cudaSuccess) {
    dflash_paged_workspace_free(w);
    return record_cuda_error(e);
  }
  *out = w;
  return DFLASH_OK;
}

int dflash_paged_workspace_free(dflash_paged_workspace* w) {
  if (!w) return DFLASH_OK;
  cudaFree(w->part_o);
  cudaFree(w->part_ml);
  cudaFree(w->plan);
  cudaFree(w->tickets);
  cudaFree(w->records);
  cudaFree(w->status);
  delete w;
  return DFLASH_OK;
}

int dflash_paged_status(dflash_paged_workspace* w, dflash_stream_t stream, int32_t* status_out) {
  REQ(w && status_out);
  int32_t v = 0;
  const cudaStream_t s = (cudaStream_t)stream;
  CK(cudaMemcpyAsync(&v, w->status, 4, cudaMemcpyDeviceToHost, s));
  CK(cudaMemsetAsync(w->status, 0, 4, s));  // (in the stream's order: the next call's bits stay)
  CK(cudaStreamSynchronize(s));
  // a call that timed out may have left pieces counted: until here later results may be wrong too
  if (v & DFLASH_STATUS_TIMEOUT) CK(cudaMemsetAsync(w->tickets, 0, w->ticket_bytes, s));
  *status_out = v;
  return DFLASH_OK;
}

int dflash_paged_append(dflash_pages* p, int32_t layer, int32_t in_dtype, const void* qkv, int64_t ld, int32_t batch,
                        int32_t n, const int32_t* n_rows, const int32_t* table, int32_t table_stride,
                        const int32_t* len, void* q_out, dflash_paged_workspace* ws, dflash_stream_t stream) {
  REQ(p && ws && qkv && table && len && layer >= 0 && layer < p->n_layers);
  REQ(batch > 0 && n > 0 && table_stride > 0 && (long long)batch * n < (1ll << 31));
  REQ(in_dtype == DFLASH_F32 || in_dtype == p->dtype);
  const int nq = q_out ? p->nq : 0;
  REQ(ld >= (long long)(nq + 2 * p->nkv) * p->hd && aligned16(q_out));
  REQ((reinterpret_cast<uintptr_t>(qkv) & (in_dtype == DFLASH_F32 ? 3 : 1)) == 0);
  const long long rows = (long long)batch * n, width = (long long)(nq + 2 * p->nkv) * p->hd;
  const long long qkv_bytes = ((rows - 1) * ld + width) * elem_size(in_dtype);
  const long long q_bytes = rows * p->nq * p->hd * elem_size(p->dtype);
  REQ(!q_out || (apart(qkv, qkv_bytes, q_out, q_bytes) && apart_from_pool(p, q_out, q_bytes)));
  REQ(apart_from_pool(p, qkv, qkv_bytes) && pool_apart(p));
  REQ(on_device(p->device) && ws->device == p->device);
  if (p->ks) {
    CK(paged_append_q8(in_dtype, p->dtype, qkv, ld, batch, n, nq, p->nkv, p->hd, n_rows, table, table_stride, len,
                       p->rope, p->max_pos, p->n_pages, p->page_size, (long long)layer * p->n_pages, q_out,
                       (uint8_t*)p->k, (uint8_t*)p->v, p->ks, p->vs, ws->status, (cudaStream_t)stream));
    return DFLASH_OK;
  }
  CK(paged_append(in_dtype, p->dtype, qkv, ld, batch, n, nq, p->nkv, p->hd, n_rows, table, table_stride, len, p->rope,
                  p->max_pos, p->n_pages, p->page_size, (long long)layer * p->n_pages, q_out, p->k, p->v, ws->status,
                  (cudaStream_t)stream));
  return DFLASH_OK;
}

int dflash_paged_read(dflash_pages* p, int32_t layer, int32_t out_dtype, int32_t batch, int32_t n,
                      const int32_t* n_rows, const int32_t* table, int32_t table_stride, const int32_t* start,
                      void* k_out, void* v_out, dflash_paged_workspace* ws, dflash_stream_t stream) {
  REQ(p && ws && table && start && (k_out || v_out) && layer >= 0 && layer < p->n_layers);
  REQ(batch > 0 && n > 0 && table_stride > 0 && (long long)batch * n < (1ll << 31));
  REQ(out_dtype == DFLASH_F32 || out_dtype == p->dtype);
  REQ(aligned16(k_out) && aligned16(v_out));
  const long long bytes = (long long)batch * n * p->nkv * p->hd * elem_size(out_dtype);
  REQ(!k_out || apart_from_pool(p, k_out, bytes));
  REQ(!v_out || apart_from_pool(p, v_out, bytes));
  REQ(!k_out || !v_out || apart(k_out, bytes, v_out, bytes));
  REQ(on_device(p->device) && ws->device == p->device);
  CK(paged_read(p->dtype, out_dtype, p->k, p->v, p->ks, p->vs, batch, n, p->nkv, p->hd, n_rows, table, table_stride,
                start, p->max_pos, p->n_pages, p->page_size, (long long)layer * p->n_pages, k_out, v_out, ws->status,
                (cudaStream_t)stream));
  return DFLASH_OK;
}

static int attend(dflash_pages* p, int32_t layer, const void* q, int32_t batch, int32_t n, const int32_t* n_rows,
                  int32_t causal, int32_t window, int32_t sinks, const int32_t* table, int32_t table_stride,
                  const int32_t* len, const int32_t* shared_len, void* out, dflash_paged_workspace* ws,
                  dflash_stream_t stream) {
  REQ(p && ws && q && out && table && len && layer >= 0 && layer < p->n_layers);
  REQ(batch > 0 && n > 0 && table_stride > 0 && window >= 0 && sinks >= 0);
  REQ(batch <= ws->max_batch && (long long)batch * n <= ws->max_rows);
  REQ(ws->nq == p->nq && ws->nkv == p->nkv && ws->hd == p->hd);
  REQ(aligned16(q) && aligned16(out));
  const long long q_bytes = (long long)batch * n * p->nq * p->hd * elem_size(p->dtype);
  REQ(apart(q, q_bytes, out, q_bytes) && apart_from_pool(p, out, q_bytes));
  REQ(on_device(p->device) && ws->device == p->device);
  if ((long long)table_stride * p->page_size > (1ll << 30)) return DFLASH_ERR_TOO_LARGE;
  PagedGeom g = {};
  g.batch = batch;
  g.n = n;
  g.nq = p->nq;
  g.nkv = p->nkv;
  g.G = p->nq / p->nkv;
  g.causal = causal ? 1 : 0;
  g.window = window;
  g.sinks = sinks;
  g.ps = p->page_size;
  g.ps_log2 = p->page_size == 16 ? 4 : p->page_size == 32 ? 5 : p->page_size == 64 ? 6 : 7;
  g.n_pages = p->n_pages;
  g.table_stride = table_stride;
  g.cap = std::min(table_stride * p->page_size, p->max_pos);
  g.page_row0 = (long long)layer * p->n_pages * p->nkv * p->page_size;
  g.len = len;
  g.n_rows = n_rows;
  g.table = table;
  g.shared = shared_len;
  g.ks = p->ks;
  g.vs = p->vs;
  g.part_o = ws->part_o;
  g.part_ml = ws->part_ml;
  g.plan = ws->plan;
  g.tickets = ws->tickets;
  g.records = ws->records;
  g.status = ws->status;
  g.wait_ns = (unsigned)std::min(wait_limit_ns(), 4000000000ull);
  const bool tc = p->dtype == DFLASH_BF16 && !p->ks, q8 = p->dtype == DFLASH_BF16 && p->ks;
  if (!paged_line_fits(g, tc ? paged_rule_tc(g) : q8 ? paged_rule_q8(g) : paged_rule_core(g)))
    return DFLASH_ERR_TOO_LARGE;
  if (q8)
    CK(paged_attention_q8(p->hd, g, q, p->k, p->v, out, ws->part_rows, (cudaStream_t)stream));
  else if (tc)
    CK(paged_attention_tc(p->hd, g, p->tk, p->tv, pool_rows(p), q, out, ws->part_rows, (cudaStream_t)stream));
  else
    CK(paged_attention_core(p->hd, g, q, p->k, p->v, out, ws->part_rows, (cudaStream_t)stream));
  return DFLASH_OK;
}

int dflash_paged_attention(dflash_pages* p, int32_t layer, const void* q, int32_t batch, int32_t n,
                           const int32_t* n_rows, int32_t causal, int32_t window, int32_t sinks, const int32_t* table,
                           int32_t table_stride, const int32_t* len, void* out, dflash_paged_workspace* ws,
                           dflash_stream_t stream) {
  return attend(p, layer, q, batch, n, n_rows, causal, window, sinks, table, table_stride, len, nullptr, out, ws,
                stream);
}

int dflash_paged_attention_shared(dflash_pages* p, int32_t layer, const void* q, int32_t batch, int32_t n,
                                  const int32_t* n_rows, int32_t causal, int32_t window, int32_t sinks,
                                  const int32_t* table, int32_t table_stride, const int32_t* len,
                                  const int32_t* shared_len, void* out, dflash_paged_workspace* ws,
                                  dflash_stream_t stream) {
  REQ(shared_len);
  return attend(p, layer, q, batch, n, n_rows, causal, window, sinks, table, table_stride, len, shared_len, out, ws,
                stream);
}

}  // extern "C"
