// paged_api.cu -- C entry points of the paged serving operators (include/
// pisa.h): argument checks on the host, then the launchers of append.cu,
// paged_decode.cu and paged_prefill.cu.
#include <math.h>

#include <algorithm>

#include "paged.cuh"

using namespace pisa;

namespace pisa {

namespace {

__global__ void __launch_bounds__(256) clear_kernel(int32_t* p, int64_t n) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int64_t i = blockIdx.x * (int64_t)blockDim.x + threadIdx.x;
  if (i < n) p[i] = 0;
}

}  // namespace

cudaError_t launch_clear(void* ws, size_t bytes, cudaStream_t st) {
  const int64_t n = (int64_t)(bytes / 4);
  note_launch();
  clear_kernel<<<(unsigned)ceil_div64(n, 256), 256, 0, st>>>((int32_t*)ws, n);
  return cudaGetLastError();
}

}  // namespace pisa

namespace {

bool aligned4(const void* x) { return ((uintptr_t)x & 3u) == 0; }

// Checks that every call shares.  *empty: nothing to do.
pisa_status common_checks(const pisa_params* p, int64_t n, Prob* pr, Pyr* s, bool* empty) {
  const pisa_status rc = check_params(p, pr, s);
  if (rc != PISA_OK) return rc;
  if (n < 0 || n > pr->N) return PISA_ERR_INVALID_ARG;
  *empty = pr->B == 0 || n == 0;
  // grids and counters index sequences x heads in 32 bits
  if (pr->B * pr->Hq >= ((int64_t)1 << 31)) return PISA_ERR_UNSUPPORTED;
  return PISA_OK;
}

pisa_status pool_checks(const Prob& pr, const Pyr& s, const void* k_pages, const void* v_pages, int64_t num_pages,
                        const int32_t* page_table, const int32_t* seq_lens, const void* ws, Pools* pools) {
  if (!k_pages || !v_pages || !page_table || !seq_lens || !ws || num_pages < 1) return PISA_ERR_INVALID_ARG;
  if (!aligned16(k_pages) || !aligned16(v_pages) || !aligned16(ws) || !aligned4(page_table) || !aligned4(seq_lens))
    return PISA_ERR_MISALIGNED;
  // rows of the pools are TMA coordinates
  if (num_pages > (((int64_t)1 << 31) - 1) / ((int64_t)pr.Hkv * pr.C)) return PISA_ERR_UNSUPPORTED;
  pools->k = k_pages;
  pools->v = v_pages;
  pools->table = page_table;
  pools->num_pages = num_pages;
  pools->nb = s.nb;
  return PISA_OK;
}

pisa_status mask_checks(const Prob& pr, const pisa_mask* mask, MaskArgs* m) {
  *m = MaskArgs{};
  if (!mask) return PISA_OK;
  if (mask->struct_size < sizeof(pisa_mask)) return PISA_ERR_INVALID_ARG;
  if (!(mask->softcap >= 0.0f) || isinf(mask->softcap) || mask->window < 0) return PISA_ERR_INVALID_ARG;
  if (!aligned4(mask->slopes) || !aligned4(mask->first_key) || !aligned4(mask->prefix_lens))
    return PISA_ERR_MISALIGNED;
  if (mask->softcap > 0.0f) {
    m->cap2 = mask->softcap * kLog2e;
    m->pre = pr.scale2 / m->cap2;
    if (!(m->cap2 > 0.0f) || isinf(m->cap2) || isinf(m->pre)) return PISA_ERR_INVALID_ARG;
    // tanh(u) / u = 1 + c1 u^2 + c2 u^4 + c3 u^6 on [-1/2, 1/2]: a linear program for the least largest relative
    // error, 6.4e-7
    const double c[4] = {1.0, -0.3332815933841437, 0.13205359737189304, -0.04475064468281561};
    const double last = fabs(c[3]) * pr.scale2 * pow(m->pre, 6);
    const bool normal = last >= 1.2e-38 && last <= 3.4e38;
    double f = pr.scale2;
    for (int i = 0; i < 4; ++i, f *= normal ? (double)m->pre * m->pre : 1.0) m->tk[i] = (float)(f * c[i]);
    m->by = normal ? 1.0f : m->pre;
    m->lim = normal ? 0.5f / m->pre : 0.5f;
  }
  m->window = mask->window;
  m->slopes = mask->slopes;
  m->first_key = mask->first_key;
  m->prefix_lens = mask->prefix_lens;
  return PISA_OK;
}

// Strides (sequence, head, token) of a [B, H, n, d] view in elements: each a
// multiple of 16 bytes, so that every row takes 16-byte accesses.  A dimension
// of one entry has no stride.
pisa_status stride_checks(const int64_t* given, int64_t B, int64_t H, int64_t n, int64_t d, int64_t per16,
                          int64_t* out) {
  const int64_t size[3] = {B, H, n};
  out[0] = H * n * d;
  out[1] = n * d;
  out[2] = d;
  if (!given) return PISA_OK;
  for (int i = 0; i < 3; ++i) {
    if (size[i] == 1) continue;
    if (given[i] < 0) return PISA_ERR_INVALID_ARG;
    if (given[i] % per16 != 0) return PISA_ERR_MISALIGNED;
    out[i] = given[i];
  }
  return PISA_OK;
}

}  // namespace

extern "C" {

size_t pisa_paged_workspace_bytes(const pisa_params* p, int64_t n) {
  Prob pr; Pyr s;
  if (check_params(p, &pr, &s) != PISA_OK || n < 0 || n > pr.N) return 0;
  return std::max(paged_decode_ws_bytes(pr), paged_prefill_ws_bytes(pr, n));
}

pisa_status pisa_append_paged(const pisa_params* p, int64_t n, const void* q, const int64_t* q_strides,
                              const void* k, const int64_t* k_strides, const void* v, const int64_t* v_strides,
                              const int32_t* seq_lens, const int32_t* new_lens, const float* rope, int32_t rot_dim,
                              int32_t interleaved, void* k_pages, void* v_pages, int64_t num_pages,
                              const int32_t* page_table, void* ws, size_t ws_bytes, void* q_out, void* k_out,
                              void* stream) {
  Prob pr; Pyr s; bool empty = false; Pools pools;
  pisa_status rc = common_checks(p, n, &pr, &s, &empty);
  if (rc != PISA_OK || empty) return rc;
  if (rot_dim < 0 || rot_dim > pr.d || (rope != nullptr) != (rot_dim > 0)) return PISA_ERR_INVALID_ARG;
  if (rot_dim % 16 != 0) return PISA_ERR_UNSUPPORTED;
  if (!k || !v || (q != nullptr) != (q_out != nullptr)) return PISA_ERR_INVALID_ARG;
  rc = pool_checks(pr, s, k_pages, v_pages, num_pages, page_table, seq_lens, ws, &pools);
  if (rc != PISA_OK) return rc;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(q_out) || !aligned16(k_out) ||
      !aligned16(rope) || !aligned4(new_lens))
    return PISA_ERR_MISALIGNED;
  const int64_t per16 = pr.dtype == PISA_BF16 ? 8 : 4;
  int64_t qs[3], ks[3], vs[3];
  rc = stride_checks(q_strides, pr.B, pr.Hq, n, pr.d, per16, qs);
  if (rc == PISA_OK) rc = stride_checks(k_strides, pr.B, pr.Hkv, n, pr.d, per16, ks);
  if (rc == PISA_OK) rc = stride_checks(v_strides, pr.B, pr.Hkv, n, pr.d, per16, vs);
  if (rc != PISA_OK) return rc;
  if (ws_bytes < pisa_paged_workspace_bytes(p, n)) return PISA_ERR_WORKSPACE;
  cudaStream_t st = (cudaStream_t)stream;
  return cuda_status(launch_append_paged(pr, n, q, qs, k, ks, v, vs, seq_lens, new_lens, rope, rot_dim, interleaved,
                                         k_pages, v_pages, page_table, s.nb, num_pages, (int32_t*)ws, q_out, k_out,
                                         st));
}

pisa_status pisa_dense_decode_paged(const pisa_params* p, const pisa_mask* mask, const void* q, const void* k_pages,
                                    const void* v_pages, int64_t num_pages, const int32_t* page_table,
                                    const int32_t* seq_lens, void* ws, size_t ws_bytes, void* out, void* stream) {
  Prob pr; Pyr s; bool empty = false; Pools pools; MaskArgs m;
  pisa_status rc = common_checks(p, 1, &pr, &s, &empty);
  if (rc != PISA_OK || empty) return rc;
  if (pr.dtype != PISA_BF16) return PISA_ERR_UNSUPPORTED;  // built for bf16 inputs
  rc = mask_checks(pr, mask, &m);
  if (rc != PISA_OK) return rc;
  m.prefix_lens = nullptr;  // the last token sees every key already
  if (!q || !out) return PISA_ERR_INVALID_ARG;
  rc = pool_checks(pr, s, k_pages, v_pages, num_pages, page_table, seq_lens, ws, &pools);
  if (rc != PISA_OK) return rc;
  if (!aligned16(q) || !aligned16(out)) return PISA_ERR_MISALIGNED;
  if (ws_bytes < paged_decode_ws_bytes(pr)) return PISA_ERR_WORKSPACE;
  return cuda_status(launch_paged_decode(pr, m, q, pools, seq_lens, nullptr, (char*)ws, out, (cudaStream_t)stream));
}

pisa_status pisa_attend_decode_paged(const pisa_params* p, const void* q, const void* k_pages, const void* v_pages,
                                     int64_t num_pages, const int32_t* page_table, const int32_t* seq_lens,
                                     const int32_t* idx, void* ws, size_t ws_bytes, void* out, void* stream) {
  Prob pr; Pyr s; bool empty = false; Pools pools;
  pisa_status rc = common_checks(p, 1, &pr, &s, &empty);
  if (rc != PISA_OK || empty) return rc;
  if (pr.dtype != PISA_BF16) return PISA_ERR_UNSUPPORTED;  // built for bf16 inputs
  if (!q || !out || !idx) return PISA_ERR_INVALID_ARG;
  rc = pool_checks(pr, s, k_pages, v_pages, num_pages, page_table, seq_lens, ws, &pools);
  if (rc != PISA_OK) return rc;
  if (!aligned16(q) || !aligned16(out) || !aligned4(idx)) return PISA_ERR_MISALIGNED;
  if (ws_bytes < paged_decode_ws_bytes(pr)) return PISA_ERR_WORKSPACE;
  return cuda_status(
      launch_paged_decode(pr, MaskArgs{}, q, pools, seq_lens, idx, (char*)ws, out, (cudaStream_t)stream));
}

pisa_status pisa_dense_prefill_paged(const pisa_params* p, const pisa_mask* mask, int64_t n, const void* q,
                                     const void* k_pages, const void* v_pages, int64_t num_pages,
                                     const int32_t* page_table, const int32_t* seq_lens, const int32_t* new_lens,
                                     void* ws, size_t ws_bytes, void* out, void* stream) {
  Prob pr; Pyr s; bool empty = false; Pools pools; MaskArgs m;
  pisa_status rc = common_checks(p, n, &pr, &s, &empty);
  if (rc != PISA_OK || empty) return rc;
  if (pr.dtype != PISA_BF16) return PISA_ERR_UNSUPPORTED;  // built for bf16 inputs
  rc = mask_checks(pr, mask, &m);
  if (rc != PISA_OK) return rc;
  if (!q || !out) return PISA_ERR_INVALID_ARG;
  rc = pool_checks(pr, s, k_pages, v_pages, num_pages, page_table, seq_lens, ws, &pools);
  if (rc != PISA_OK) return rc;
  if (!aligned16(q) || !aligned16(out) || !aligned4(new_lens)) return PISA_ERR_MISALIGNED;
  // groups of rows (16 tokens and more of a key head) are numbered in 32 bits
  if (pr.B * pr.Hkv * ceil_div64(n, 32) >= ((int64_t)1 << 31)) return PISA_ERR_UNSUPPORTED;
  if (ws_bytes < paged_prefill_ws_bytes(pr, n)) return PISA_ERR_WORKSPACE;
  return cuda_status(launch_paged_prefill(pr, m, n, q, pools, seq_lens, new_lens, (char*)ws, out,
                                          (cudaStream_t)stream));
}

}  // extern "C"
