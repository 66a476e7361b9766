// paged.cuh -- what the paged serving operators share: the mask of a dense
// attention call, the checks of device-side lengths and pages, and the
// workspace of a call.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "pisa_common.cuh"
#include "pisa_internal.h"
#include "tc_ptx.cuh"

namespace pisa {

// Key and value pools [num_pages, Hkv, 64, d] behind one page table [B, nb].
struct Pools {
  const void* k;
  const void* v;
  const int32_t* table;
  int64_t num_pages, nb;
};

// A dense call's mask (pisa_mask), scores in log2 units.
struct MaskArgs {
  float cap2;                  // softcap * log2(e), 0: none
  float pre;                   // with a cap: scale / softcap, the argument of tanh per unit of q . k
  // cap2 tanh(pre x) = x (tk[0] + w (tk[1] + w (tk[2] + w tk[3]))) with y = by x and w = y^2 for |y| <= lim, which
  // stands for |pre x| <= 1/2, off by less than 2^-20 of itself: tk[0] is the scale, and the rest makes the largest
  // relative error least.  by is 1, or pre where a cap is so large that the coefficients would leave fp32's normal range.
  float tk[4], by, lim;
  int64_t window;              // 0: none
  const float* slopes;         // null: none
  const int32_t* first_key;    // null: none; [B, n]
  const int32_t* prefix_lens;  // null: none
};

// Lengths of sequence b: total positions and new tokens among them; false
// (and new = its rows to zero) when they do not fit.
__device__ __forceinline__ bool new_span(const int32_t* seq_lens, const int32_t* new_lens, int64_t b, int64_t n,
                                         int64_t N, int64_t* len, int64_t* cnt) {
  *len = seq_lens[b];
  *cnt = new_lens ? (int64_t)new_lens[b] : n;
  const bool ok = *cnt >= 0 && *cnt <= n && *cnt <= *len && *len <= N;
  if (!ok) *cnt = *cnt < 0 ? 0 : (*cnt > n ? n : *cnt);
  return ok;
}

// First and last key that the token at position t sees (last < first: none).
__device__ __forceinline__ void key_span(const MaskArgs& m, int64_t b, int64_t n, int64_t i, int64_t t, int64_t len,
                                         int64_t* lo, int64_t* hi) {
  int64_t l = 0, h = t;
  if (m.window > 0 && t - m.window + 1 > l) l = t - m.window + 1;
  if (m.first_key) {
    const int64_t f = m.first_key[b * n + i];
    if (f > l) l = f;
  }
  if (m.prefix_lens) {
    const int64_t p = (int64_t)m.prefix_lens[b] - 1;
    if (p > h) h = p < len - 1 ? p : len - 1;
  }
  *lo = l;
  *hi = h;
}

// cap2 tanh(pre x), off by less than 2^-19 of itself whatever the cap: the
// polynomial where the score is small against the cap (a large cap is no cap),
// tanh u = 1 - 2 / (1 + e^2u), whose error is a few 2^-24 of the cap, elsewhere.
__device__ __forceinline__ float cap_score(const MaskArgs& m, float x) {
  const float y = x * m.by, w = y * y;
  const float small = x * fmaf(w, fmaf(w, fmaf(w, m.tk[3], m.tk[2]), m.tk[1]), m.tk[0]);
  const float large = fmaf(-2.0f * m.cap2, __frcp_rn(1.0f + ptx::ex2(x * m.pre * (2.0f * kLog2e))), m.cap2);
  return fabsf(y) <= m.lim ? small : large;
}

cudaError_t launch_append_paged(const Prob& pr, int64_t n, const void* q, const int64_t* qs, const void* k,
                                const int64_t* ks, const void* v, const int64_t* vs, const int32_t* seq_lens,
                                const int32_t* new_lens, const float* rope, int rot_dim, int interleaved,
                                void* k_pages, void* v_pages, const int32_t* table, int64_t nb, int64_t num_pages,
                                int32_t* status, void* q_out, void* k_out, cudaStream_t st);
cudaError_t launch_paged_decode(const Prob& pr, const MaskArgs& m, const void* q, const Pools& pools,
                                const int32_t* seq_lens, const int32_t* idx, char* ws, void* out, cudaStream_t st);
cudaError_t launch_paged_prefill(const Prob& pr, const MaskArgs& m, int64_t n, const void* q, const Pools& pools,
                                 const int32_t* seq_lens, const int32_t* new_lens, char* ws, void* out,
                                 cudaStream_t st);
// Clears the first `bytes` (a multiple of 4) of a workspace in a kernel that
// lets the next one of its call start at once: that one, launched with
// launch_pdl, may read the caller's inputs before pdl_wait() and the cleared
// words only behind it.  (A memset in its place costs a call 2 us.)
cudaError_t launch_clear(void* ws, size_t bytes, cudaStream_t st);
// Workspace bytes of the two launchers, the status word's 256 included; for calls of up to n tokens.
size_t paged_decode_ws_bytes(const Prob& pr);
size_t paged_prefill_ws_bytes(const Prob& pr, int64_t n);

}  // namespace pisa
