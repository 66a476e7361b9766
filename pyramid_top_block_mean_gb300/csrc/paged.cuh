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

// Key and value pools [num_pages, Hkv, 64, d] behind one page table [B, nb];
// with scales [num_pages, Hkv, 64] (not null) their elements are e4m3.
struct Pools {
  const void* k;
  const void* v;
  const int32_t* table;
  int64_t num_pages, nb;
  const uint8_t *ks, *vs;
  void* scratch;  // nullable: room for e4m3 pages expanded to bf16
  size_t scratch_bytes;
};

// What appending does besides moving rows: norms (weights null: none), angles.
struct NormArgs {
  const float *q, *k;
  float eps, one_over_d;
};

// e4m3 rows.  A code c of a row with the scale s stands for c 2^(s - 127): the
// bits of c, its sign apart, placed 4 bits up are the bf16 number c 2^-120 (for
// subnormal codes too), and a product with 2^(s - 7) makes it the row's number,
// exactly.  That power is a bf16 number up to s = 134; beyond (rows with values
// over 57344) a second product does the rest.  A scale of 255 gives NaN.
__device__ __forceinline__ uint32_t row_factor(uint32_t scale) {  // in both halves of a pair
  const uint32_t f = scale == 255u ? 0x7fc0u : (scale < 134u ? scale + 120u : 254u) << 7;
  return f * 0x10001u;
}
__device__ __forceinline__ bool row_is_large(uint32_t scale) { return scale > 134u && scale != 255u; }
__device__ __forceinline__ uint32_t row_factor_large(uint32_t scale) {
  return (row_is_large(scale) ? scale - 134u + 127u : 127u) * 0x800080u;
}
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
// Two codes, each with its sign in all bits of the byte above it (prmt's
// replicating selectors), as bf16 numbers times 2^-120.
__device__ __forceinline__ uint32_t codes_to_bf16(uint32_t x) { return (x << 4) & 0x87f087f0u; }
// The codes of bytes 0 and 1, and of bytes 2 and 3, of a word.
__device__ __forceinline__ uint32_t codes_lo(uint32_t w) {
  uint32_t x;
  asm("prmt.b32 %0, %1, 0, 0x9180;" : "=r"(x) : "r"(w));
  return codes_to_bf16(x);
}
__device__ __forceinline__ uint32_t codes_hi(uint32_t w) {
  uint32_t x;
  asm("prmt.b32 %0, %1, 0, 0xb3a2;" : "=r"(x) : "r"(w));
  return codes_to_bf16(x);
}
// The codes of bytes 0 and 1, and of bytes 2 and 3, in fp16, of which every
// code is a number (NaN's codes stay NaN).
__device__ __forceinline__ void codes_to_half(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 a, b;\n\t"
      "mov.b32 {a, b}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, a;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}
// Two numbers, already over their row's power, to the nearest codes.
__device__ __forceinline__ uint32_t to_codes(float lo, float hi) {
  uint16_t d;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(d) : "f"(hi), "f"(lo));
  return d;
}

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
__device__ __forceinline__ float cap_small(const MaskArgs& m, float x) {
  const float y = x * m.by, w = y * y;
  return x * fmaf(w, fmaf(w, fmaf(w, m.tk[3], m.tk[2]), m.tk[1]), m.tk[0]);
}
__device__ __forceinline__ float cap_score(const MaskArgs& m, float x) {
  const float y = x * m.by, small = cap_small(m, x);
  const float large = fmaf(-2.0f * m.cap2, __frcp_rn(1.0f + ptx::ex2(x * m.pre * (2.0f * kLog2e))), m.cap2);
  return fabsf(y) <= m.lim ? small : large;
}

cudaError_t launch_append_paged(const Prob& pr, int64_t n, const void* q, const int64_t* qs, const void* k,
                                const int64_t* ks, const void* v, const int64_t* vs, const int32_t* seq_lens,
                                const int32_t* new_lens, const NormArgs& norm, const float* rope, int rot_dim,
                                int interleaved, const Pools& pools, int32_t* status, void* q_out, void* k_out,
                                cudaStream_t st);
cudaError_t launch_read_paged(const Prob& pr, int64_t n, const Pools& pools, const int32_t* seq_lens,
                              const int32_t* new_lens, int32_t* status, void* k_out, void* v_out, cudaStream_t st);
// Expands the e4m3 pages that a call of n tokens (with a window, 0: none) can see
// to bf16 pages: page j of sequence b becomes page b nb + j of `wide`, whose
// table it gets (-1 for one outside the pool).
cudaError_t launch_expand_paged(const Prob& pr, int64_t n, int64_t window, const Pools& codes, const Pools& wide,
                                const int32_t* seq_lens, const int32_t* new_lens, cudaStream_t st);
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
size_t paged_prefill_scratch_bytes(const Prob& pr, int64_t n);

}  // namespace pisa
