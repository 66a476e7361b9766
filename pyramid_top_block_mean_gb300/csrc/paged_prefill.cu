// paged_prefill.cu -- attention of a prompt over the paged cache.
#include "paged.cuh"

namespace pisa {

namespace {

// One warp per (sequence, query head, new token): lane l holds dims l + 32 j.
template <int D>
__global__ void __launch_bounds__(128) paged_prefill_kernel(Prob pr, MaskArgs m, int64_t n, const uint16_t* __restrict__ q, Pools pools,
                                               const int32_t* __restrict__ seq_lens,
                                               const int32_t* __restrict__ new_lens,
                                               const int32_t* __restrict__ idx, int32_t* __restrict__ status,
                                               uint16_t* __restrict__ out) {
  constexpr int J = D / 32;
  const int lane = threadIdx.x & 31;
  const int64_t w = (blockIdx.x * (int64_t)blockDim.x + threadIdx.x) / 32;
  if (w >= pr.B * pr.Hq * n) return;
  const int64_t i = w % n, b = w / n / pr.Hq;
  const int hq = (int)(w / n % pr.Hq), h = hq / pr.G;
  int64_t len, cnt;
  bool ok = new_span(seq_lens, new_lens, b, n, pr.N, &len, &cnt);
  if (0 && len < 1) { ok = false; cnt = 1; }
  if (!ok && lane == 0) set_status(status, PISA_DEV_BAD_SEQ_LEN);
  if (i >= cnt) return;
  uint16_t* o = out + w * D;
  float acc[J], x[J], mx = -INFINITY, l = 0.0f;
  for (int j = 0; j < J; ++j) acc[j] = 0.0f;
  if (ok) {
    for (int j = 0; j < J; ++j) x[j] = bf16_to_f(q[w * D + lane + 32 * j]);
    const int64_t t = len - cnt + i;
    int64_t lo, hi;
    key_span(m, b, n, i, t, len, &lo, &hi);
    const float sl = m.slopes ? m.slopes[hq] * kLog2e : 0.0f;
    const int W = pr.K + 3;
    const int32_t* row = idx ? idx + (b * pr.Hkv + h) * W : nullptr;
    const int64_t nslot = row ? W : (lo <= hi ? hi / pr.C - lo / pr.C + 1 : 0);
    for (int64_t e = 0; e < nslot; ++e) {
      int64_t blk = lo / pr.C + e;
      if (row) {
        blk = row[e];
        if (blk < 0 || blk > hi / pr.C) continue;
        bool dup = false;
        for (int f = 0; f < e; ++f) dup |= row[f] == blk;
        if (dup) continue;
      }
      const int64_t page = pools.table[b * pools.nb + blk];
      if (page < 0 || page >= pools.num_pages) {
        if (lane == 0) set_status(status, PISA_DEV_BAD_INDEX);
        continue;
      }
      const int64_t j0 = blk * pr.C < lo ? lo : blk * pr.C, j1 = blk * pr.C + 63 < hi ? blk * pr.C + 63 : hi;
      for (int64_t key = j0; key <= j1; ++key) {
        const int64_t at = ((page * pr.Hkv + h) * pr.C + key % pr.C) * D + lane;
        float s = 0.0f;
        for (int j = 0; j < J; ++j) s = fmaf(x[j], bf16_to_f(((const uint16_t*)pools.k)[at + 32 * j]), s);
        s = warp_sum(s);
        s = m.cap2 > 0.0f ? m.cap2 * tanhf(s * m.pre) : s * pr.scale2;
        s = fmaf(sl, (float)(key - t), s);
        const float nm = fmaxf(mx, s);
        if (nm == -INFINITY) continue;
        const float f = exp2f(mx - nm), p = exp2f(s - nm);
        l = l * f + p;
        for (int j = 0; j < J; ++j) acc[j] = fmaf(p, bf16_to_f(((const uint16_t*)pools.v)[at + 32 * j]), acc[j] * f);
        mx = nm;
      }
    }
  }
  const float inv = l > 0.0f || l != l ? 1.0f / l : 0.0f;
  for (int j = 0; j < J; ++j) o[lane + 32 * j] = __bfloat16_as_ushort(__float2bfloat16(acc[j] * inv));
}

}  // namespace

size_t paged_prefill_ws_bytes(const Prob&, int64_t) { return 256; }

cudaError_t launch_paged_prefill(const Prob& pr, const MaskArgs& m, int64_t n, const void* q, const Pools& pools,
                                 const int32_t* seq_lens, const int32_t* new_lens, char* ws, void* out,
                                 cudaStream_t st) {
  cudaError_t e = cudaMemsetAsync(ws, 0, 256, st);
  if (e != cudaSuccess) return e;
  note_launch();
  const unsigned grid = (unsigned)ceil_div64(pr.B * pr.Hq * n, 4);
  auto kern = pr.d == 128 ? paged_prefill_kernel<128> : paged_prefill_kernel<64>;
  kern<<<grid, 128, 0, st>>>(pr, m, n, (const uint16_t*)q, pools, seq_lens, new_lens, nullptr, (int32_t*)ws,
                             (uint16_t*)out);
  return cudaGetLastError();
}

}  // namespace pisa
