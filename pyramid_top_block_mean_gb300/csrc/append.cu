// append.cu -- new tokens into the paged cache, keys and queries normed head by
// head and rotated by their positions on the way, and rows read back from it.
//
// A head's norm: x -> x / sqrt(sum x^2 / d + eps) * w, in fp32 and in that
// order (the root's reciprocal times a weight may leave fp32's range).
// For a pair (a, b) of dims with angle theta of the token's position:
//   (a, b) -> (a cos theta - b sin theta, b cos theta + a sin theta)
// with the pairs (i, i + rot / 2) or (2i, 2i + 1); cosines and sines come from
// the caller's table in fp32, so that a model's own frequencies and far
// positions (whose angles need more than 32 bits) are the caller's choice.
// Bound by HBM: every row is read once and written once.  A thread owns 32
// bytes of a row -- the two 16-byte vectors that pair up -- so that a rotation
// needs no exchange and an in-place call reads its pair before it writes it.
// What a norm or an e4m3 row needs of the whole row (its sum of squares, its
// largest magnitude) the 4 to 16 threads of a row exchange by shuffles.  Two
// prompts of up to 4096 tokens, 16 / 4 heads (floor 12.0 us): normed 20.6 us
// (32 with heads of all kinds in a warp, one row's sum after the other), normed
// into e4m3 pages 25.6 us, read back from there 7.1 us.
#include <algorithm>

#include "paged.cuh"

namespace pisa {

namespace {

struct AppendArgs {
  const void *q, *k, *v;
  int64_t qs[3], ks[3], vs[3];
  const int32_t *seq_lens, *new_lens, *table;
  const float* rope;
  void *k_pages, *v_pages, *q_out, *k_out;
  uint8_t *k_scales, *v_scales;
  NormArgs norm;
  int64_t n, nb, num_pages;
  int32_t* status;
  int32_t rot, interleaved;
};

// 16 bytes of T as floats and back (one rounding to T).
template <typename T>
struct Vec;
template <>
struct Vec<float> {
  static constexpr int E = 4;
  static __device__ __forceinline__ void load(const uint4& w, float* x) {
    x[0] = __uint_as_float(w.x); x[1] = __uint_as_float(w.y);
    x[2] = __uint_as_float(w.z); x[3] = __uint_as_float(w.w);
  }
  static __device__ __forceinline__ uint4 store(const float* x) {
    return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
  }
};
template <>
struct Vec<__nv_bfloat16> {
  static constexpr int E = 8;
  static __device__ __forceinline__ void load(const uint4& w, float* x) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(u[i] << 16);
      x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ uint4 store(const float* x) {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
      u[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    return make_uint4(u[0], u[1], u[2], u[3]);
  }
};

// Packed pairs of fp32 values, subnormals kept.
__device__ __forceinline__ uint64_t fma_pair(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t mul_pair(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// Of a row of which this thread holds x[0 .. N): its part of the sum of squares.
template <int N>
__device__ __forceinline__ float sum_of_squares(const float (&x)[N]) {
  uint64_t part[2] = {0ull, 0ull};
#pragma unroll
  for (int j = 0; j < N; j += 2) {
    const uint64_t v = ptx::pack2(x[j], x[j + 1]);
    part[(j >> 1) & 1] = fma_pair(v, v, part[(j >> 1) & 1]);
  }
  float p0, p1, p2, p3;
  ptx::unpack2(part[0], p0, p1);
  ptx::unpack2(part[1], p2, p3);
  return (p0 + p1) + (p2 + p3);
}
// 1 / sqrt(sum / d + eps) of a row whose squares, or their mean and eps, leave
// fp32's range: from the elements over 2^80 and eps over 2^160.  The row's
// threads are those of `mask`, neighbours; 1 / d is exact.
template <int N>
__device__ __forceinline__ float far_row_norm(const float (&x)[N], uint32_t units, unsigned mask, float one_over_d,
                                              float eps) {
  float ss = 0.0f;
#pragma unroll
  for (int j = 0; j < N; ++j) ss = fmaf(x[j] * 0x1p-80f, x[j] * 0x1p-80f, ss);
  for (uint32_t o = 1; o < units; o <<= 1) ss += __shfl_xor_sync(mask, ss, o);
  return 0x1p-80f * rsqrtf(fmaf(ss, one_over_d, eps * 0x1p-80f * 0x1p-80f));
}
// Whether the sum and what the root is taken of are in range.
__device__ __forceinline__ bool near_row(float sum, float mean) { return sum < 3.0e38f && mean < 3.0e38f; }
// 1 / sqrt(sum / d + eps) of a row.
template <int N>
__device__ __forceinline__ float row_norm(const float (&x)[N], uint32_t units, unsigned mask, float one_over_d,
                                          float eps) {
  float ss = sum_of_squares(x);
  for (uint32_t o = 1; o < units; o <<= 1) ss += __shfl_xor_sync(mask, ss, o);
  const float mean = fmaf(ss, one_over_d, eps);
  return near_row(ss, mean) ? rsqrtf(mean) : far_row_norm(x, units, mask, one_over_d, eps);
}

// The bits of the largest magnitude among x (those of infinities and NaN lie above all others').
template <int N>
__device__ __forceinline__ uint32_t largest_bits(const float (&x)[N]) {
  uint32_t top = 0;
#pragma unroll
  for (int j = 0; j < N; ++j) top = max(top, __float_as_uint(x[j]) & 0x7fffffffu);
  return top;
}
// The scale of a row with that largest magnitude: the smallest power of two
// with which it is at most 448 = 1.75 2^8 (a carry out of the mantissa where it
// is above 1.75), 255 if it is not finite.
__device__ __forceinline__ uint32_t scale_of_bits(uint32_t top) {
  if (top >= 0x7f800000u) return 255u;
  const int e = (int)((top + 0x1fffffu) >> 23) - 8;  // biased
  return (uint32_t)min(max(e, 10), 246);
}
template <int N>
__device__ __forceinline__ uint32_t row_scale(const float (&x)[N], uint32_t units, unsigned mask) {
  uint32_t top = largest_bits(x);
  for (uint32_t o = 1; o < units; o <<= 1) top = max(top, __shfl_xor_sync(mask, top, o));
  return scale_of_bits(top);
}

// The E codes of x over the row's power.
template <int E>
__device__ __forceinline__ void store_codes(uint8_t* dst, const float* x, uint32_t scale) {
  const float by = scale == 255u ? 0.0f : __uint_as_float((254u - scale) << 23);
  uint32_t w[E / 4];
#pragma unroll
  for (int j = 0; j < E; j += 4) {
    w[j / 4] = to_codes(x[j] * by, x[j + 1] * by) | to_codes(x[j + 2] * by, x[j + 3] * by) << 16;
    if (scale == 255u) w[j / 4] = 0;  // (a product of zero and infinity is not)
  }
  if constexpr (E == 8) *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[1]);
  else *reinterpret_cast<uint32_t*>(dst) = w[0];
}

// One thread: one 32-byte unit of R rows (q, k and v heads, every groups-th)
// of one token, all of whose loads are in flight together; the token's
// cosines and sines are read once for them.  NORM: with norms; Q8: into e4m3
// pages.
template <typename T, int R, bool NORM, bool Q8>
__device__ __forceinline__ void append_units(const Prob& pr, const AppendArgs& a, int64_t b) {
  constexpr int E = Vec<T>::E;
  const uint32_t units = pr.d / (2 * E);
  const uint32_t kv0 = a.q ? pr.Hq : 0, rows = kv0 + 2 * pr.Hkv, groups = (rows + R - 1) / R;
  const uint32_t per = blockDim.x / units;  // (token, group) pairs of a block
  const uint32_t u = threadIdx.x % units;
  const unsigned mates = ((1u << units) - 1u) << (threadIdx.x % 32 / units * units);  // the row's threads
  const int64_t y = (int64_t)blockIdx.x * per + threadIdx.x / units;
  const int64_t i = y < (int64_t)0xffffffff ? (int64_t)((uint32_t)y / groups) : y / groups;
  const uint32_t r0 = (uint32_t)(y - i * groups);
  if (i >= a.n) return;
  int64_t len, cnt;
  if (!new_span(a.seq_lens, a.new_lens, b, a.n, pr.N, &len, &cnt) || i >= cnt) return;
  const int64_t pos = len - cnt + i;
  const uint32_t page = (uint32_t)a.table[b * a.nb + pos / pr.C];  // a negative entry is past any pool
  const bool in_pool = page < a.num_pages;
  const int half = a.rot / 2;
  const bool turns = (int)(2 * E * u) < a.rot;  // this unit's dims are among the rotated ones
  float cs[E], sn[E];
  if (turns) {
    const float* at = a.rope + pos * a.rot + E * u;
#pragma unroll
    for (int j = 0; j < E; j += 4) {
      const float4 c = *reinterpret_cast<const float4*>(at + j), s = *reinterpret_cast<const float4*>(at + half + j);
      cs[j] = c.x; cs[j + 1] = c.y; cs[j + 2] = c.z; cs[j + 3] = c.w;
      sn[j] = s.x; sn[j + 1] = s.y; sn[j + 2] = s.z; sn[j + 3] = s.w;
    }
  }
  // the unit's two vectors: partners in the rotated dims, neighbours elsewhere
  auto place = [&](bool rotated, int* e0, int* e1) {
    const bool split = rotated && !a.interleaved;
    *e0 = split ? E * u : 2 * E * u;
    *e1 = split ? E * u + half : 2 * E * u + E;
  };
  uint4 w[R][2];
#pragma unroll
  for (int k = 0; k < R; ++k) {
    const uint32_t r = r0 + k * groups;
    if (r >= rows) break;
    const bool is_q = r < kv0, is_v = r >= kv0 + pr.Hkv;
    const int64_t* sd = is_q ? a.qs : (is_v ? a.vs : a.ks);
    const int64_t h = is_q ? r : (is_v ? r - kv0 - pr.Hkv : r - kv0);
    const T* src = (const T*)(is_q ? a.q : (is_v ? a.v : a.k)) + b * sd[0] + h * sd[1] + i * sd[2];
    int e0, e1;
    place(turns && !is_v, &e0, &e1);
    w[k][0] = *reinterpret_cast<const uint4*>(src + e0);
    w[k][1] = *reinterpret_cast<const uint4*>(src + e1);
  }
#pragma unroll
  for (int k = 0; k < R; ++k) {
    const uint32_t r = r0 + k * groups;
    if (r >= rows) break;
    const bool is_q = r < kv0, is_v = r >= kv0 + pr.Hkv;
    const int64_t h = is_q ? r : (is_v ? r - kv0 - pr.Hkv : r - kv0);
    int e0, e1;
    place(turns && !is_v, &e0, &e1);
    const float* weight = !NORM || is_v ? nullptr : (is_q ? a.norm.q : a.norm.k);
    float o[2 * E];
    if (Q8 || weight || (turns && !is_v)) {
      Vec<T>::load(w[k][0], o);
      Vec<T>::load(w[k][1], o + E);
    }
    if (weight) {
      const float by = row_norm(o, units, mates, a.norm.one_over_d, a.norm.eps);
      const uint64_t by2 = ptx::pack2(by, by);
#pragma unroll
      for (int j = 0; j < 2 * E; j += 4) {
        const float4 x = *reinterpret_cast<const float4*>(weight + (j < E ? e0 + j : e1 + j - E));
        ptx::unpack2(mul_pair(mul_pair(ptx::pack2(o[j], o[j + 1]), by2), ptx::pack2(x.x, x.y)), o[j], o[j + 1]);
        ptx::unpack2(mul_pair(mul_pair(ptx::pack2(o[j + 2], o[j + 3]), by2), ptx::pack2(x.z, x.w)), o[j + 2], o[j + 3]);
      }
    }
    if (turns && !is_v) {
      auto turn = [&](float& x, float& z, int j) {
        const float xr = x * cs[j] - z * sn[j], zr = z * cs[j] + x * sn[j];
        x = xr;
        z = zr;
      };
      if (a.interleaved) {
#pragma unroll
        for (int j = 0; j < E; ++j) turn(o[2 * j], o[2 * j + 1], j);
      } else if (NORM || Q8) {  // two pairs at a time
#pragma unroll
        for (int j = 0; j < E; j += 2) {
          const uint64_t x = ptx::pack2(o[j], o[j + 1]), z = ptx::pack2(o[E + j], o[E + j + 1]);
          const uint64_t c = ptx::pack2(cs[j], cs[j + 1]), sp = ptx::pack2(sn[j], sn[j + 1]);
          const uint64_t sm = ptx::pack2(-sn[j], -sn[j + 1]);
          ptx::unpack2(fma_pair(x, c, mul_pair(z, sm)), o[j], o[j + 1]);
          ptx::unpack2(fma_pair(z, c, mul_pair(x, sp)), o[E + j], o[E + j + 1]);
        }
      } else {
#pragma unroll
        for (int j = 0; j < E; ++j) turn(o[j], o[E + j], j);
      }
    }
    if (weight || (turns && !is_v)) {
      w[k][0] = Vec<T>::store(o);
      w[k][1] = Vec<T>::store(o + E);
    }
    if (is_q || (!is_v && a.k_out)) {
      T* dst = (T*)(is_q ? a.q_out : a.k_out) + ((b * (is_q ? pr.Hq : pr.Hkv) + h) * a.n + i) * pr.d;
      *reinterpret_cast<uint4*>(dst + e0) = w[k][0];
      *reinterpret_cast<uint4*>(dst + e1) = w[k][1];
    }
    if (is_q) continue;
    const int64_t row = ((int64_t)page * pr.Hkv + h) * pr.C + pos % pr.C;
    if constexpr (Q8) {
      const uint32_t scale = row_scale(o, units, mates);
      if (in_pool) {
        uint8_t* dst = (uint8_t*)(is_v ? a.v_pages : a.k_pages) + row * pr.d;
        store_codes<E>(dst + e0, o, scale);
        store_codes<E>(dst + e1, o + E, scale);
        if (u == 0) (is_v ? a.v_scales : a.k_scales)[row] = (uint8_t)scale;
      }
    } else if (in_pool) {
      T* dst = (T*)(is_v ? a.v_pages : a.k_pages) + row * pr.d;
      *reinterpret_cast<uint4*>(dst + e0) = w[k][0];
      *reinterpret_cast<uint4*>(dst + e1) = w[k][1];
    }
  }
}

// Long calls with norms or into e4m3 pages: a CTA takes R heads of one kind (q,
// k or v) of its tokens, a thread one 32-byte unit of each, so that all of a
// CTA's threads do the same, the weights and angles of the unit are read once
// for its R rows, and their sums go through the shuffles side by side.
template <typename T, int R, bool NORM, bool Q8>
__device__ __forceinline__ void append_heads(const Prob& pr, const AppendArgs& a, int64_t b) {
  constexpr int E = Vec<T>::E;
  const uint32_t units = pr.d / (2 * E);
  const uint32_t gq = a.q ? (pr.Hq + R - 1) / R : 0, gk = (pr.Hkv + R - 1) / R, groups = gq + 2 * gk;
  const uint32_t chunk = blockIdx.x / groups, g = blockIdx.x - chunk * groups;
  const bool is_q = g < gq, is_v = g >= gq + gk;
  const int h0 = R * (int)(is_q ? g : is_v ? g - gq - gk : g - gq), H = is_q ? pr.Hq : pr.Hkv;
  const uint32_t u = threadIdx.x % units;
  const unsigned mates = ((1u << units) - 1u) << (threadIdx.x % 32 / units * units);  // the row's threads
  const int64_t i = (int64_t)chunk * (blockDim.x / units) + threadIdx.x / units;
  if (i >= a.n) return;
  int64_t len, cnt;
  if (!new_span(a.seq_lens, a.new_lens, b, a.n, pr.N, &len, &cnt) || i >= cnt) return;
  const int64_t pos = len - cnt + i;
  const uint32_t page = is_q ? 0u : (uint32_t)a.table[b * a.nb + pos / pr.C];  // a negative entry is past any pool
  const bool in_pool = !is_q && page < a.num_pages;
  const int half = a.rot / 2;
  const bool turns = !is_v && (int)(2 * E * u) < a.rot;  // this unit's dims are among the rotated ones
  const bool split = turns && !a.interleaved;
  const int e0 = split ? E * u : 2 * E * u, e1 = split ? E * u + half : 2 * E * u + E;
  const int64_t* sd = is_q ? a.qs : (is_v ? a.vs : a.ks);
  const T* src = (const T*)(is_q ? a.q : (is_v ? a.v : a.k)) + b * sd[0] + h0 * sd[1] + i * sd[2];
  uint4 w[R][2];
#pragma unroll
  for (int k = 0; k < R; ++k) {
    if (h0 + k >= H) break;
    w[k][0] = *reinterpret_cast<const uint4*>(src + k * sd[1] + e0);
    w[k][1] = *reinterpret_cast<const uint4*>(src + k * sd[1] + e1);
  }
  float cs[E], sn[E];
  if (turns) {
    const float* at = a.rope + pos * a.rot + E * u;
#pragma unroll
    for (int j = 0; j < E; j += 4) {
      const float4 c = *reinterpret_cast<const float4*>(at + j), s = *reinterpret_cast<const float4*>(at + half + j);
      cs[j] = c.x; cs[j + 1] = c.y; cs[j + 2] = c.z; cs[j + 3] = c.w;
      sn[j] = s.x; sn[j + 1] = s.y; sn[j + 2] = s.z; sn[j + 3] = s.w;
    }
  }
  const float* weight = !NORM || is_v ? nullptr : (is_q ? a.norm.q : a.norm.k);
  uint64_t wt[E];
  float by[R];
  if (weight) {
#pragma unroll
    for (int j = 0; j < 2 * E; j += 4) {
      const float4 x = *reinterpret_cast<const float4*>(weight + (j < E ? e0 + j : e1 + j - E));
      wt[j / 2] = ptx::pack2(x.x, x.y);
      wt[j / 2 + 1] = ptx::pack2(x.z, x.w);
    }
#pragma unroll
    for (int k = 0; k < R; ++k) {
      float x[2 * E];
      Vec<T>::load(w[k][0], x);
      Vec<T>::load(w[k][1], x + E);
      by[k] = h0 + k < H ? sum_of_squares(x) : 0.0f;
    }
    for (uint32_t o = 1; o < units; o <<= 1) {
#pragma unroll
      for (int k = 0; k < R; ++k) by[k] += __shfl_xor_sync(mates, by[k], o);
    }
#pragma unroll
    for (int k = 0; k < R; ++k) {
      const float mean = fmaf(by[k], a.norm.one_over_d, a.norm.eps);
      if (near_row(by[k], mean)) {
        by[k] = rsqrtf(mean);
      } else {
        float x[2 * E];
        Vec<T>::load(w[k][0], x);
        Vec<T>::load(w[k][1], x + E);
        by[k] = far_row_norm(x, units, mates, a.norm.one_over_d, a.norm.eps);
      }
    }
  }
  // row k, normed and rotated
  auto finish = [&](int k, float (&x)[2 * E]) {
    Vec<T>::load(w[k][0], x);
    Vec<T>::load(w[k][1], x + E);
    if (weight) {
      const uint64_t by2 = ptx::pack2(by[k], by[k]);
#pragma unroll
      for (int j = 0; j < 2 * E; j += 2)
        ptx::unpack2(mul_pair(mul_pair(ptx::pack2(x[j], x[j + 1]), by2), wt[j / 2]), x[j], x[j + 1]);
    }
    if (!turns) return;
    if (a.interleaved) {
#pragma unroll
      for (int j = 0; j < E; ++j) {
        const float p = x[2 * j], z = x[2 * j + 1];
        x[2 * j] = p * cs[j] - z * sn[j];
        x[2 * j + 1] = z * cs[j] + p * sn[j];
      }
    } else {
#pragma unroll
      for (int j = 0; j < E; j += 2) {
        const uint64_t p = ptx::pack2(x[j], x[j + 1]), z = ptx::pack2(x[E + j], x[E + j + 1]);
        const uint64_t c = ptx::pack2(cs[j], cs[j + 1]), s = ptx::pack2(sn[j], sn[j + 1]);
        ptx::unpack2(fma_pair(p, c, mul_pair(z, ptx::pack2(-sn[j], -sn[j + 1]))), x[j], x[j + 1]);
        ptx::unpack2(fma_pair(z, c, mul_pair(p, s)), x[E + j], x[E + j + 1]);
      }
    }
  };
  const int64_t ostep = a.n * pr.d, pstep = pr.C * pr.d;  // from head to head
  T* out = is_q ? (T*)a.q_out : is_v ? nullptr : (T*)a.k_out;
  if (out) out += ((b * H + h0) * a.n + i) * pr.d;
  const int64_t row0 = ((int64_t)page * H + h0) * pr.C + pos % pr.C;
  const bool kept = Q8 && !is_q;  // the rows go into e4m3 pages: their numbers are made twice, once for the scale
  uint32_t top[R];
#pragma unroll
  for (int k = 0; k < R; ++k) {
    top[k] = 0;
    if (h0 + k >= H) break;
    uint4 y0 = w[k][0], y1 = w[k][1];
    if (kept || weight || turns) {
      float x[2 * E];
      finish(k, x);
      if (kept) top[k] = largest_bits(x);
      y0 = Vec<T>::store(x);
      y1 = Vec<T>::store(x + E);
    }
    if (out) {
      T* dst = out + k * ostep;
      *reinterpret_cast<uint4*>(dst + e0) = y0;
      *reinterpret_cast<uint4*>(dst + e1) = y1;
    }
    if (!Q8 && in_pool) {
      T* dst = (T*)(is_v ? a.v_pages : a.k_pages) + row0 * pr.d + k * pstep;
      *reinterpret_cast<uint4*>(dst + e0) = y0;
      *reinterpret_cast<uint4*>(dst + e1) = y1;
    }
  }
  if (!kept) return;
  for (uint32_t s = 1; s < units; s <<= 1) {
#pragma unroll
    for (int k = 0; k < R; ++k) top[k] = max(top[k], __shfl_xor_sync(mates, top[k], s));
  }
  if (!in_pool) return;
#pragma unroll
  for (int k = 0; k < R; ++k) {
    if (h0 + k >= H) break;
    float x[2 * E];
    finish(k, x);
    const uint32_t scale = scale_of_bits(top[k]);
    uint8_t* dst = (uint8_t*)(is_v ? a.v_pages : a.k_pages) + row0 * pr.d + k * pstep;
    store_codes<E>(dst + e0, x, scale);
    store_codes<E>(dst + e1, x + E, scale);
    if (u == 0) (is_v ? a.v_scales : a.k_scales)[row0 + k * pr.C] = (uint8_t)scale;
  }
}

// One CTA looks at every length and page for faults and writes the status
// word, so that nothing has to clear it before the call.
__device__ __forceinline__ void write_status(const Prob& pr, const int32_t* seq_lens, const int32_t* new_lens,
                                             const int32_t* table, int64_t n, int64_t nb, int64_t num_pages,
                                             int32_t* status) {
  int bad_len = 0, bad_page = 0;
  const int mates = n > pr.C ? 32 : 1;  // threads that share a sequence's pages
  for (int64_t b = threadIdx.x / mates; b < pr.B; b += blockDim.x / mates) {
    int64_t len, cnt;
    if (!new_span(seq_lens, new_lens, b, n, pr.N, &len, &cnt)) {
      bad_len = 1;
    } else if (cnt > 0) {
      for (int64_t j = (len - cnt) / pr.C + threadIdx.x % mates; j <= (len - 1) / pr.C; j += mates)
        bad_page |= (uint32_t)table[b * nb + j] >= num_pages;
    }
  }
  bad_len = __syncthreads_or(bad_len);
  bad_page = __syncthreads_or(bad_page);
  if (threadIdx.x == 0) *status = bad_len ? PISA_DEV_BAD_SEQ_LEN : (bad_page ? PISA_DEV_BAD_INDEX : PISA_DEV_OK);
}

// Three CTAs on an SM: with four rows a thread the compiler takes 91 registers
// if it may, which leaves two (a 2 x 4096-token prompt 15.1 us, against 13.2).
// HEADS: append_heads(), by CTAs of 128 threads.
constexpr int kHeadsThreads = 128;
template <typename T, int R, bool NORM, bool Q8, bool HEADS>
__global__ void __launch_bounds__(HEADS ? kHeadsThreads : 256, HEADS ? 4 : 3) append_kernel(Prob pr, AppendArgs a) {
  for (int64_t b = blockIdx.y; b < pr.B; b += gridDim.y) {
    if constexpr (HEADS) append_heads<T, R, NORM, Q8>(pr, a, b);
    else append_units<T, R, NORM, Q8>(pr, a, b);
  }
  if (blockIdx.x == 0 && blockIdx.y == 0)
    write_status(pr, a.seq_lens, a.new_lens, a.table, a.n, a.nb, a.num_pages, a.status);
}

struct ReadArgs {
  const void *k_pages, *v_pages;
  const uint8_t *k_scales, *v_scales;
  const int32_t *seq_lens, *new_lens, *table;
  void *k_out, *v_out;
  int64_t n, nb, num_pages;
  int32_t* status;
};

// 16 elements of a row from the pages.
template <typename T, bool Q8>
__device__ __forceinline__ void read_unit(const void* pages, const uint8_t* scales, int64_t row, int e0, int d,
                                          void* out, int64_t to) {
  constexpr int V = sizeof(T);  // 16-byte vectors of the output
  uint4* dst = reinterpret_cast<uint4*>((T*)out + to * d + e0);
  if constexpr (!Q8) {
    const uint4* src = reinterpret_cast<const uint4*>((const T*)pages + row * d + e0);
#pragma unroll
    for (int j = 0; j < V; ++j) dst[j] = src[j];
  } else {
    const uint32_t s = scales[row];
    const uint4 c = *reinterpret_cast<const uint4*>((const uint8_t*)pages + row * d + e0);
    const uint4 lo = row_pairs(make_uint2(c.x, c.y), s), hi = row_pairs(make_uint2(c.z, c.w), s);
    const uint32_t x[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
    for (int j = 0; j < V; ++j) {
      if constexpr (V == 2)
        dst[j] = make_uint4(x[4 * j], x[4 * j + 1], x[4 * j + 2], x[4 * j + 3]);
      else
        dst[j] = make_uint4(x[2 * j] << 16, x[2 * j] & 0xffff0000u, x[2 * j + 1] << 16, x[2 * j + 1] & 0xffff0000u);
    }
  }
}

// One thread: 16 dims of one head of one token, of its key and its value.
template <typename T, bool Q8>
__global__ void __launch_bounds__(256) read_kernel(Prob pr, ReadArgs a) {
  const uint32_t units = pr.d / 16, chunk = blockIdx.x / (uint32_t)pr.Hkv;
  const int e0 = 16 * (int)(threadIdx.x % units);
  const int64_t h = blockIdx.x - chunk * pr.Hkv, i = (int64_t)chunk * (256 / units) + threadIdx.x / units;
  for (int64_t b = blockIdx.y; b < pr.B && i < a.n; b += gridDim.y) {
    int64_t len, cnt;
    if (!new_span(a.seq_lens, a.new_lens, b, a.n, pr.N, &len, &cnt) || i >= cnt) continue;
    const int64_t pos = len - cnt + i;
    const uint32_t page = (uint32_t)a.table[b * a.nb + pos / pr.C];  // a negative entry is past any pool
    if (page >= a.num_pages) continue;
    const int64_t row = ((int64_t)page * pr.Hkv + h) * pr.C + pos % pr.C, to = (b * pr.Hkv + h) * a.n + i;
    if (a.k_out) read_unit<T, Q8>(a.k_pages, a.k_scales, row, e0, pr.d, a.k_out, to);
    if (a.v_out) read_unit<T, Q8>(a.v_pages, a.v_scales, row, e0, pr.d, a.v_out, to);
  }
  if (blockIdx.x == 0 && blockIdx.y == 0)
    write_status(pr, a.seq_lens, a.new_lens, a.table, a.n, a.nb, a.num_pages, a.status);
}

struct ExpandArgs {
  Pools codes, wide;
  const int32_t *seq_lens, *new_lens;
  int64_t n, window;
};

// One CTA: a page of a sequence and a key head; a thread 16 dims of a row of
// keys and of values at a time.  (16384 positions of 4 heads; a CTA for all
// heads of a page, a quarter of the grid, 16 us.)
__global__ void __launch_bounds__(256) expand_kernel(Prob pr, ExpandArgs a) {
  const int64_t j = blockIdx.x, nb = a.codes.nb;
  const int h = blockIdx.z;
  for (int64_t b = blockIdx.y; b < pr.B; b += gridDim.y) {
    int64_t len, cnt;
    if (!new_span(a.seq_lens, a.new_lens, b, a.n, pr.N, &len, &cnt) || cnt == 0 || j > (len - 1) / pr.C) continue;
    // the first new token's window
    if (a.window > 0 && (j + 1) * pr.C <= len - cnt - a.window + 1) continue;
    const uint32_t page = (uint32_t)a.codes.table[b * nb + j];  // a negative entry is past any pool
    const bool in_pool = page < a.codes.num_pages;
    const int64_t to = b * nb + j;
    if (h == 0 && threadIdx.x == 0) const_cast<int32_t*>(a.wide.table)[to] = in_pool ? (int32_t)to : -1;
    if (!in_pool) continue;
    const int units = pr.d / 16;
    const int64_t from = ((int64_t)page * pr.Hkv + h) * pr.C, row0 = (to * pr.Hkv + h) * pr.C;
#pragma unroll 2
    for (int x = threadIdx.x; x < (int)pr.C * units; x += 256) {
      const int r = x / units, e0 = 16 * (x % units);
      read_unit<__nv_bfloat16, true>(a.codes.k, a.codes.ks, from + r, e0, pr.d, const_cast<void*>(a.wide.k), row0 + r);
      read_unit<__nv_bfloat16, true>(a.codes.v, a.codes.vs, from + r, e0, pr.d, const_cast<void*>(a.wide.v), row0 + r);
    }
  }
}

}  // namespace

cudaError_t launch_expand_paged(const Prob& pr, int64_t n, int64_t window, const Pools& codes, const Pools& wide,
                                const int32_t* seq_lens, const int32_t* new_lens, cudaStream_t st) {
  const ExpandArgs a{codes, wide, seq_lens, new_lens, n, window};
  note_launch();
  expand_kernel<<<dim3((unsigned)codes.nb, (unsigned)std::min<int64_t>(pr.B, 65535), (unsigned)pr.Hkv), 256, 0, st>>>(
      pr, a);
  return cudaGetLastError();
}

cudaError_t launch_append_paged(const Prob& pr, int64_t n, const void* q, const int64_t* qs, const void* k,
                                const int64_t* ks, const void* v, const int64_t* vs, const int32_t* seq_lens,
                                const int32_t* new_lens, const NormArgs& norm, const float* rope, int rot_dim,
                                int interleaved, const Pools& pools, int32_t* status, void* q_out, void* k_out,
                                cudaStream_t st) {
  AppendArgs a{};
  a.q = q; a.k = k; a.v = v;
  for (int i = 0; i < 3; ++i) { a.qs[i] = qs[i]; a.ks[i] = ks[i]; a.vs[i] = vs[i]; }
  a.seq_lens = seq_lens; a.new_lens = new_lens; a.table = pools.table;
  a.rope = rope; a.rot = rot_dim; a.interleaved = interleaved != 0;
  a.k_pages = const_cast<void*>(pools.k); a.v_pages = const_cast<void*>(pools.v);
  a.k_scales = const_cast<uint8_t*>(pools.ks); a.v_scales = const_cast<uint8_t*>(pools.vs);
  a.norm = norm; a.norm.one_over_d = 1.0f / (float)pr.d; a.q_out = q_out; a.k_out = k_out;
  a.n = n; a.nb = pools.nb; a.num_pages = pools.num_pages; a.status = status;
  const int per = 256 / (pr.d / (pr.dtype == PISA_BF16 ? 16 : 8));
  const int64_t rows = (q ? pr.Hq : 0) + 2 * pr.Hkv;
  // Four rows a thread once that fills the GPU: 13.2 us for 2 x 4096 tokens of
  // 16 + 2 x 4 heads (12.0 us at the copy rate), where one row a thread took
  // 18.2; a step of 64 tokens (2.7 us) has too few rows to give up any thread.
  const bool many = pr.B * n * rows * (256 / per) >= 4 * 152 * 2048;
  const bool normed = norm.q || norm.k, in8 = pools.ks != nullptr, heads = many && (normed || in8) && n >= per / 2;
  const int R = heads || (many && !normed && !in8) ? 4 : 1;
  const int64_t groups = (q ? ceil_div64(pr.Hq, R) : 0) + 2 * ceil_div64(pr.Hkv, R);
  const int threads = heads ? kHeadsThreads : 256, hper = kHeadsThreads / (256 / per);
  const dim3 grid((unsigned)(heads ? ceil_div64(n, hper) * groups : ceil_div64(n * ceil_div64(rows, R), per)),
                  (unsigned)std::min<int64_t>(pr.B, 65535));
  auto pick = [&](auto type) {
    using T = decltype(type);
    auto form = [&](auto nn, auto qq) {
      constexpr bool N = decltype(nn)::value, Q = decltype(qq)::value;
      if (heads) return append_kernel<T, 4, N, Q, N || Q>;
      return R == 4 ? append_kernel<T, 4, false, false, false> : append_kernel<T, 1, N, Q, false>;
    };
    using Yes = std::true_type;
    using No = std::false_type;
    return normed ? (in8 ? form(Yes(), Yes()) : form(Yes(), No())) : (in8 ? form(No(), Yes()) : form(No(), No()));
  };
  auto kern = pr.dtype == PISA_BF16 ? pick(__nv_bfloat16()) : pick(float());
  note_launch();
  kern<<<grid, threads, 0, st>>>(pr, a);
  return cudaGetLastError();
}

cudaError_t launch_read_paged(const Prob& pr, int64_t n, const Pools& pools, const int32_t* seq_lens,
                              const int32_t* new_lens, int32_t* status, void* k_out, void* v_out, cudaStream_t st) {
  ReadArgs a{};
  a.k_pages = pools.k; a.v_pages = pools.v;
  a.k_scales = pools.ks; a.v_scales = pools.vs;
  a.seq_lens = seq_lens; a.new_lens = new_lens; a.table = pools.table;
  a.k_out = k_out; a.v_out = v_out;
  a.n = n; a.nb = pools.nb; a.num_pages = pools.num_pages; a.status = status;
  const dim3 grid((unsigned)(ceil_div64(n * (pr.d / 16), 256) * pr.Hkv), (unsigned)std::min<int64_t>(pr.B, 65535));
  const bool in8 = pools.ks != nullptr;
  auto kern = pr.dtype == PISA_BF16 ? (in8 ? read_kernel<__nv_bfloat16, true> : read_kernel<__nv_bfloat16, false>)
                                    : (in8 ? read_kernel<float, true> : read_kernel<float, false>);
  note_launch();
  kern<<<grid, 256, 0, st>>>(pr, a);
  return cudaGetLastError();
}

}  // namespace pisa
