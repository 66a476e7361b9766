// append.cu -- new tokens into the paged cache, keys and queries rotated by
// their positions on the way.
//
// For a pair (a, b) of dims with angle theta of the token's position:
//   (a, b) -> (a cos theta - b sin theta, b cos theta + a sin theta)
// with the pairs (i, i + rot / 2) or (2i, 2i + 1); cosines and sines come from
// the caller's table in fp32, so that a model's own frequencies and far
// positions (whose angles need more than 32 bits) are the caller's choice.
// Bound by HBM: every row is read once and written once.  A thread owns 32
// bytes of a row -- the two 16-byte vectors that pair up -- so that a rotation
// needs no exchange and an in-place call reads its pair before it writes it.
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

// One thread: one 32-byte unit of one row (q, k or v head) of one token.
template <typename T>
__device__ __forceinline__ void append_unit(const Prob& pr, const AppendArgs& a, int64_t b) {
  constexpr int E = Vec<T>::E;
  const int units = pr.d / (2 * E);
  const int rows = (a.q ? pr.Hq : 0) + 2 * pr.Hkv;
  const int64_t x = blockIdx.x * (int64_t)blockDim.x + threadIdx.x;
  const int u = (int)(x % units);
  const int64_t y = x / units;
  const int r = (int)(y % rows);
  const int64_t i = y / rows;
  if (i >= a.n) return;
  int64_t len, cnt;
  if (!new_span(a.seq_lens, a.new_lens, b, a.n, pr.N, &len, &cnt)) {
    if (x == 0) {
      pdl_wait();
      set_status(a.status, PISA_DEV_BAD_SEQ_LEN);
    }
    return;
  }
  if (i >= cnt) return;
  const int64_t pos = len - cnt + i;
  const int kv0 = a.q ? pr.Hq : 0;
  const bool is_q = r < kv0, is_k = !is_q && r < kv0 + pr.Hkv;
  const int h = is_q ? r : (is_k ? r - kv0 : r - kv0 - pr.Hkv);
  const int half = a.rot / 2;
  // the unit's two vectors: partners in the rotated dims, neighbours elsewhere
  int e0 = 2 * E * u, e1 = e0 + E;
  const bool rotated = (is_q || is_k) && 2 * E * u < a.rot;
  if (rotated && !a.interleaved) {
    e0 = E * u;
    e1 = e0 + half;
  }
  const int64_t* sd = is_q ? a.qs : (is_k ? a.ks : a.vs);
  const T* src = (const T*)(is_q ? a.q : (is_k ? a.k : a.v)) + b * sd[0] + h * sd[1] + i * sd[2];
  uint4 w0 = *reinterpret_cast<const uint4*>(src + e0), w1 = *reinterpret_cast<const uint4*>(src + e1);
  if (rotated) {
    float p[2 * E], o[2 * E];
    Vec<T>::load(w0, p);
    Vec<T>::load(w1, p + E);
    const float* cs = a.rope + pos * a.rot + E * u;
    if (a.interleaved) {
#pragma unroll
      for (int j = 0; j < E; ++j) {
        const float c = cs[j], sn = cs[half + j];
        o[2 * j] = p[2 * j] * c - p[2 * j + 1] * sn;
        o[2 * j + 1] = p[2 * j + 1] * c + p[2 * j] * sn;
      }
    } else {
#pragma unroll
      for (int j = 0; j < E; ++j) {
        const float c = cs[j], sn = cs[half + j];
        o[j] = p[j] * c - p[E + j] * sn;
        o[E + j] = p[E + j] * c + p[j] * sn;
      }
    }
    w0 = Vec<T>::store(o);
    w1 = Vec<T>::store(o + E);
  }
  if (is_q) {
    T* dst = (T*)a.q_out + ((b * pr.Hq + h) * a.n + i) * pr.d;
    *reinterpret_cast<uint4*>(dst + e0) = w0;
    *reinterpret_cast<uint4*>(dst + e1) = w1;
    return;
  }
  if (is_k && a.k_out) {
    T* dst = (T*)a.k_out + ((b * pr.Hkv + h) * a.n + i) * pr.d;
    *reinterpret_cast<uint4*>(dst + e0) = w0;
    *reinterpret_cast<uint4*>(dst + e1) = w1;
  }
  const int64_t page = a.table[b * a.nb + pos / pr.C];
  if (page < 0 || page >= a.num_pages) {
    if (u == 0) {
      pdl_wait();
      set_status(a.status, PISA_DEV_BAD_INDEX);
    }
    return;
  }
  T* dst = (T*)(is_k ? a.k_pages : a.v_pages) + ((page * pr.Hkv + h) * pr.C + pos % pr.C) * pr.d;
  *reinterpret_cast<uint4*>(dst + e0) = w0;
  *reinterpret_cast<uint4*>(dst + e1) = w1;
}

template <typename T>
__global__ void __launch_bounds__(256) append_kernel(Prob pr, AppendArgs a) {
  for (int64_t b = blockIdx.y; b < pr.B; b += gridDim.y) append_unit<T>(pr, a, b);
  pdl_wait();
}

}  // namespace

cudaError_t launch_append_paged(const Prob& pr, int64_t n, const void* q, const int64_t* qs, const void* k,
                                const int64_t* ks, const void* v, const int64_t* vs, const int32_t* seq_lens,
                                const int32_t* new_lens, const float* rope, int rot_dim, int interleaved,
                                void* k_pages, void* v_pages, const int32_t* table, int64_t nb, int64_t num_pages,
                                int32_t* status, void* q_out, void* k_out, cudaStream_t st) {
  AppendArgs a{};
  a.q = q; a.k = k; a.v = v;
  for (int i = 0; i < 3; ++i) { a.qs[i] = qs[i]; a.ks[i] = ks[i]; a.vs[i] = vs[i]; }
  a.seq_lens = seq_lens; a.new_lens = new_lens; a.table = table;
  a.rope = rope; a.rot = rot_dim; a.interleaved = interleaved != 0;
  a.k_pages = k_pages; a.v_pages = v_pages; a.q_out = q_out; a.k_out = k_out;
  a.n = n; a.nb = nb; a.num_pages = num_pages; a.status = status;
  const int E = pr.dtype == PISA_BF16 ? 8 : 4;
  const int64_t threads = n * ((q ? pr.Hq : 0) + 2 * pr.Hkv) * (pr.d / (2 * E));
  const dim3 grid((unsigned)ceil_div64(threads, 256), (unsigned)std::min<int64_t>(pr.B, 65535));
  note_launch();
  return launch_pdl(true, pr.dtype == PISA_BF16 ? append_kernel<__nv_bfloat16> : append_kernel<float>, grid, dim3(256),
                    0, st, pr, a);
}

}  // namespace pisa
