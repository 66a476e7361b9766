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

// One thread: one 32-byte unit of R rows (q, k and v heads, every groups-th)
// of one token, all of whose loads are in flight together; the token's
// cosines and sines are read once for them.
template <typename T, int R>
__device__ __forceinline__ void append_units(const Prob& pr, const AppendArgs& a, int64_t b) {
  constexpr int E = Vec<T>::E;
  const uint32_t units = pr.d / (2 * E);
  const uint32_t kv0 = a.q ? pr.Hq : 0, rows = kv0 + 2 * pr.Hkv, groups = (rows + R - 1) / R;
  const uint32_t per = blockDim.x / units;  // (token, group) pairs of a block
  const uint32_t u = threadIdx.x % units;
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
    if (turns && !is_v) {
      float p[2 * E], o[2 * E];
      Vec<T>::load(w[k][0], p);
      Vec<T>::load(w[k][1], p + E);
#pragma unroll
      for (int j = 0; j < E; ++j) {
        const float x = a.interleaved ? p[2 * j] : p[j], z = a.interleaved ? p[2 * j + 1] : p[E + j];
        const float xr = x * cs[j] - z * sn[j], zr = z * cs[j] + x * sn[j];
        if (a.interleaved) {
          o[2 * j] = xr;
          o[2 * j + 1] = zr;
        } else {
          o[j] = xr;
          o[E + j] = zr;
        }
      }
      w[k][0] = Vec<T>::store(o);
      w[k][1] = Vec<T>::store(o + E);
    }
    if (is_q || (!is_v && a.k_out)) {
      T* dst = (T*)(is_q ? a.q_out : a.k_out) + ((b * (is_q ? pr.Hq : pr.Hkv) + h) * a.n + i) * pr.d;
      *reinterpret_cast<uint4*>(dst + e0) = w[k][0];
      *reinterpret_cast<uint4*>(dst + e1) = w[k][1];
    }
    if (!is_q && in_pool) {
      T* dst = (T*)(is_v ? a.v_pages : a.k_pages) + (((int64_t)page * pr.Hkv + h) * pr.C + pos % pr.C) * pr.d;
      *reinterpret_cast<uint4*>(dst + e0) = w[k][0];
      *reinterpret_cast<uint4*>(dst + e1) = w[k][1];
    }
  }
}

// Three CTAs on an SM: with four rows a thread the compiler takes 91 registers
// if it may, which leaves two (a 2 x 4096-token prompt 15.1 us, against 13.2).
template <typename T, int R>
__global__ void __launch_bounds__(256, 3) append_kernel(Prob pr, AppendArgs a) {
  for (int64_t b = blockIdx.y; b < pr.B; b += gridDim.y) append_units<T, R>(pr, a, b);
  // One CTA looks at every length and page for faults and writes the status
  // word, so that nothing has to clear it before the call.
  if (blockIdx.x != 0 || blockIdx.y != 0) return;
  int bad_len = 0, bad_page = 0;
  for (int64_t b = threadIdx.x; b < pr.B; b += blockDim.x) {
    int64_t len, cnt;
    if (!new_span(a.seq_lens, a.new_lens, b, a.n, pr.N, &len, &cnt)) {
      bad_len = 1;
    } else if (cnt > 0) {
      for (int64_t j = (len - cnt) / pr.C; j <= (len - 1) / pr.C; ++j)
        bad_page |= (uint32_t)a.table[b * a.nb + j] >= a.num_pages;
    }
  }
  bad_len = __syncthreads_or(bad_len);
  bad_page = __syncthreads_or(bad_page);
  if (threadIdx.x == 0) *a.status = bad_len ? PISA_DEV_BAD_SEQ_LEN : (bad_page ? PISA_DEV_BAD_INDEX : PISA_DEV_OK);
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
  const int per = 256 / (pr.d / (pr.dtype == PISA_BF16 ? 16 : 8));
  const int64_t rows = (q ? pr.Hq : 0) + 2 * pr.Hkv;
  // Four rows a thread once that fills the GPU: 13.2 us for 2 x 4096 tokens of
  // 16 + 2 x 4 heads (12.0 us at the copy rate), where one row a thread took
  // 18.2; a step of 64 tokens (2.7 us) has too few rows to give up any thread.
  const bool many = pr.B * n * rows * (256 / per) >= 4 * 152 * 2048;
  const dim3 grid((unsigned)ceil_div64(n * ceil_div64(rows, many ? 4 : 1), per),
                  (unsigned)std::min<int64_t>(pr.B, 65535));
  auto kern = pr.dtype == PISA_BF16 ? (many ? append_kernel<__nv_bfloat16, 4> : append_kernel<__nv_bfloat16, 1>)
                                    : (many ? append_kernel<float, 4> : append_kernel<float, 1>);
  note_launch();
  kern<<<grid, 256, 0, st>>>(pr, a);
  return cudaGetLastError();
}

}  // namespace pisa
