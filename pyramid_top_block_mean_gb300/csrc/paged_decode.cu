// paged_decode.cu -- attention of one new token per sequence over the paged
// cache: all of it (pisa_dense_decode_paged) or the blocks that the selector
// chose (pisa_attend_decode_paged).
//
// For each query head, o = sum_j p_j v_j / sum_j p_j with p_j = 2^(x_j - m),
// x_j the key's score in log2 units and m their running maximum; parts over
// disjoint keys join by (m, l, o) -> (M, sum l 2^(m - M), sum o 2^(m - M)).
// Bound by HBM: the G heads of a group share every key and value, so a page
// costs 256 d bytes and G / 2 multiply-adds per byte.
//
// The unit of work is one page (64 keys and values) of one (sequence, key
// head).  All units of a call are numbered sequence by sequence, head by head
// and cut into equal runs, one per CTA and SM, so a long sequence spreads over
// the GPU and short ones share a CTA; every CTA derives the cut from the
// lengths on the device.  A producer warp brings the run's pages by TMA
// (128-byte swizzle, so that every ldmatrix below is free of bank conflicts)
// into a ring of stages (128 to 192 KB in flight on an SM); two groups of four warps
// take alternate pages, a warp 16 of a page's 64 keys, and hold their own (m,
// l, o): S = K q by m16n8k16 MMAs with the heads as the 8 columns, O^T += V^T P
// with P turned in registers by movmatrix.  A page takes a group about 1300
// cycles, nearly all latency, which is what the second group hides.  At the
// end of its part of a (sequence, head) three more warps merge the eight while
// the stream goes on.  A part that is not the whole goes to the workspace in
// fp32, and the CTA that brings the last one joins them in the order of the
// CTAs, so results do not depend on timing.
//
// 8-bit pages (Q8) are half the bytes, and the work on them has to keep up: a
// page's loads take 700 cycles of an SM at the copy rate.
//   - S = K q by m16n8k32 MMAs on the codes as they are.  A bf16 query is the sum
//     of two e4m3 rows (split_query): for up to four heads both are columns of
//     one MMA, for eight each has its own.  A key's power of two is a factor of
//     its scores.  Of a query with dims far below its largest the two rows leave
//     something out: where that may count with a page's keys (a bound, found with
//     the query, on their scales), its scores are made again in bf16.
//   - The values' codes become bf16 as their bits stand (c 2^-120), paired over
//     neighbouring keys by byte permutes, and O^T += V^T P in bf16 with the powers
//     of two of the rows in P.  bf16 has fp32's range: a weight keeps its 8 bits
//     however small it is, and whatever the sizes of the other rows.  (In fp16,
//     two codes an instruction, 64 x 8k took 136 us for 139, but weights far
//     below the largest row's were lost.)
//   - The reference of the weights follows the maximum only when that has
//     grown by 2^8: as a rule one vote takes the place of the reductions.
//   - A thread reads whole 16-byte pieces: the order of the contraction, and
//     of O's rows, is the one in which they come, so that nothing is exchanged,
//     and the stage is free before the work on it begins.
//   - Four groups of two warps, 32 keys each; the producer fills two stages at
//     a time, whose waits and addresses then share their latency.
// 64 sequences of up to 8192 tokens, capped, 140 us (5.6 TB/s), 2 x 131072
// tokens 90 us (5.5 TB/s), 64 sequences' 35 selected blocks 69 us (4.3 TB/s).
// With the work left out the loads alone take 125 and 81 us.  Steps: keys and
// values converted to bf16 in registers 214, 124 and 86 us; keys as operands,
// a stage at a time 205 and 124; a stage of every group at once 199 and 101;
// fp16 values, early release, 32 keys a warp 157 and 94; votes 150 and 91;
// both parts of the queries in one MMA 133 and 84; values' bits as bf16 137 and
// 87; the look at what queries leave out 138 and 87 (kernel times).  Two producer
// warps in turn: 154 and 92 against 150 and 91.
//
// Measured (GB300): 64 ragged sequences of up to 8192 tokens, 32 / 8 heads, d
// = 128: 237 us, 6.6 TB/s of keys and values (the copy rate is 6.8); 2 x 131072
// tokens 150 us (6.5 TB/s); 64 sequences' 35 selected blocks 97 us (6.0 TB/s);
// one sequence of 197 tokens 6.8 us.
#include <cuda_fp16.h>

#include <algorithm>

#include "paged.cuh"
#include "tc_ptx.cuh"

namespace pisa {

namespace {

constexpr int kMerge = 96;              // threads that merge a part while the consumers are at the next one
constexpr int kPage = 64;
constexpr int kMaxCtas = 1024;          // part slots in the workspace: two per CTA
constexpr float kSlack = 8.0f;          // Q8: log2 of how far weights may exceed 1
// Q8: P = p 2^(scale - 127 + 111) and values times 2^-120 give O times 2^-9.  Of
// rows over 448 2^kNear that P would leave the range (with p up to 2^8, 2^126):
// from there on a part has P = p 2^(scale - 127), values times 2^-34 and so O.
constexpr int kNear = 134, kNearLift = 111, kNearO = 9, kFarO = 34;
constexpr uint32_t kFarValues = (uint32_t)(127 + 120 - kFarO) * 0x800080u;
constexpr int kScaleLanes = 2 * kPage / 16;  // lanes that bring a page's scales

// Q8: pages of e4m3.
template <int D, int G, bool Q8>
struct Shape {
  static constexpr int kGroups = Q8 ? 4 : 2;  // of consumer warps, which take turns at the pages
  static constexpr int kKeys = Q8 ? 32 : 16;  // of a page a warp takes
  static constexpr int kGroupWarps = kPage / kKeys;
  static constexpr int kWarps = kGroupWarps * kGroups;
  static constexpr int kCons = 32 * kWarps;        // consumer threads
  static constexpr int kThreads = kCons + 32 + kMerge;  // and the producer warp
  static constexpr int kBatch = 2;  // stages that the producer fills at once
  static_assert(!Q8 || kBatch * kScaleLanes <= 32, "a warp brings the scales of a batch at once");
  // as many as fit beside the merge buffer; a multiple of the groups, so that
  // a stage always goes to the same one, which then sees each of its phases
  static constexpr int kStages = Q8 ? (D == 128 ? 8 : 16) : D == 128 ? (G == 8 ? 4 : 6) : (G == 8 ? 10 : 12);
  static_assert(kStages % kGroups == 0, "a group must see every phase of its stages");
  
  static constexpr uint32_t kTile = kPage * D * (Q8 ? 1 : 2);  // bytes of a page's keys
};

// What a stage holds and what to do with it.
struct __align__(16) Meta {
  int32_t item;      // b * Hkv + h, -1: the end
  int32_t rel;       // position of the page's first key minus the query's
  int16_t klo, khi;  // keys klo .. khi of the page are seen
  int16_t first, last;    // of what a group gets of this CTA's part of the item
  int32_t cfirst, parts;  // with last: the item's first CTA and how many share it
  int32_t slot;           // with last and parts > 1: where this part goes
  int32_t slot0;          // and where the first CTA's part goes
};

// The join of an item's parts: 8 dims a thread; where that leaves threads
// over, they take every kLanes-th part.
template <int D, int G>
struct Join {
  static constexpr int kCols = G * D / 8;
  static constexpr int kLanes = kCols * 2 <= kMerge ? kMerge / kCols : 1;
  static constexpr int kStep = kLanes > 1 ? kCols : kMerge;
};

template <int D, int G, bool Q8>
struct Smem {
  using S = Shape<D, G, Q8>;
  uint8_t kv[S::kStages][2][S::kTile];
  uint16_t q[S::kStages][G * D];
  uint8_t scale[Q8 ? S::kStages : 1][2][Q8 ? kPage : 16];
  float o[S::kWarps][G * D];                  // a part's merge
  float m[S::kWarps][8], l[S::kWarps][8];
  // Q8: the columns' 1 / s, and a page's scores for which the query's parts do not do
  float by[Q8 ? S::kWarps : 1][8], more[Q8 && G <= 4 ? S::kWarps : 1][2][2][Q8 && G <= 4 ? 32 : 1];
  float jo[kMerge][8], jm[kMerge], jl[kMerge];
  Meta meta[S::kStages], part;
  uint64_t full[S::kStages], empty[S::kStages], mfull, mempty;
  int32_t abort, zero, last_part;
};
// Where a merge buffer keeps dim c of head g: permuted, so that the stores of
// a warp's fragments spread over the banks (see the two forms of them below).
template <int D, bool Q8>
__device__ __forceinline__ int o_at(int g, int c) {
  if (!Q8) return g * D + (c ^ (8 * (g >> 1)));
  return g * D + (c ^ (2 * (c / (D / 8) & (D / 16 - 1))) ^ (2 * (g >> 1 & 1)));
}

// Parts: fp32 m[G], l[G], o[G][D] per slot; counters of arrived parts per item.
struct Parts {
  int32_t* counter;
  float* ml;
  float* o;
};

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ bool merge_all(bool ok) {  // true for all merging threads if for all
  uint32_t x;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %1, 0;\n\t"
      "bar.red.and.pred q, 2, %2, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(x)
      : "r"((uint32_t)ok), "n"(kMerge)
      : "memory");
  return x != 0;
}
__device__ __forceinline__ void merge_sync() { asm volatile("bar.sync 1, %0;" ::"n"(kMerge) : "memory"); }

// 16-byte piece c of row r of an e4m3 page in shared memory (128- or 64-byte
// rows, swizzled by TMA over their own length).
template <int D>
__device__ __forceinline__ const uint8_t* piece_at(const uint8_t* page, int r, int c) {
  return page + r * D + ((c ^ (D == 128 ? r & 7 : (r >> 1) & 3)) << 4);
}

// The D / 4 codes of quarter t of row r: the contraction's order is theirs, so
// that they are an MMA's operand as they come.  The 8 lanes of one pass over
// the banks read two neighbouring rows: quarter t of a row of 128 is its
// pieces 2 t and 2 t + 1, so that the two rows' pieces never share banks.
template <int D>
__device__ __forceinline__ void row_codes(const uint8_t* page, int r, int t, uint32_t (&w)[D / 16]) {
#pragma unroll
  for (int i = 0; i < D / 64; ++i) {
    const uint4 x = *reinterpret_cast<const uint4*>(piece_at<D>(page, r, (D / 64) * t + i));
    w[4 * i] = x.x; w[4 * i + 1] = x.y; w[4 * i + 2] = x.z; w[4 * i + 3] = x.w;
  }
}
__device__ __forceinline__ void mma16832_e4m3(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t pack_half(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}
// Two fp16 numbers as codes and those of 32 times what they leave.
__device__ __forceinline__ void split_pair(uint32_t x, uint32_t& c, uint32_t& r) {
  asm("{\n\t.reg .b16 h, l;\n\t.reg .b32 y;\n\t"
      "cvt.rn.satfinite.e4m3x2.f16x2 h, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 y, h;\n\t"
      "sub.rn.f16x2 y, %2, y;\n\t"
      "mul.rn.f16x2 y, y, %3;\n\t"
      "cvt.rn.satfinite.e4m3x2.f16x2 l, y;\n\t"
      "cvt.u32.u16 %0, h;\n\t"
      "cvt.u32.u16 %1, l;\n\t}"
      : "=r"(c), "=r"(r)
      : "r"(x), "r"(0x50005000u));  // 32 in fp16
}
// A query as the sum of two e4m3 rows: with s the power of two that brings the
// head's largest magnitude to 128 .. 256, x = q s is hi + lo / 32.  Of a bf16
// number, whose 8 bits are twice e4m3's, hi takes four and leaves at most 4 and
// a sign, so that the sum is exact; for |x| < 2^-7, where e4m3's steps no longer
// shrink, it is off by up to 2^-15: `off` says whether there are such elements.
// Returns 1 / s, or NaN for a query that is not finite.
template <int D>
__device__ __forceinline__ float split_query(const uint16_t* row, bool there, uint32_t (&hi)[D / 16],
                                             uint32_t (&lo)[D / 16], bool& off) {
  uint4 w[D / 32];
#pragma unroll
  for (int i = 0; i < D / 32; ++i)
    w[i] = there ? reinterpret_cast<const uint4*>(row)[i] : make_uint4(0u, 0u, 0u, 0u);
  uint32_t pair = 0;             // largest magnitudes of the even and the odd elements
  uint32_t least = 0x7fff7fffu;  // and their smallest but zero, less 1 + 2^15 (zeros: 2^15 - 1)
#pragma unroll
  for (int i = 0; i < D / 32; ++i) {
    const uint32_t u[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t a = u[k] & 0x7fff7fffu;
      pair = __vmaxu2(pair, a);
      least = __vmins2(least, a + 0x7fff7fffu);
    }
  }
  uint32_t top = max(pair & 0xffffu, pair >> 16);
  top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
  top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
  const uint32_t e = max(top >> 7, 14u);  // biased; 2^(134 - 127 - e) stays a normal number
  const float s = __uint_as_float((134u + 127u - e) << 23);
  off = min((int)(int16_t)(least & 0xffffu), (int)(int16_t)(least >> 16)) + 32769 < ((int)e - 14) << 7;
#pragma unroll
  for (int i = 0; i < D / 32; ++i) {
    const uint32_t u[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      uint32_t c[2], r[2];
#pragma unroll
      for (int n = 0; n < 2; ++n) {  // in fp16, of which x and the rest are numbers (down to 2^-24)
        const uint32_t v = u[2 * k + n];
        const uint32_t x = pack_half(__uint_as_float(v << 16) * s, __uint_as_float(v & 0xffff0000u) * s);
        split_pair(x, c[n], r[n]);
      }
      hi[2 * i + k] = c[0] | c[1] << 16;
      lo[2 * i + k] = r[0] | r[1] << 16;
    }
  }
  return e == 255u ? NAN : __uint_as_float((e + 127u - 134u) << 23);
}

// What split_query() leaves out of a thread's elements, as a sum of magnitudes.
template <int D>
__device__ __forceinline__ float left_out(const uint16_t* row, float by) {
  const float s = __uint_as_float((254u << 23) - __float_as_uint(by));  // by is a power of two
  float sum = 0.0f;
#pragma unroll 4
  for (int i = 0; i < D / 4; i += 2) {
    const uint32_t v = *reinterpret_cast<const uint32_t*>(row + i);
    const float x = __uint_as_float(v << 16) * s, z = __uint_as_float(v & 0xffff0000u) * s;
    uint32_t c, r, ch, rh;
    split_pair(pack_half(x, z), c, r);
    codes_to_half(c | r << 16, ch, rh);
    const float2 hi = __half22float2(*reinterpret_cast<const __half2*>(&ch));
    const float2 lo = __half22float2(*reinterpret_cast<const __half2*>(&rh));
    sum += fabsf(x - hi.x - lo.x * (1.0f / 32)) + fabsf(z - hi.y - lo.y * (1.0f / 32));
  }
  return sum;
}

// Scores times s of a tile of 16 keys, in bf16: of queries that leave too much
// out.  by: the heads' 1 / s.  d is the MMA's result, for columns past the heads
// zero.
template <int D, int G>
__device__ __forceinline__ void whole_scores(const uint8_t* keys, const uint16_t* row, const float* by, float (&d)[4]) {
  const int grp = threadIdx.x >> 2 & 7, tig = threadIdx.x & 3;
  const bool there = grp < G;
  row += (there ? grp : 0) * D + (D / 4) * tig;
  keys += grp * D + (D / 4) * tig;
  const uint32_t s2 = (254u - (__float_as_uint(by[grp]) >> 23)) * 0x800080u;
  d[0] = d[1] = d[2] = d[3] = 0.0f;
#pragma unroll 1
  for (int i = 0; i < D / 16; ++i) {
    const uint2 w = *reinterpret_cast<const uint2*>(row + 4 * i);
    const uint32_t x0 = *reinterpret_cast<const uint32_t*>(keys + 4 * i);
    const uint32_t x1 = *reinterpret_cast<const uint32_t*>(keys + 8 * D + 4 * i);
    const uint4 p = code_pairs(make_uint2(x0, x1), row_factor(127));
    const uint32_t a[4] = {p.x, p.z, p.y, p.w};
    mma16816(d, a, there ? mul_bf16x2(w.x, s2) : 0u, there ? mul_bf16x2(w.y, s2) : 0u);
  }
}
// The same of two tiles, as the lanes go on with them where both parts are
// columns of one MMA.  (A call, whose registers are not the caller's: in the
// loop itself 64 sequences of up to 8192 tokens take 143.8 us for 140.7; of eight
// heads it is the other way round, 155.6 for 163.6.)
template <int D, int G>
__device__ __noinline__ void whole_folded(const uint8_t* keys, const uint16_t* row, const float* by, float* x) {
  const int lane = threadIdx.x & 31;
  const bool low = (lane & 3) < 2;
#pragma unroll 1
  for (int u = 0; u < 2; ++u) {
    float d[4];
    whole_scores<D, G>(keys + 16 * u * D, row, by, d);
    const float r0 = __shfl_xor_sync(0xffffffffu, d[2], 2), r1 = __shfl_xor_sync(0xffffffffu, d[3], 2);
    x[64 * u + lane] = low ? d[0] : r0;
    x[64 * u + 32 + lane] = low ? d[1] : r1;
  }
}

// The D / 8 codes of part g of row r.
template <int D>
__device__ __forceinline__ void part_codes(const uint8_t* page, int r, int g, uint32_t (&w)[D / 32]) {
  if constexpr (D == 128) {
    const uint4 x = *reinterpret_cast<const uint4*>(piece_at<D>(page, r, g));
    w[0] = x.x; w[1] = x.y; w[2] = x.z; w[3] = x.w;
  } else {
    const uint2 x = *reinterpret_cast<const uint2*>(piece_at<D>(page, r, g >> 1) + 8 * (g & 1));
    w[0] = x.x; w[1] = x.y;
  }
}
// Two such parts in pairs: dims 2 j and 2 j + 1 of both as a[j][at] and a[j][at
// + 1], in bf16 times 2^-120 (a byte of each and their signs' copies by one prmt).
template <int kSelector>
__device__ __forceinline__ uint32_t code_pair(uint32_t x, uint32_t y) {
  uint32_t w;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(w) : "r"(x), "r"(y), "n"(kSelector));
  return codes_to_bf16(w);
}
template <int D>
__device__ __forceinline__ void pair_codes(const uint32_t (&x)[D / 32], const uint32_t (&y)[D / 32],
                                           uint32_t (&a)[D / 16][4], int at) {
#pragma unroll
  for (int j = 0; j < D / 32; ++j) {
    a[2 * j][at] = code_pair<0xc480>(x[j], y[j]);
    a[2 * j][at + 1] = code_pair<0xd591>(x[j], y[j]);
    a[2 * j + 1][at] = code_pair<0xe6a2>(x[j], y[j]);
    a[2 * j + 1][at + 1] = code_pair<0xf7b3>(x[j], y[j]);
  }
}
// Keys that the query of sequence b sees, and the pages that hold them; a
// query that sees none has one page, dead.
struct Span {
  int64_t t, lo;
  int32_t j0, np;
  bool dead, bad;
};
__device__ __forceinline__ Span seq_span(const MaskArgs& m, const int32_t* seq_lens, int64_t b, int64_t N) {
  Span s;
  const int64_t len = seq_lens[b];
  s.bad = len < 1 || len > N;
  s.t = len - 1;
  int64_t hi = 0;
  s.lo = 0;
  if (!s.bad) key_span(m, b, 1, 0, s.t, len, &s.lo, &hi);
  s.dead = s.bad || s.lo > s.t;
  s.j0 = s.dead ? 0 : (int32_t)(s.lo / kPage);
  s.np = s.dead ? 1 : (int32_t)(s.t / kPage) - s.j0 + 1;
  return s;
}

template <int D, int G, bool Q8>
__global__ void __launch_bounds__(Shape<D, G, Q8>::kThreads, 1)
    paged_decode_kernel(Prob pr, MaskArgs mk, const __grid_constant__ CUtensorMap kmap,
                        const __grid_constant__ CUtensorMap vmap, const uint8_t* __restrict__ kcodes,
                        const uint8_t* __restrict__ kscales,
                        const uint8_t* __restrict__ vscales, const uint16_t* __restrict__ q,
                        const int32_t* __restrict__ table, int64_t nb, int64_t num_pages,
                        const int32_t* __restrict__ seq_lens, const int32_t* __restrict__ idx, Parts parts,
                        int32_t min_run, int32_t* __restrict__ status, uint16_t* __restrict__ out) {
  using S = Shape<D, G, Q8>;
  constexpr int kStages = S::kStages, kGroups = S::kGroups, kWarps = S::kWarps, kCons = S::kCons, kBatch = S::kBatch;
  constexpr uint32_t kTile = S::kTile;
  constexpr int kHalf = kPage * 128;  // bytes of a tile's 64-column half
  extern __shared__ unsigned char smem_raw[];
  Smem<D, G, Q8>& sm = *reinterpret_cast<Smem<D, G, Q8>*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile int32_t* abort = &sm.abort;
  auto give_up = [&] {  // a wait ran out
    *abort = 1;
    if (lane == 0) set_status(status, PISA_DEV_TIMEOUT);
  };
  if (threadIdx.x == kCons) {
    ptx::prefetch_map(&kmap);
    ptx::prefetch_map(&vmap);
  }
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      ptx::mbar_init(ptx::smem_u32(&sm.full[s]), 1 + (Q8 ? kScaleLanes : 0));
      ptx::mbar_init(ptx::smem_u32(&sm.empty[s]), S::kGroupWarps);
    }
    ptx::mbar_init(ptx::smem_u32(&sm.mfull), kWarps);
    ptx::mbar_init(ptx::smem_u32(&sm.mempty), kMerge / 32);
    sm.abort = 0;
    sm.zero = 0;
    ptx::fence_mbar_init();
    ptx::fence_proxy_async_smem();
  }
  // The cut: T units in runs of `run`, this CTA's is [u0, u1).  Every warp
  // derives it for itself.
  const int W = pr.K + 3;
  int64_t T;
  if (idx) {
    T = pr.B * pr.Hkv * W;
  } else {
    int64_t n = 0;
    for (int64_t b = lane; b < pr.B; b += 32) n += seq_span(mk, seq_lens, b, pr.N).np;
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
    T = n * pr.Hkv;
  }
  const int64_t run = max((int64_t)min_run, ceil_div64(T, gridDim.x));
  const int64_t u0 = blockIdx.x * run, u1 = min(T, u0 + run);
  __syncthreads();
  pdl_wait();  // from here on the status word and the counters are clear
  if (u0 >= T) return;

  if (warp == kWarps) {
    // ------------------------------------------------------------ producer
    // the sequence, head and page of u0
    int64_t b = 0, i0 = 0;
    if (idx) {
      b = u0 / (pr.Hkv * W);
      i0 = b * pr.Hkv * W;
    } else {
      for (int64_t c = 0; c < pr.B; c += 32) {
        const int64_t x0 = c + lane < pr.B ? (int64_t)seq_span(mk, seq_lens, c + lane, pr.N).np * pr.Hkv : 0;
        int64_t x = x0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
          if (lane >= o) x += y;
        }
        const unsigned over = __ballot_sync(0xffffffffu, i0 + x > u0);
        if (over) {
          const int at = __ffs(over) - 1;
          i0 += __shfl_sync(0xffffffffu, x - x0, at);
          b = c + at;
          break;
        }
        i0 += __shfl_sync(0xffffffffu, x, 31);
      }
    }
    Span sp = seq_span(mk, seq_lens, b, pr.N);
    int32_t np = idx ? W : sp.np;
    int32_t h = (int32_t)((u0 - i0) / np);
    i0 += (int64_t)h * np;  // first unit of the item
    // (64-bit divisions take a hundred cycles and more)
    auto over_run = [&](int64_t x) { return T < (int64_t)1 << 32 ? (int64_t)((uint32_t)x / (uint32_t)run) : x / run; };
    int it = 0, st = 0, ph = 0;  // stages filled; the next one and its phase
    bool ok = true;
    // The next n stages (at most kBatch), one a lane from lane `first` on, whose
    // meta and page it holds (page < 0: none to load): a page's waits, barriers
    // and addresses take some 600 cycles of a warp, whether for one lane or two.
    auto emit = [&](int n, int first, const Meta& meta, int32_t page, int32_t head, int64_t seq) -> bool {
      const int k = lane - first;
      const bool mine = k >= 0 && k < n;
      const bool wrap = st + k >= kStages;
      const int s = mine ? (wrap ? st + k - kStages : st + k) : 0;
      bool got = true;
      if (mine && it + k >= kStages)
        got = ptx::mbar_wait_fast(ptx::smem_u32(&sm.empty[s]), wrap ? ph : ph ^ 1, abort);
      if (!__all_sync(0xffffffffu, got)) return false;
      const int32_t y = page >= 0 ? (int32_t)(((int64_t)page * pr.Hkv + head) * kPage) : -1;  // its first row
      if (mine) {
        sm.meta[s] = meta;
        const uint32_t full = ptx::smem_u32(&sm.full[s]);
        const uint32_t bytes = (page >= 0 ? 2 * kTile : 0u) + (meta.first ? (uint32_t)(G * D * 2) : 0u);
        ptx::mbar_arrive_expect_tx(full, bytes);
        if (page >= 0) {
          if constexpr (Q8) {
            ptx::tma_load_2d(ptx::smem_u32(sm.kv[s][0]), &kmap, 0, y, full);
            ptx::tma_load_2d(ptx::smem_u32(sm.kv[s][1]), &vmap, 0, y, full);
          } else {
            ptx::tma_load_3d(ptx::smem_u32(sm.kv[s][0]), &kmap, 0, y, 0, full);
            ptx::tma_load_3d(ptx::smem_u32(sm.kv[s][1]), &vmap, 0, y, 0, full);
          }
        }
        if (meta.first)
          ptx::bulk_g2s(ptx::smem_u32(sm.q[s]), q + (seq * pr.Hq + head * G) * D, G * D * 2, full);
      }
      if constexpr (Q8) {  // the scales, 16 bytes a lane, all in one go
        const int r = lane / kScaleLanes, piece = lane % kScaleLanes;
        const int ys = __shfl_sync(0xffffffffu, y, first + (r < n ? r : 0));
        const int ss = __shfl_sync(0xffffffffu, s, first + (r < n ? r : 0));
        if (r < n) {
          if (ys >= 0)
            ptx::cp_async_16(ptx::smem_u32(&sm.scale[ss][piece / 4][16 * (piece % 4)]),
                             (piece < 4 ? kscales : vscales) + ys + 16 * (piece % 4));
          ptx::cp_async_arrive_noinc(ptx::smem_u32(&sm.full[ss]));
        }
      }
      __syncwarp();
      it += n;
      if ((st += n) >= kStages) {
        st -= kStages;
        ph ^= 1;
      }
      return true;
    };
    for (int64_t u = u0; u < u1 && ok;) {
      if (lane == 0 && sp.bad) set_status(status, PISA_DEV_BAD_SEQ_LEN);
      const int32_t s0 = (int32_t)(u - i0), s1 = (int32_t)min((int64_t)np, u1 - i0);
      Meta meta;
      meta.item = (int32_t)(b * pr.Hkv + h);
      meta.first = 1;
      meta.last = 0;
      meta.rel = 0;
      meta.klo = kPage;
      meta.khi = -1;
      const int64_t c0 = over_run(i0), c1 = over_run(i0 + np - 1);
      meta.cfirst = (int32_t)c0;
      meta.parts = (int32_t)(c1 - c0 + 1);
      meta.slot0 = (int32_t)(2 * c0 + (c0 * run < i0 ? 1 : 0));
      meta.slot = blockIdx.x == c0 ? meta.slot0 : 2 * (int32_t)blockIdx.x;
      const int32_t* trow = table + b * nb;
      int32_t count = 0;  // stages of this part so far
      if (!sp.dead) {
        // the entries of this part, 32 at a time: lane l looks after entry s + l
        int32_t r0 = -1, r1 = -1;
        if (idx) {
          const int32_t* row = idx + (b * pr.Hkv + h) * W;
          if (lane < W) r0 = row[lane];
          if (lane + 32 < W) r1 = row[lane + 32];
        }
        const int32_t qb = (int32_t)(sp.t / kPage);
        int32_t left = 0;  // entries of the part that hold a page, not yet emitted; the last ones are the groups' last
        uint64_t keep = 0;
        if (idx) {
          const bool k0 = r0 >= 0 && r0 <= qb, k1 = r1 >= 0 && r1 <= qb;
          const unsigned below = (1u << lane) - 1u;
          const unsigned m0 = __match_any_sync(0xffffffffu, k0 ? r0 : -1 - lane);  // others match nothing
          const unsigned m1 = __match_any_sync(0xffffffffu, k1 ? r1 : -1 - lane);
          bool dup1 = (m1 & below) != 0u;
          for (int x = 0; x < 32 && W > 32; ++x) {
            const int32_t o = __shfl_sync(0xffffffffu, k0 ? r0 : -1, x);
            dup1 |= k1 && o == r1;
          }
          const unsigned b0 = __ballot_sync(0xffffffffu, k0 && (m0 & below) == 0u);
          const unsigned b1 = __ballot_sync(0xffffffffu, k1 && !dup1);
          keep = ((uint64_t)b1 << 32 | b0) >> s0 << s0;  // this part's entries
          if (s1 < 64) keep &= ((uint64_t)1 << s1) - 1;
          left = __popcll(keep);
        } else {
          left = s1 - s0;
        }
        for (int32_t s = s0 & ~31; s < s1 && ok; s += 32) {
          // lane l: block and page of entry s + l
          int32_t blk = idx ? (s == 0 ? r0 : r1) : sp.j0 + s + lane;
          bool mine = idx ? ((keep >> (s + lane)) & 1) != 0 : s + lane >= s0 && s + lane < s1;
          int32_t page = -1;
          if (mine) {
            page = trow[blk];
            if (page < 0 || page >= num_pages) {
              page = -1;
              set_status(status, PISA_DEV_BAD_INDEX);
            }
          }
          // lane k takes over the k-th of them
          const unsigned todo = __ballot_sync(0xffffffffu, mine);
          const int cnt = __popc(todo), from = __fns(todo, 0, lane + 1) & 31;
          blk = __shfl_sync(0xffffffffu, blk, from);
          page = __shfl_sync(0xffffffffu, page, from);
          const int64_t key0 = (int64_t)blk * kPage;
          meta.rel = (int32_t)(key0 - sp.t);
          meta.klo = page < 0 ? kPage : (int16_t)max((int64_t)0, min((int64_t)kPage, sp.lo - key0));
          meta.khi = (int16_t)min((int64_t)(kPage - 1), sp.t - key0);
          meta.last = left - lane <= kGroups;
          meta.first = count + lane < kGroups;
          for (int k = 0; k < cnt && ok; k += kBatch) ok = emit(min(kBatch, cnt - k), k, meta, page, h, b);
          left -= cnt;
          count += cnt;
        }
      }
      // each group has a stage of every part, if an empty one
      if (count < kGroups) {
        meta.klo = kPage;
        meta.first = meta.last = 1;
        for (; count < kGroups && ok; count += kBatch) ok = emit(min(kBatch, kGroups - count), 0, meta, -1, h, b);
      }
      u = i0 + s1;
      if (s1 == np) {
        i0 += np;
        if (++h == pr.Hkv) {
          h = 0;
          if (++b < pr.B) {
            sp = seq_span(mk, seq_lens, b, pr.N);
            if (!idx) np = sp.np;
          }
        }
      }
    }
    // a stage without an item ends a group
    if (ok) {
      Meta meta;
      meta.item = -1;
      meta.first = 0;
      for (int k = 0; k < kGroups && ok; k += kBatch) ok = emit(min(kBatch, kGroups - k), 0, meta, -1, 0, 0);
    }
    // every copy lands before the CTA ends
    if (lane == 0)
      for (int k = max(0, it - kStages); k < it; ++k)
        ptx::mbar_wait_fast(ptx::smem_u32(&sm.full[k % kStages]), (k / kStages) & 1, &sm.zero);
    if (!ok) give_up();
    return;
  }

  if (warp > kWarps) {
    // ------------------------------------------------- merging a part's warps
    const int mt = threadIdx.x - (kCons + 32);
    for (int n = 0;; ++n) {
      const bool ok = ptx::mbar_wait_fast(ptx::smem_u32(&sm.mfull), n & 1, abort);
      // all of the merging warps go on, or none
      if (!merge_all(ok)) {
        give_up();
        break;
      }
      const Meta part = sm.part;
      if (part.item < 0) break;
      const int64_t orow = (int64_t)part.item * G * D;  // an item's G rows of out are adjacent
      float* po = parts.o + (int64_t)part.slot * G * D;
      for (int e = mt; e < G * D / 2; e += kMerge) {
        const int g = e / (D / 2), c = 2 * (e % (D / 2));
        const float* at = sm.o[0] + o_at<D, Q8>(g, c);
        float a = 0.0f, z = 0.0f, L = 0.0f, M = -INFINITY;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) M = fmaxf(M, sm.m[w][g]);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          // without a maximum a warp saw no key (or nothing but NaN scores)
          const float f = sm.m[w][g] == -INFINITY ? 1.0f : ptx::ex2(sm.m[w][g] - M);
          const float2 x = *reinterpret_cast<const float2*>(at + w * (G * D));
          a = fmaf(x.x, f, a);
          z = fmaf(x.y, f, z);
          L = fmaf(sm.l[w][g], f, L);
        }
        if (part.parts == 1) {
          const float inv = L == 0.0f ? 0.0f : 1.0f / L;
          *reinterpret_cast<uint32_t*>(out + orow + g * D + c) = pack_bf16(a * inv, z * inv);
        } else {
          *reinterpret_cast<float2*>(po + g * D + c) = make_float2(a, z);
          if (c == 0) *reinterpret_cast<float2*>(parts.ml + ((int64_t)part.slot * G + g) * 2) = make_float2(M, L);
        }
      }
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(&sm.mempty));
      if (part.parts == 1) continue;
      __threadfence();
      merge_sync();
      if (mt == 0) sm.last_part = atomicAdd(parts.counter + part.item, 1) == part.parts - 1;
      merge_sync();
      if (!sm.last_part) continue;
      __threadfence();
      constexpr int kCols = Join<D, G>::kCols, kLanes = Join<D, G>::kLanes, kStep = Join<D, G>::kStep;
      const int pl = kLanes > 1 ? mt / kCols : 0;
      static_assert(kLanes == 1 || kCols * kLanes == kMerge, "every merging thread has a column");
      for (int e = kLanes > 1 ? mt % kCols : mt; e < kCols; e += kStep) {
        const int g = e / (D / 8), c = 8 * (e % (D / 8));
        float M = -INFINITY, L = 0.0f, acc[8] = {};
        constexpr int kBatch = 8;  // parts in flight
        for (int p0 = pl; p0 < part.parts; p0 += kBatch * kLanes) {
          float2 ml[kBatch];
          float4 o[kBatch][2];
#pragma unroll
          for (int k = 0; k < kBatch; ++k) {
            const int p = p0 + k * kLanes;
            const int64_t slot = p == 0 ? part.slot0 : 2 * (int64_t)(part.cfirst + p);
            ml[k] = make_float2(-INFINITY, 0.0f);
            o[k][0] = o[k][1] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (p < part.parts) {
              const float4* po = reinterpret_cast<const float4*>(parts.o + slot * G * D + g * D + c);
              ml[k] = __ldcg(reinterpret_cast<const float2*>(parts.ml + (slot * G + g) * 2));
              o[k][0] = __ldcg(po);
              o[k][1] = __ldcg(po + 1);
            }
          }
          float bm = M;
#pragma unroll
          for (int k = 0; k < kBatch; ++k) bm = fmaxf(bm, ml[k].x);
          if (bm > M) {
            const float f = M == -INFINITY ? 1.0f : ptx::ex2(M - bm);
            L *= f;
#pragma unroll
            for (int d = 0; d < 8; ++d) acc[d] *= f;
            M = bm;
          }
#pragma unroll
          for (int k = 0; k < kBatch; ++k) {
            const float f = ml[k].x == -INFINITY ? 1.0f : ptx::ex2(ml[k].x - M);
            L = fmaf(ml[k].y, f, L);
            const float ov[8] = {o[k][0].x, o[k][0].y, o[k][0].z, o[k][0].w,
                                 o[k][1].x, o[k][1].y, o[k][1].z, o[k][1].w};
#pragma unroll
            for (int d = 0; d < 8; ++d) acc[d] = fmaf(ov[d], f, acc[d]);
          }
        }
        if (kLanes > 1) {  // (one round of the loop, for all threads)
          sm.jm[mt] = M;
          sm.jl[mt] = L;
#pragma unroll
          for (int d = 0; d < 8; ++d) sm.jo[mt][d] = acc[d];
          merge_sync();
          if (pl == 0) {
#pragma unroll
            for (int k = 1; k < kLanes; ++k) {
              const float m2 = sm.jm[e + k * kCols], top = fmaxf(M, m2);
              const float f = M == -INFINITY ? 1.0f : ptx::ex2(M - top);
              const float f2 = m2 == -INFINITY ? 1.0f : ptx::ex2(m2 - top);
              L = L * f + sm.jl[e + k * kCols] * f2;
#pragma unroll
              for (int d = 0; d < 8; ++d) acc[d] = acc[d] * f + sm.jo[e + k * kCols][d] * f2;
              M = top;
            }
          }
          merge_sync();
        }
        if (pl == 0) {
          const float inv = L == 0.0f ? 0.0f : 1.0f / L;
          *reinterpret_cast<uint4*>(out + orow + g * D + c) =
              make_uint4(pack_bf16(acc[0] * inv, acc[1] * inv), pack_bf16(acc[2] * inv, acc[3] * inv),
                         pack_bf16(acc[4] * inv, acc[5] * inv), pack_bf16(acc[6] * inv, acc[7] * inv));
        }
      }
    }
    return;
  }

  // ------------------------------------------------------------- consumers
  const int grp = lane >> 2, tig = lane & 3;
  const int r16 = S::kKeys * (warp % S::kGroupWarps);  // this warp's keys of a page
  // ldmatrix rows: lane l addresses row l % 8 of matrix l / 8
  const int krow = r16 + (lane & 7) + ((lane >> 3) & 1) * 8, kch = lane >> 4;
  const int vrow = r16 + (lane & 7) + (lane >> 4) * 8, vch = (lane >> 3) & 1;
  // FOLD (up to four heads): of an MMA's eight columns the heads' upper parts are
  // the first four and their lower ones the others, so that one takes both.
  // The lanes of the first four (tig < 2) then go on with the keys grp of a tile
  // and those of the others with the keys grp + 8, each with heads hd and hd +
  // 1; as columns of P they hold those keys alone, with an m, l and o of
  // their own.
  constexpr bool FOLD = Q8 && G <= 4;
  constexpr int KL = FOLD ? 1 : 2;  // keys of a tile that a lane goes on with
  const bool low = !FOLD || tig < 2;
  const int hd = FOLD ? 2 * (tig & 1) : 2 * tig, kofs = low ? 0 : 8;
  // the query's fragments; Q8: its upper part and its lower one, each head's
  // 1 / s, and whether the part has seen rows over 448 2^kNear
  uint32_t bq[Q8 ? D / 16 : D / 8], bl[Q8 && !FOLD ? D / 16 : 1];
  float hf0 = 1.0f, hf1 = 1.0f;
  bool far = false;
  int most_scale = 255;  // of keys for which the two parts do
  float oacc[D / 16][4];
  float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.0f, l1 = 0.0f;  // heads hd, hd + 1
  float sl0 = 0.0f, sl1 = 0.0f;
  // a group takes every kGroups-th stage
  int st = warp / S::kGroupWarps - kGroups, ph = 0, merges = 0;
  auto wait_merged = [&] {  // the merge buffer is free
    const bool ok = merges == 0 || ptx::mbar_wait_fast(ptx::smem_u32(&sm.mempty), (merges - 1) & 1, abort);
    if (!__all_sync(0xffffffffu, ok)) {
      give_up();
      return false;
    }
    return true;
  };
  for (;;) {
    if ((st += kGroups) >= kStages) {
      st -= kStages;
      ph ^= 1;
    }
    const bool okw = ptx::mbar_wait_fast(ptx::smem_u32(&sm.full[st]), ph, abort);
    if (!__all_sync(0xffffffffu, okw)) {
      give_up();
      break;
    }
    const Meta meta = sm.meta[st];
    if (meta.item < 0) break;
    if (meta.first) {
      if constexpr (Q8) {
        const int head = FOLD ? grp & 3 : grp;
        const uint16_t* row = sm.q[st] + (head < G ? head : 0) * D + (D / 4) * tig;
        float f;
        bool off;
        if constexpr (FOLD) {
          uint32_t rest[D / 16];
          f = split_query<D>(row, head < G, bq, rest, off);
#pragma unroll
          for (int k = 0; k < D / 16; ++k) bq[k] = grp < 4 ? bq[k] : rest[k];
        } else {
          f = split_query<D>(row, head < G, bq, bl, off);
        }
        hf0 = __shfl_sync(0xffffffffu, f, 4 * hd);
        hf1 = __shfl_sync(0xffffffffu, f, 4 * hd + 4);
        far = false;
        most_scale = 255;
        if (__any_sync(0xffffffffu, off)) {
          float left = grp < G ? left_out<D>(row, f) : 0.0f;
          left += __shfl_xor_sync(0xffffffffu, left, 1);
          left += __shfl_xor_sync(0xffffffffu, left, 2);
          left *= f;
#pragma unroll
          for (int o = 4; o <= 16; o <<= 1) left = fmaxf(left, __shfl_xor_sync(0xffffffffu, left, o));
          // it adds up to 448 times a key's power times `left` in a score: 2^-11 (log2
          // units) and less are let be
          const uint32_t bits = __float_as_uint(left * 448.0f * fabsf(pr.scale2));
          most_scale = bits == 0u ? 255 : 127 - 11 - ((int)(bits >> 23) - 126);
          if (tig == 0) sm.by[warp][grp] = f;
          __syncwarp();
        }
      } else {
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          const uint32_t* qr = reinterpret_cast<const uint32_t*>(sm.q[st] + (grp < G ? grp : 0) * D + 16 * ks);
          bq[2 * ks] = grp < G ? qr[tig] : 0u;
          bq[2 * ks + 1] = grp < G ? qr[tig + 4] : 0u;
        }
      }
#pragma unroll
      for (int mt = 0; mt < D / 16; ++mt) oacc[mt][0] = oacc[mt][1] = oacc[mt][2] = oacc[mt][3] = 0.0f;
      m0 = m1 = -INFINITY;
      l0 = l1 = 0.0f;
      if (mk.slopes) {
        const float* sl = mk.slopes + (int64_t)(meta.item % pr.Hkv) * G;
        sl0 = hd < G ? sl[hd] * kLog2e : 0.0f;
        sl1 = hd + 1 < G ? sl[hd + 1] * kLog2e : 0.0f;
      }
    }
    const bool seen_any = meta.klo <= meta.khi && r16 <= meta.khi && r16 + S::kKeys - 1 >= meta.klo;
    // Q8: 16 keys and their values are 32 registers (of d = 128), so that the
    // stage is free again before they are worked on.
    constexpr int T = S::kKeys / 16;  // tiles of 16 keys
    uint32_t kc[Q8 ? T : 1][2][D / 16], vc[Q8 ? T : 1][4][D / 32];
    int ksc[T][KL], vsc[T][KL];  // and the scales
    bool large_key = false;      // of one for which the query's parts do not do
    if constexpr (Q8) {
      if (seen_any) {
#pragma unroll
        for (int u = 0; u < T; ++u) {
          const int r = r16 + 16 * u + grp, c = r16 + 16 * u + 2 * tig;
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            row_codes<D>(sm.kv[st][0], r + 8 * j, tig, kc[u][j]);
            part_codes<D>(sm.kv[st][1], c + 8 * j, grp, vc[u][2 * j]);
            part_codes<D>(sm.kv[st][1], c + 8 * j + 1, grp, vc[u][2 * j + 1]);
          }
#pragma unroll
          for (int j = 0; j < KL; ++j) {
            ksc[u][j] = sm.scale[st][0][r + kofs + 8 * j];
            large_key |= ksc[u][j] > most_scale;
            vsc[u][j] = sm.scale[st][1][r + kofs + 8 * j];
          }
        }
      }
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(&sm.empty[st]));
    }
    if (seen_any) {
      if constexpr (Q8) {
        // keys grp + kofs (and 8 further) of each tile, heads hd and hd + 1
        float x[T][2 * KL];
#pragma unroll
        for (int u = 0; u < T; ++u) {
          const uint32_t (&k0)[D / 16] = kc[u][0], (&k1)[D / 16] = kc[u][1];
          float d[4] = {}, e[4] = {};  // of the query's upper part and its lower one; FOLD: two chains of both
#pragma unroll
          for (int k = 0; k < D / 16; k += 2) {
            if constexpr (FOLD) {
              mma16832_e4m3(k & 2 ? e : d, k0[k], k1[k], k0[k + 1], k1[k + 1], bq[k], bq[k + 1]);
            } else {
              mma16832_e4m3(d, k0[k], k1[k], k0[k + 1], k1[k + 1], bq[k], bq[k + 1]);
              mma16832_e4m3(e, k0[k], k1[k], k0[k + 1], k1[k + 1], bl[k], bl[k + 1]);
            }
          }
          if constexpr (FOLD) {
#pragma unroll
            for (int j = 0; j < 4; ++j) d[j] += e[j];
            // each half of the lanes sends what the other goes on with
            const float r0 = __shfl_xor_sync(0xffffffffu, low ? d[2] : d[0], 2);
            const float r1 = __shfl_xor_sync(0xffffffffu, low ? d[3] : d[1], 2);
            x[u][0] = low ? fmaf(r0, 1.0f / 32, d[0]) : fmaf(d[2], 1.0f / 32, r0);
            x[u][1] = low ? fmaf(r1, 1.0f / 32, d[1]) : fmaf(d[3], 1.0f / 32, r1);
          } else {
#pragma unroll
            for (int j = 0; j < 2 * KL; ++j) x[u][j] = fmaf(e[j], 1.0f / 32, d[j]);
          }
#pragma unroll
          for (int j = 0; j < KL; ++j) {
            // (255 makes an infinity of it, and NaN of the product: such a row's codes are zero)
            const float f = __uint_as_float((uint32_t)ksc[u][j] << 23);
            x[u][2 * j] *= hf0 * f;  // the powers first: one of them may take x out of fp32's range
            x[u][2 * j + 1] *= hf1 * f;
          }
        }
        if (mk.cap2 > 0.0f) {  // cap_score(), the form of large scores where there are some
          bool large = false;
#pragma unroll
          for (int u = 0; u < T; ++u)
#pragma unroll
            for (int j = 0; j < 2 * KL; ++j) large |= !(fabsf(x[u][j] * mk.by) <= mk.lim);
          if (__any_sync(0xffffffffu, large)) {
#pragma unroll
            for (int u = 0; u < T; ++u)
#pragma unroll
              for (int j = 0; j < 2 * KL; ++j) x[u][j] = cap_score(mk, x[u][j]);
          } else {
#pragma unroll
            for (int u = 0; u < T; ++u)
#pragma unroll
              for (int j = 0; j < 2 * KL; ++j) x[u][j] = cap_small(mk, x[u][j]);
          }
        } else {
#pragma unroll
          for (int u = 0; u < T; ++u)
#pragma unroll
            for (int j = 0; j < 2 * KL; ++j) x[u][j] *= pr.scale2;
        }
        const int ka = r16 + grp + kofs;  // this lane's first key
        if (mk.slopes) {
#pragma unroll
          for (int u = 0; u < T; ++u)
#pragma unroll
            for (int j = 0; j < KL; ++j) {
              const float back = (float)(meta.rel + ka + 16 * u + 8 * j);
              x[u][2 * j] = fmaf(sl0, back, x[u][2 * j]);
              x[u][2 * j + 1] = fmaf(sl1, back, x[u][2 * j + 1]);
            }
        }
        const bool part = r16 < meta.klo || r16 + S::kKeys - 1 > meta.khi;  // some of the keys are not seen
        if (part) {
#pragma unroll
          for (int u = 0; u < T; ++u)
#pragma unroll
            for (int j = 0; j < KL; ++j) {
              const int k = ka + 16 * u + 8 * j;
              if (k < meta.klo || k > meta.khi) {
                x[u][2 * j] = x[u][2 * j + 1] = -INFINITY;
                vsc[u][j] = 0;  // its power has no say
              }
            }
        }
        float c0 = -INFINITY, c1 = -INFINITY;
        int top = 0;
#pragma unroll
        for (int u = 0; u < T; ++u)
#pragma unroll
          for (int j = 0; j < KL; ++j) {
            c0 = fmaxf(c0, x[u][2 * j]);
            c1 = fmaxf(c1, x[u][2 * j + 1]);
            top = max(top, vsc[u][j]);
          }
        // The reference follows the maximum when that has grown by 2^8, and rows of
        // any size change P's and O's units: as a rule neither, and one vote says so.
        // A row of NaN (255) is over every power.
        if (__any_sync(0xffffffffu, large_key || c0 > m0 + kSlack || c1 > m1 + kSlack || top > (far ? 254 : kNear))) {
          if (__any_sync(0xffffffffu, large_key)) {  // the scores again, of the codes and the query in bf16
            const int64_t b = meta.item / pr.Hkv, key0 = meta.rel + (int64_t)seq_lens[b] - 1;
            const int64_t row0 = ((int64_t)table[b * nb + key0 / kPage] * pr.Hkv + meta.item % pr.Hkv) * kPage + r16;
            const uint16_t* row = q + (int64_t)meta.item * G * D;
            if constexpr (FOLD) whole_folded<D, G>(kcodes + row0 * D, row, sm.by[warp], sm.more[warp][0][0]);
            c0 = c1 = -INFINITY;
#pragma unroll
            for (int u = 0; u < T; ++u) {
              float d[4];
              if constexpr (FOLD) {
                d[0] = sm.more[warp][u][0][lane];
                d[1] = sm.more[warp][u][1][lane];
              } else {
                whole_scores<D, G>(kcodes + (row0 + 16 * u) * D, row, sm.by[warp], d);
              }
#pragma unroll
              for (int j = 0; j < KL; ++j) {
                const int k = ka + 16 * u + 8 * j;
                const float f = __uint_as_float((uint32_t)kscales[row0 + k - r16] << 23), back = (float)(meta.rel + k);
                const bool hidden = k < meta.klo || k > meta.khi;
                float y0 = d[2 * j] * (hf0 * f), y1 = d[2 * j + 1] * (hf1 * f);
                y0 = mk.cap2 > 0.0f ? cap_score(mk, y0) : y0 * pr.scale2;
                y1 = mk.cap2 > 0.0f ? cap_score(mk, y1) : y1 * pr.scale2;
                if (mk.slopes) {
                  y0 = fmaf(sl0, back, y0);
                  y1 = fmaf(sl1, back, y1);
                }
                x[u][2 * j] = hidden ? -INFINITY : y0;
                x[u][2 * j + 1] = hidden ? -INFINITY : y1;
                c0 = fmaxf(c0, x[u][2 * j]);
                c1 = fmaxf(c1, x[u][2 * j + 1]);
              }
            }
          }
          top = 0;
#pragma unroll
          for (int u = 0; u < T; ++u)
#pragma unroll
            for (int j = 0; j < KL; ++j) {
              if (vsc[u][j] == 255) x[u][2 * j] = x[u][2 * j + 1] = NAN;
              else top = max(top, vsc[u][j]);
            }
          top = __reduce_max_sync(0xffffffffu, top);
#pragma unroll
          for (int o = 4; o <= 16; o <<= 1) {
            c0 = fmaxf(c0, __shfl_xor_sync(0xffffffffu, c0, o));
            c1 = fmaxf(c1, __shfl_xor_sync(0xffffffffu, c1, o));
          }
          const float n0 = fmaxf(m0, c0), n1 = fmaxf(m1, c1);
          float f0 = m0 == -INFINITY ? 0.0f : ptx::ex2(m0 - n0);
          float f1 = m1 == -INFINITY ? 0.0f : ptx::ex2(m1 - n1);
          m0 = n0;
          m1 = n1;
          l0 *= f0;
          l1 *= f1;
          if (!far && top > kNear) {
            far = true;
            f0 *= 1.0f / (1 << (kFarO - kNearO));
            f1 *= 1.0f / (1 << (kFarO - kNearO));
          }
#pragma unroll
          for (int mt = 0; mt < D / 16; ++mt) {
            oacc[mt][0] *= f0; oacc[mt][2] *= f0;
            oacc[mt][1] *= f1; oacc[mt][3] *= f1;
          }
        }
        // a key without weight: its score is -inf (m is, only if all were)
        const float z0 = m0 == -INFINITY ? 0.0f : m0, z1 = m1 == -INFINITY ? 0.0f : m1;
#pragma unroll
        for (int u = 0; u < T; ++u) {
          // The rows' powers go with the weights.  P is rounded to bf16 for the MMA:
          // 2^-9 of each weight.
          uint32_t pk[2] = {0u, 0u};
#pragma unroll
          for (int j = 0; j < KL; ++j) {
            const float p0 = ptx::ex2(x[u][2 * j] - z0), p1 = ptx::ex2(x[u][2 * j + 1] - z1);
            l0 += p0;
            l1 += p1;
            const float f = __uint_as_float((uint32_t)(vsc[u][j] + (far ? 0 : kNearLift)) << 23);
            pk[j] = pack_bf16(p0 * f, p1 * f);
          }
          if constexpr (FOLD) {
            pk[1] = low ? 0u : pk[0];
            pk[0] = low ? pk[0] : 0u;
          }
          const uint32_t b0 = transpose8(pk[0]), b1 = transpose8(pk[1]);
          // The values' rows are the MMA's columns: a thread takes D / 8 codes of
          // its four keys, 2 tig, 2 tig + 1 and 8 further, and pairs the keys
          // byte by byte; the dims D / 8 grp + 2 mt and the next are rows grp and
          // grp + 8 of step mt.
          const int k2 = r16 + 16 * u + 2 * tig;
          uint32_t av[D / 16][4];
          pair_codes<D>(vc[u][0], vc[u][1], av, 0);
          pair_codes<D>(vc[u][2], vc[u][3], av, 2);
          if (far) {
#pragma unroll
            for (int mt = 0; mt < D / 16; ++mt)
#pragma unroll
              for (int j = 0; j < 4; ++j) av[mt][j] = mul_bf16x2(av[mt][j], kFarValues);
          }
          uint32_t va = 0xffffffffu, vz = 0xffffffffu;  // masks of the value pairs
          if (part) {
            auto seen = [&](int k) { return k >= meta.klo && k <= meta.khi; };
            va = (seen(k2) ? 0xffffu : 0u) | (seen(k2 + 1) ? 0xffff0000u : 0u);
            vz = (seen(k2 + 8) ? 0xffffu : 0u) | (seen(k2 + 9) ? 0xffff0000u : 0u);
          }
#pragma unroll
          for (int mt = 0; mt < D / 16; ++mt) {
            if (part) {  // a value that is not seen may be anything
              av[mt][0] &= va; av[mt][1] &= va;
              av[mt][2] &= vz; av[mt][3] &= vz;
            }
            mma16816(oacc[mt], av[mt], b0, b1);
          }
        }
      } else {
        const uint32_t kb = ptx::smem_u32(sm.kv[st][0]), vb = ptx::smem_u32(sm.kv[st][1]);
        float d[4] = {0.0f, 0.0f, 0.0f, 0.0f}, e[4] = {0.0f, 0.0f, 0.0f, 0.0f};  // two chains
        {
          uint32_t a[D / 16][4];
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks) {
            const int ch = 2 * ks + kch;
            ldsm4(kb + (ch >> 3) * kHalf + krow * 128 + (((ch & 7) ^ (krow & 7)) << 4), a[ks]);
          }
#pragma unroll
          for (int ks = 0; ks < D / 16; ks += 2) {
            mma16816(d, a[ks], bq[2 * ks], bq[2 * ks + 1]);
            mma16816(e, a[ks + 1], bq[2 * ks + 2], bq[2 * ks + 3]);
          }
        }
        uint32_t av[D / 16][4];  // the values' fragments, on their way during the softmax
#pragma unroll
        for (int mt = 0; mt < D / 16; ++mt) {
          const int ch = 2 * mt + vch;
          ldsm4_t(vb + (ch >> 3) * kHalf + vrow * 128 + (((ch & 7) ^ (vrow & 7)) << 4), av[mt]);
        }
        // keys grp and grp + 8 of this warp's 16, heads 2 tig and 2 tig + 1
        float x[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          x[j] = d[j] + e[j];
          x[j] = mk.cap2 > 0.0f ? cap_score(mk, x[j]) : x[j] * pr.scale2;
        }
        const int ka = r16 + grp;
        if (mk.slopes) {
          const float ra = (float)(meta.rel + ka), rb = (float)(meta.rel + ka + 8);
          x[0] = fmaf(sl0, ra, x[0]); x[1] = fmaf(sl1, ra, x[1]);
          x[2] = fmaf(sl0, rb, x[2]); x[3] = fmaf(sl1, rb, x[3]);
        }
        const bool part = r16 < meta.klo || r16 + 15 > meta.khi;  // some of the 16 keys are not seen
        uint32_t va = 0xffffffffu, vz = 0xffffffffu;              // masks of the value pairs below
        if (part) {
          if (ka < meta.klo || ka > meta.khi) x[0] = x[1] = -INFINITY;
          if (ka + 8 < meta.klo || ka + 8 > meta.khi) x[2] = x[3] = -INFINITY;
          const int k2 = r16 + 2 * tig;
          auto seen = [&](int k) { return k >= meta.klo && k <= meta.khi; };
          va = (seen(k2) ? 0xffffu : 0u) | (seen(k2 + 1) ? 0xffff0000u : 0u);
          vz = (seen(k2 + 8) ? 0xffffu : 0u) | (seen(k2 + 9) ? 0xffff0000u : 0u);
        }
        float c0 = fmaxf(x[0], x[2]), c1 = fmaxf(x[1], x[3]);
#pragma unroll
        for (int o = 4; o <= 16; o <<= 1) {
          c0 = fmaxf(c0, __shfl_xor_sync(0xffffffffu, c0, o));
          c1 = fmaxf(c1, __shfl_xor_sync(0xffffffffu, c1, o));
        }
        const float n0 = fmaxf(m0, c0), n1 = fmaxf(m1, c1);
        if (__any_sync(0xffffffffu, n0 > m0 || n1 > m1)) {
          const float f0 = m0 == -INFINITY ? 0.0f : ptx::ex2(m0 - n0);
          const float f1 = m1 == -INFINITY ? 0.0f : ptx::ex2(m1 - n1);
          m0 = n0;
          m1 = n1;
          l0 *= f0;
          l1 *= f1;
#pragma unroll
          for (int mt = 0; mt < D / 16; ++mt) {
            oacc[mt][0] *= f0; oacc[mt][2] *= f0;
            oacc[mt][1] *= f1; oacc[mt][3] *= f1;
          }
        }
        // a key without weight: its score is -inf (m is, only if all were)
        const float z0 = m0 == -INFINITY ? 0.0f : m0, z1 = m1 == -INFINITY ? 0.0f : m1;
        const float p0 = ptx::ex2(x[0] - z0), p1 = ptx::ex2(x[1] - z1);
        const float p2 = ptx::ex2(x[2] - z0), p3 = ptx::ex2(x[3] - z1);
        l0 += p0 + p2;
        l1 += p1 + p3;
        // P is rounded to bf16 for the MMA (2^-8 of each weight, the values' own step)
        const uint32_t b0 = transpose8(pack_bf16(p0, p1)), b1 = transpose8(pack_bf16(p2, p3));
#pragma unroll
        for (int mt = 0; mt < D / 16; ++mt) {
          if (part) {  // a value that is not seen may be anything
            av[mt][0] &= va; av[mt][1] &= va;
            av[mt][2] &= vz; av[mt][3] &= vz;
          }
          mma16816(oacc[mt], av[mt], b0, b1);
        }
      }
    }
    if constexpr (!Q8) {
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(&sm.empty[st]));
    }
    if (!meta.last) continue;

    // ------------------ end of a part: hand (m, l, o) to the merging warps
#pragma unroll
    for (int o = 4; o <= 16; o <<= 1) {
      l0 += __shfl_xor_sync(0xffffffffu, l0, o);
      l1 += __shfl_xor_sync(0xffffffffu, l1, o);
    }
    if constexpr (FOLD) {  // both halves of the lanes' keys into one (m, l, o)
      const float o0 = __shfl_xor_sync(0xffffffffu, m0, 2), o1 = __shfl_xor_sync(0xffffffffu, m1, 2);
      const float M0 = fmaxf(m0, o0), M1 = fmaxf(m1, o1);
      // without a maximum a half saw no key (or nothing but NaN scores)
      const float a0 = m0 == -INFINITY ? 1.0f : ptx::ex2(m0 - M0), a1 = m1 == -INFINITY ? 1.0f : ptx::ex2(m1 - M1);
      m0 = M0;
      m1 = M1;
      l0 *= a0;
      l1 *= a1;
      l0 += __shfl_xor_sync(0xffffffffu, l0, 2);
      l1 += __shfl_xor_sync(0xffffffffu, l1, 2);
#pragma unroll
      for (int mt = 0; mt < D / 16; ++mt) {
        oacc[mt][0] *= a0; oacc[mt][1] *= a1; oacc[mt][2] *= a0; oacc[mt][3] *= a1;
#pragma unroll
        for (int j = 0; j < 4; ++j) oacc[mt][j] += __shfl_xor_sync(0xffffffffu, oacc[mt][j], 2);
      }
    }
    if (!wait_merged()) break;
    if (warp == 0 && lane == 0) sm.part = meta;
    if (grp == 0) {
      *reinterpret_cast<float2*>(&sm.m[warp][2 * tig]) = make_float2(m0, m1);
      *reinterpret_cast<float2*>(&sm.l[warp][2 * tig]) = make_float2(l0, l1);
    }
    if constexpr (Q8) {  // O as it is
      const float f = __uint_as_float((uint32_t)(127 + (far ? kFarO : kNearO)) << 23);
#pragma unroll
      for (int mt = 0; mt < D / 16; ++mt) {
        oacc[mt][0] *= f; oacc[mt][1] *= f; oacc[mt][2] *= f; oacc[mt][3] *= f;
      }
    }
    float* ow = sm.o[warp];  // [head][dim], see o_at
#pragma unroll
    for (int mt = 0; mt < D / 16; ++mt) {
      if constexpr (Q8) {
        const int c = (D / 8) * grp + 2 * mt;  // and the next
        if (2 * tig < G)
          *reinterpret_cast<float2*>(ow + o_at<D, Q8>(2 * tig, c)) = make_float2(oacc[mt][0], oacc[mt][2]);
        if (2 * tig + 1 < G)
          *reinterpret_cast<float2*>(ow + o_at<D, Q8>(2 * tig + 1, c)) = make_float2(oacc[mt][1], oacc[mt][3]);
      } else {
        const int c0 = 16 * mt + grp, c1 = c0 + 8;
        if (2 * tig < G) {
          ow[o_at<D, Q8>(2 * tig, c0)] = oacc[mt][0];
          ow[o_at<D, Q8>(2 * tig, c1)] = oacc[mt][2];
        }
        if (2 * tig + 1 < G) {
          ow[o_at<D, Q8>(2 * tig + 1, c0)] = oacc[mt][1];
          ow[o_at<D, Q8>(2 * tig + 1, c1)] = oacc[mt][3];
        }
      }
    }
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(&sm.mfull));
    ++merges;
  }
  // no more parts
  if (wait_merged()) {
    if (warp == 0 && lane == 0) sm.part.item = -1;
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(&sm.mfull));
  }
}

// Pages a CTA takes at least.  Joining costs 2 us and a page 0.4: 197 tokens of 4
// heads 6.8 us with 4 (one CTA a head), 8.2 with 2, 9.2 with 8; 4096 tokens 10.0,
// 10.8 and 10.6.  Over 8-bit pages, with the clearing kernel: 197 tokens 8.6, 10.0
// and 11.3, 4096 tokens 11.2 and, with 2, 12.5.
constexpr int kMinRun = 4;

struct Ws {
  size_t counter, ml, o, total;
};
Ws ws_layout(const Prob& pr) {
  Ws w;
  size_t o = 256;  // the status word's; the counters follow, so that one kernel clears both
  w.counter = o; o = align_up(o + (size_t)pr.B * pr.Hkv * 4, 256);
  w.ml = o; o = align_up(o + (size_t)2 * kMaxCtas * 2 * pr.G * 4, 256);
  w.o = o; o = align_up(o + (size_t)2 * kMaxCtas * pr.G * pr.d * 4, 256);
  w.total = o;
  return w;
}

template <int D, int G, bool Q8>
cudaError_t launch_t(const Prob& pr, const MaskArgs& m, const void* q, const Pools& pools, const int32_t* seq_lens,
                     const int32_t* idx, char* ws, void* out, cudaStream_t st) {
  const Ws w = ws_layout(pr);
  CUtensorMap kmap, vmap;
  const int64_t rows = pools.num_pages * pr.Hkv * kPage;
  if (Q8 ? !make_tmap_codes(&kmap, pools.k, rows, D, kPage) || !make_tmap_codes(&vmap, pools.v, rows, D, kPage)
         : !make_tmap_page(&kmap, pools.k, rows, D) || !make_tmap_page(&vmap, pools.v, rows, D))
    return cudaErrorInvalidValue;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const size_t smem = sizeof(Smem<D, G, Q8>) + 1024;
  auto kern = paged_decode_kernel<D, G, Q8>;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  e = launch_clear(ws, w.counter + (size_t)pr.B * pr.Hkv * 4, st);
  if (e != cudaSuccess) return e;
  // a CTA per SM; fewer where the capacity has fewer units
  const int64_t units = pr.B * pr.Hkv * (idx ? pr.K + 3 : pools.nb);
  const int64_t grid = std::min<int64_t>(std::min(sm_count(dev), kMaxCtas), ceil_div64(units, kMinRun));
  Parts parts{(int32_t*)(ws + w.counter), (float*)(ws + w.ml), (float*)(ws + w.o)};
  note_launch();
  return launch_pdl(true, kern, dim3((unsigned)grid), dim3(Shape<D, G, Q8>::kThreads), smem, st, pr, m, kmap, vmap,
                    (const uint8_t*)pools.k, pools.ks, pools.vs, (const uint16_t*)q, pools.table, pools.nb,
                    pools.num_pages, seq_lens, idx, parts, kMinRun, (int32_t*)ws, (uint16_t*)out);
}

}  // namespace

size_t paged_decode_ws_bytes(const Prob& pr) { return ws_layout(pr).total; }

cudaError_t launch_paged_decode(const Prob& pr, const MaskArgs& m, const void* q, const Pools& pools,
                                const int32_t* seq_lens, const int32_t* idx, char* ws, void* out, cudaStream_t st) {
#define PISA_PD_CASE(DD, GG) \
  if (pr.d == DD && pr.G == GG)                                                                  \
    return pools.ks ? launch_t<DD, GG, true>(pr, m, q, pools, seq_lens, idx, ws, out, st) \
                    : launch_t<DD, GG, false>(pr, m, q, pools, seq_lens, idx, ws, out, st);
  PISA_PD_CASE(128, 1) PISA_PD_CASE(128, 2) PISA_PD_CASE(128, 4) PISA_PD_CASE(128, 8)
  PISA_PD_CASE(64, 1) PISA_PD_CASE(64, 2) PISA_PD_CASE(64, 4) PISA_PD_CASE(64, 8)
#undef PISA_PD_CASE
  return cudaErrorInvalidValue;
}

}  // namespace pisa
