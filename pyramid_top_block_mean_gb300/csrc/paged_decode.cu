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
// Measured (GB300): 64 ragged sequences of up to 8192 tokens, 32 / 8 heads, d
// = 128: 237 us, 6.6 TB/s of keys and values (the copy rate is 6.8); 2 x 131072
// tokens 150 us (6.5 TB/s); 64 sequences' 35 selected blocks 97 us (6.0 TB/s);
// one sequence of 197 tokens 6.8 us.
#include <algorithm>

#include "paged.cuh"
#include "tc_ptx.cuh"

namespace pisa {

namespace {

constexpr int kWarps = 8;               // consumer warps, 16 keys each: two groups, which take turns at the pages
constexpr int kCons = 32 * kWarps;      // consumer threads
constexpr int kMerge = 96;              // threads that merge a part while the consumers are at the next one
constexpr int kThreads = kCons + 32 + kMerge;  // and the producer warp
constexpr int kPage = 64;
constexpr int kMaxCtas = 1024;          // part slots in the workspace: two per CTA

template <int D, int G>
struct Shape {
  // as many as fit beside the merge buffer; even, so that a stage always goes
  // to the same group, which then sees each of its phases
  static constexpr int kStages = D == 128 ? (G == 8 ? 4 : 6) : (G == 8 ? 10 : 12);
  static_assert(kStages % 2 == 0, "a group must see every phase of its stages");
  static constexpr uint32_t kTile = kPage * D * 2;  // bytes of a page's keys
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

template <int D, int G>
struct Smem {
  uint8_t kv[Shape<D, G>::kStages][2][Shape<D, G>::kTile];
  uint16_t q[Shape<D, G>::kStages][G * D];
  float o[kWarps][G * D];                  // a part's merge
  float m[kWarps][8], l[kWarps][8];
  float jo[kMerge][8], jm[kMerge], jl[kMerge];
  Meta meta[Shape<D, G>::kStages], part;
  uint64_t full[Shape<D, G>::kStages], empty[Shape<D, G>::kStages], mfull, mempty;
  int32_t abort, zero, last_part;
};

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

template <int D, int G>
__global__ void __launch_bounds__(kThreads, 1)
    paged_decode_kernel(Prob pr, MaskArgs mk, const __grid_constant__ CUtensorMap kmap,
                        const __grid_constant__ CUtensorMap vmap, const uint16_t* __restrict__ q,
                        const int32_t* __restrict__ table, int64_t nb, int64_t num_pages,
                        const int32_t* __restrict__ seq_lens, const int32_t* __restrict__ idx, Parts parts,
                        int32_t min_run, int32_t* __restrict__ status, uint16_t* __restrict__ out) {
  constexpr int kStages = Shape<D, G>::kStages;
  constexpr uint32_t kTile = Shape<D, G>::kTile;
  constexpr int kHalf = kPage * 128;  // bytes of a tile's 64-column half
  extern __shared__ unsigned char smem_raw[];
  Smem<D, G>& sm = *reinterpret_cast<Smem<D, G>*>(
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
      ptx::mbar_init(ptx::smem_u32(&sm.full[s]), 1);
      ptx::mbar_init(ptx::smem_u32(&sm.empty[s]), kWarps / 2);
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
    // one stage; page < 0: none to load
    auto emit = [&](const Meta& meta, int32_t page, int32_t head, int64_t seq) -> bool {
      if (it >= kStages &&
          !__all_sync(0xffffffffu, ptx::mbar_wait_fast(ptx::smem_u32(&sm.empty[st]), ph ^ 1, abort)))
        return false;
      if (lane == 0) {
        sm.meta[st] = meta;
        const uint32_t full = ptx::smem_u32(&sm.full[st]);
        const uint32_t bytes = (page >= 0 ? 2 * kTile : 0u) + (meta.first ? (uint32_t)(G * D * 2) : 0u);
        ptx::mbar_arrive_expect_tx(full, bytes);
        if (page >= 0) {
          const int32_t y = (int32_t)(((int64_t)page * pr.Hkv + head) * kPage);
          ptx::tma_load_3d(ptx::smem_u32(sm.kv[st][0]), &kmap, 0, y, 0, full);
          ptx::tma_load_3d(ptx::smem_u32(sm.kv[st][1]), &vmap, 0, y, 0, full);
        }
        if (meta.first)
          ptx::bulk_g2s(ptx::smem_u32(sm.q[st]), q + (seq * pr.Hq + head * G) * D, G * D * 2, full);
      }
      __syncwarp();
      ++it;
      if (++st == kStages) {
        st = 0;
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
        int32_t left = 0;  // entries of the part that hold a page, not yet emitted; the last two are the groups' last
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
          unsigned todo = __ballot_sync(0xffffffffu, mine);
          while (todo && ok) {
            const int x = __ffs(todo) - 1;
            todo &= todo - 1;
            const int32_t bx = __shfl_sync(0xffffffffu, blk, x), px = __shfl_sync(0xffffffffu, page, x);
            const int64_t key0 = (int64_t)bx * kPage;
            meta.rel = (int32_t)(key0 - sp.t);
            meta.klo = px < 0 ? kPage : (int16_t)max((int64_t)0, min((int64_t)kPage, sp.lo - key0));
            meta.khi = (int16_t)min((int64_t)(kPage - 1), sp.t - key0);
            meta.last = --left < 2;
            meta.first = ++count <= 2;
            ok = emit(meta, px, h, b);
          }
        }
      }
      // each group has a stage of every part, if an empty one
      for (; count < 2 && ok; ++count) {
        meta.klo = kPage;
        meta.first = meta.last = 1;
        ok = emit(meta, -1, h, b);
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
      ok = emit(meta, -1, 0, 0) && emit(meta, -1, 0, 0);
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
        const float* at = sm.o[0] + g * D + (c ^ (8 * (g >> 1)));
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
  const int r16 = 16 * (warp & 3);
  // ldmatrix rows: lane l addresses row l % 8 of matrix l / 8
  const int krow = r16 + (lane & 7) + ((lane >> 3) & 1) * 8, kch = lane >> 4;
  const int vrow = r16 + (lane & 7) + (lane >> 4) * 8, vch = (lane >> 3) & 1;
  uint32_t bq[D / 16][2];
  float oacc[D / 16][4];
  float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.0f, l1 = 0.0f;  // heads 2 tig, 2 tig + 1
  float sl0 = 0.0f, sl1 = 0.0f;
  // group warp / 4 takes every other stage
  int st = (warp >> 2) - 2, ph = 0, merges = 0;
  auto wait_merged = [&] {  // the merge buffer is free
    const bool ok = merges == 0 || ptx::mbar_wait_fast(ptx::smem_u32(&sm.mempty), (merges - 1) & 1, abort);
    if (!__all_sync(0xffffffffu, ok)) {
      give_up();
      return false;
    }
    return true;
  };
  for (;;) {
    if ((st += 2) >= kStages) {
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
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks) {
        const uint32_t* qr = reinterpret_cast<const uint32_t*>(sm.q[st] + (grp < G ? grp : 0) * D + 16 * ks);
        bq[ks][0] = grp < G ? qr[tig] : 0u;
        bq[ks][1] = grp < G ? qr[tig + 4] : 0u;
        oacc[ks][0] = oacc[ks][1] = oacc[ks][2] = oacc[ks][3] = 0.0f;
      }
      m0 = m1 = -INFINITY;
      l0 = l1 = 0.0f;
      if (mk.slopes) {
        const float* sl = mk.slopes + (int64_t)(meta.item % pr.Hkv) * G;
        sl0 = 2 * tig < G ? sl[2 * tig] * kLog2e : 0.0f;
        sl1 = 2 * tig + 1 < G ? sl[2 * tig + 1] * kLog2e : 0.0f;
      }
    }
    if (meta.klo <= meta.khi && r16 <= meta.khi && r16 + 15 >= meta.klo) {
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
          mma16816(d, a[ks], bq[ks][0], bq[ks][1]);
          mma16816(e, a[ks + 1], bq[ks + 1][0], bq[ks + 1][1]);
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
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(&sm.empty[st]));
    if (!meta.last) continue;

    // ------------------ end of a part: hand (m, l, o) to the merging warps
#pragma unroll
    for (int o = 4; o <= 16; o <<= 1) {
      l0 += __shfl_xor_sync(0xffffffffu, l0, o);
      l1 += __shfl_xor_sync(0xffffffffu, l1, o);
    }
    if (!wait_merged()) break;
    if (warp == 0 && lane == 0) sm.part = meta;
    if (grp == 0) {
      *reinterpret_cast<float2*>(&sm.m[warp][2 * tig]) = make_float2(m0, m1);
      *reinterpret_cast<float2*>(&sm.l[warp][2 * tig]) = make_float2(l0, l1);
    }
    // o[warp][head][dim]; the dims of a head are permuted by 8 (head / 2), which spreads tig over the banks
    float* ow = sm.o[warp];
#pragma unroll
    for (int mt = 0; mt < D / 16; ++mt) {
      const int c0 = (16 * mt + grp) ^ (8 * tig), c1 = (16 * mt + grp + 8) ^ (8 * tig);
      if (2 * tig < G) {
        ow[2 * tig * D + c0] = oacc[mt][0];
        ow[2 * tig * D + c1] = oacc[mt][2];
      }
      if (2 * tig + 1 < G) {
        ow[(2 * tig + 1) * D + c0] = oacc[mt][1];
        ow[(2 * tig + 1) * D + c1] = oacc[mt][3];
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
// 10.8 and 10.6.
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

template <int D, int G>
cudaError_t launch_t(const Prob& pr, const MaskArgs& m, const void* q, const Pools& pools, const int32_t* seq_lens,
                     const int32_t* idx, char* ws, void* out, cudaStream_t st) {
  const Ws w = ws_layout(pr);
  CUtensorMap kmap, vmap;
  const int64_t rows = pools.num_pages * pr.Hkv * kPage;
  if (!make_tmap_page(&kmap, pools.k, rows, D) || !make_tmap_page(&vmap, pools.v, rows, D))
    return cudaErrorInvalidValue;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const size_t smem = sizeof(Smem<D, G>) + 1024;
  auto kern = paged_decode_kernel<D, G>;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  e = launch_clear(ws, w.counter + (size_t)pr.B * pr.Hkv * 4, st);
  if (e != cudaSuccess) return e;
  // a CTA per SM; fewer where the capacity has fewer units
  const int64_t units = pr.B * pr.Hkv * (idx ? pr.K + 3 : pools.nb);
  const int64_t grid = std::min<int64_t>(std::min(sm_count(dev), kMaxCtas), ceil_div64(units, kMinRun));
  Parts parts{(int32_t*)(ws + w.counter), (float*)(ws + w.ml), (float*)(ws + w.o)};
  note_launch();
  return launch_pdl(true, kern, dim3((unsigned)grid), dim3(kThreads), smem, st, pr, m, kmap, vmap,
                    (const uint16_t*)q, pools.table, pools.nb, pools.num_pages, seq_lens, idx, parts, kMinRun,
                    (int32_t*)ws, (uint16_t*)out);
}

}  // namespace

size_t paged_decode_ws_bytes(const Prob& pr) { return ws_layout(pr).total; }

cudaError_t launch_paged_decode(const Prob& pr, const MaskArgs& m, const void* q, const Pools& pools,
                                const int32_t* seq_lens, const int32_t* idx, char* ws, void* out, cudaStream_t st) {
#define PISA_PD_CASE(DD, GG) \
  if (pr.d == DD && pr.G == GG) return launch_t<DD, GG>(pr, m, q, pools, seq_lens, idx, ws, out, st);
  PISA_PD_CASE(128, 1) PISA_PD_CASE(128, 2) PISA_PD_CASE(128, 4) PISA_PD_CASE(128, 8)
  PISA_PD_CASE(64, 1) PISA_PD_CASE(64, 2) PISA_PD_CASE(64, 4) PISA_PD_CASE(64, 8)
#undef PISA_PD_CASE
  return cudaErrorInvalidValue;
}

}  // namespace pisa
