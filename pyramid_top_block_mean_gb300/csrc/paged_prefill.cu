// paged_prefill.cu -- dense attention of new tokens (a prompt, or a chunk of
// one behind a cached part) over the paged cache, on the tcgen05 tensor cores.
//
// For every row (token, query head): o = sum_j p_j v_j / sum_j p_j over the
// keys that it sees, p_j = 2^(x_j - m), in one pass over the keys.  The
// reference m only follows the running maximum when that has grown by more
// than 2^8: until then the weights stay below 2^8, which neither fp32 sums nor
// bf16 weights mind, and the output tile needs no rescaling.
//
// One CTA takes 256 rows -- 256 / G tokens of the G heads that share a key
// head -- as two tiles of 128, against tiles of 128 keys (two pages):
//   - a loader warp brings the query tiles once, then keys and values through
//     one ring of stages by TMA (128-byte swizzle); a page is found through
//     the table, so a tile is four boxes;
//   - a warp per row tile issues S = Q K^T into TMEM and, when its weights P
//     are there, O += P V with P read from TMEM (over the columns of S, which
//     the warps have read by then) and V in its natural key-major layout.  The
//     two tiles alternate: while one's softmax runs, the other's MMAs do;
//   - two groups of four warps do the softmax, one thread per row, so that a
//     row's maximum and sum need no exchange.
// Work: 4 d flops for each (row, key).  For d = 128 the two tiles' MMAs of a
// step take about 2300 cycles (2048 at the nominal rate; both operands of S
// come from shared memory, which they saturate) and one tile's chain -- S,
// softmax, P V, the next S -- about 2800, which is what a step takes.
// CTAs are persistent: the loader claims the next 256 rows when it has loaded
// what the current ones need.
//
// Measured (GB300, 16 / 4 heads, d = 128): 16384 tokens 662 us (1660 TFLOP/s of
// the seen pairs, 86 % of cuBLAS's measured rate), 65536 tokens 10.7 ms (1640),
// 16384 with a tanh cap 950 to 963 us (1621 where scores pass half the cap),
// with a distance bias 983, with a window of 1024 141, at d = 64 583 us; prompts
// of 4096 and 3000 tokens 93 us, 61 tokens behind 65536 cached ones 50 us.
//
// Rows with few tokens and a long cache: the keys of a CTA's rows are split
// over several CTAs, whose parts a second kernel joins.
//
// 8-bit pages (Q8): TMA brings a tile's codes into its stage, and a fourth
// warpgroup turns them into the bf16 numbers that they stand for in place
// (exactly: the results are those over bf16 pages of these numbers), which is
// all that the MMAs see.  Shared memory, which the MMAs saturate, bounds that:
// 4400 cycles a step, of which 300 are the hand-over, 300 the register split,
// and 1000 the conversion (without its arithmetic 690 of 785 us, without its
// accesses 566).  So a long prompt expands the pages to bf16 first and reads
// those.  8192 tokens behind 8192: 547 us (1507 TFLOP/s; 785 from the codes), 61
// behind 65536 from the codes 56 us.  (Two warps for the keys and two for the
// values, each with a step's time for its tile: 928 us.)
#include <cudaTypedefs.h>

#include <algorithm>

#include "paged.cuh"
#include "tc_ptx.cuh"

namespace pisa {

namespace {

constexpr int kRows = 128;  // rows of a tile
constexpr int kKeys = 128;  // keys of a tile
constexpr int kPage = 64;
constexpr int kMmaWarp = 8;   // warps 0-3 and 4-7: softmax of tile 0 and 1; 8 and 9: their MMAs
constexpr int kLoadWarp = 10;
constexpr int kConvWarp = 12;  // Q8: warps 12-15 convert
// Registers a thread: the softmax warpgroups hold a row of S each, the others
// give up what they need (2 x 216 + 72 = 3 x 168, the launch's share; with the
// converting warpgroup 2 x 192 + 64 + 64 = 4 x 128).
#define PISA_SOFTMAX_REGS "216"
#define PISA_OTHER_REGS "72"
#define PISA_SOFTMAX_REGS_Q8 "192"
#define PISA_OTHER_REGS_Q8 "64"
#define PISA_CONVERT_REGS_Q8 "64"
constexpr float kSlack = 8.0f;  // log2 of how far weights may exceed 1

// Q8: pages of e4m3.
template <int D, bool Q8>
struct Cfg {
  static constexpr int kThreads = Q8 ? 512 : 384;  // warp 11 only makes up the third warpgroup
  static constexpr int kStages = D == 128 ? 5 : (Q8 ? 7 : 10);
  static constexpr uint32_t kTile = kKeys * D * 2;  // bytes of a key or value tile, and of a query tile
  static constexpr uint32_t kCodes = kKeys * D;     // and of a tile in e4m3
};

constexpr int kItems = 2;  // items in flight: the loader is at most one ahead

// What the loader tells the other warps about an item: 256 rows against a run
// of key tiles.
struct Item {
  int32_t bh, tile, split;  // bh < 0: no more items
  int32_t number, clean;    // its place among all; taken a second time
  int32_t len, cnt;         // of the sequence; cnt rows before it are new
  int32_t fits;             // its lengths do
  int32_t ja, jb;           // key tiles
  int32_t wa[2], wb[2];     // and those that each row tile takes part in
  int32_t klo, khi;         // first and last key that any row sees
  int32_t fill;             // fills of the ring before the item's first
};

template <int D, bool Q8>
struct Smem {
  using C = Cfg<D, Q8>;
  uint8_t q[2][C::kTile];
  uint8_t kv[C::kStages][C::kTile];
  // Q8: a tile's codes.  Of d = 128 they take the second half of its stage: the
  // thread that turns a row's codes into its numbers puts the second half of
  // these where the codes were, and nobody else's.
  uint8_t codes[Q8 && D == 64 ? C::kStages : 1][Q8 && D == 64 ? C::kCodes : 16];
  uint8_t scale[Q8 ? C::kStages : 1][Q8 ? kKeys : 16];  // the rows'
  int32_t have[C::kStages];                             // bit p: page p of the tile is there
  uint64_t raw[C::kStages];                             // the codes are
  uint64_t full[C::kStages], empty[C::kStages];
  uint64_t ifull[kItems], iempty[kItems];
  uint64_t qfull[2], qempty[2], scrub, sfull[2], pfull[2][2], odone[2], done[2], lent, rows_out;
  Item item[kItems];
  uint32_t tmem;
  int32_t abort, zero, bad_page;
  int32_t again[kItems];  // a row of the item is not finite
};

struct Args {
  int64_t n, nb, num_pages;
  const uint16_t *q, *k, *v;
  const uint8_t *ks, *vs;  // scales of e4m3 rows
  const int32_t *seq_lens, *new_lens, *table;
  int32_t *status, *claimed;  // claimed: items taken beyond each CTA's first
  uint16_t* out;
  float *part_o, *part_ml;  // [split][256-row group][256][D] and [..][2] (m in log2 units, l)
  // 256-row groups per (sequence, key head), parts of the keys, log2 of a tile's tokens, items in all
  int32_t tiles, splits, lg_tokens, items;
};

__device__ __forceinline__ uint64_t desc_mn_sw128(uint32_t saddr, uint32_t lbo) {
  uint64_t d = 0;
  d |= (uint64_t)((saddr & 0x3FFFFu) >> 4);
  d |= (uint64_t)((lbo >> 4) & 0x3FFFu) << 16;  // next 64 MN elements
  d |= (uint64_t)(1024u >> 4) << 32;            // next 8 K rows
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)2 << 61;
  return d;
}

// D[tmem] (+)= A[tmem] * B[smem desc]^T
__device__ __forceinline__ void mma_ts_bf16(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                                            uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
      "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, int32_t x, int32_t y, int32_t z,
                                            int32_t w, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar)
      : "memory");
}

__device__ __forceinline__ bool elect_one() {
  uint32_t x;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(x));
  return x != 0;
}

__device__ __forceinline__ void prefetch_l1(const void* p) { asm volatile("prefetch.global.L1 [%0];" ::"l"(p)); }

// Both MMA warps meet; true for both if both say so.
__device__ __forceinline__ bool both_ok(bool ok) {
  uint32_t x;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %1, 0;\n\t"
      "bar.red.and.pred q, 3, 64, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(x)
      : "r"((uint32_t)ok)
      : "memory");
  return x != 0;
}

// The two MMA warps' turns: warp v waits for its own, and hands over to the other.
__device__ __forceinline__ void turn_wait(int v) { asm volatile("bar.sync %0, 64;" ::"r"(1 + v) : "memory"); }
__device__ __forceinline__ void turn_pass(int v) { asm volatile("bar.arrive %0, 64;" ::"r"(2 - v) : "memory"); }

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.ftz.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
// The factor that caps two small scores, from MaskArgs::by times each.
__device__ __forceinline__ uint64_t cap_factor(const MaskArgs& m, uint64_t y2) {
  const uint64_t w2 = mul2(y2, y2);
  uint64_t f = ptx::fma2(w2, ptx::pack2(m.tk[3], m.tk[3]), ptx::pack2(m.tk[2], m.tk[2]));
  f = ptx::fma2(w2, f, ptx::pack2(m.tk[1], m.tk[1]));
  return ptx::fma2(w2, f, ptx::pack2(m.tk[0], m.tk[0]));
}
__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// |x| <= lim ? a : b.  (In PTX: over a row's worth of scores the compiler takes
// the expression for 128 branches and spills 3 KB, three times the time.)
__device__ __forceinline__ float within(float x, float lim, float a, float b) {
  float y;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.le.f32 p, %1, %2;\n\t"
      "selp.f32 %0, %3, %4, p;\n\t}"
      : "=f"(y)
      : "f"(fabsf(x)), "f"(lim), "f"(a), "f"(b));
  return y;
}

// A weight of zero does not undo a value that is not finite: the MMA takes the
// values of all keys of a tile into all of its rows.  An item with a row that
// came out without being finite is therefore taken a second time, "clean": the
// loader puts zeros in the place of such values, the softmax warps note for
// each row in which dims it sees one, and those outputs are set at the end.
// (At the pipeline's pace, so that its waits stay short whatever the cache
// holds; not inlined, to keep the code of the first way small.)

// A tile's values in shared memory, by the loader warp.
template <uint32_t BYTES>
__device__ __noinline__ void clean_tile(uint8_t* tile) {
  auto clean = [](uint32_t x) {
    if ((x & 0x7f80u) == 0x7f80u) x &= 0xffff0000u;
    if ((x & 0x7f800000u) == 0x7f800000u) x &= 0xffffu;
    return x;
  };
#pragma unroll 4
  for (uint32_t e = (threadIdx.x & 31) * 16; e < BYTES; e += 512) {
    uint4 x = *reinterpret_cast<const uint4*>(tile + e);
    x.x = clean(x.x); x.y = clean(x.y); x.z = clean(x.z); x.w = clean(x.w);
    *reinterpret_cast<uint4*>(tile + e) = x;
  }
}

// The dims in which a row sees values that are +inf or NaN, and -inf or NaN:
// bit l of word (i, e) stands for dim 64 i + 2 l + e.
template <int D>
struct Marks {
  uint32_t up[D / 64][2], down[D / 64][2];
};

// Notes what the key tiles ja .. jb - 1 hold for the rows of a warp, a lane's
// seeing lo .. hi.  (About 1 us a tile, some 5 us one full of such values, so
// that the waits on these warps stay within their limits for any cache.)
template <int D>
__device__ __noinline__ void mark_tiles(const Args& a, int32_t Hkv, int32_t bh, int32_t ja, int32_t jb, int32_t lo,
                                        int32_t hi, Marks<D>* marks) {
  constexpr int kBatch = 16, W = D / 64;  // keys in flight
  const int lane = threadIdx.x & 31;
  const int64_t b = (uint32_t)bh / (uint32_t)Hkv;
  const int64_t h = bh - b * Hkv;
  // bits 4 i + 2 e and 4 i + 2 e + 1: up and down of dim 64 i + 2 lane + e in the words of a key
  auto flags = [](uint32_t w, int i) {
    uint32_t f = 0;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const uint32_t y = e ? w >> 16 : w & 0xffffu, m = y & 0x7fffu;
      if (m >= 0x7f80u) f |= (m > 0x7f80u ? 3u : (y >> 15 ? 2u : 1u)) << (4 * i + 2 * e);
    }
    return f;
  };
  auto note = [&](uint32_t f, bool seen) {
    for (int i = 0; i < W; ++i) {
      for (int e = 0; e < 2; ++e) {
        const uint32_t up = __ballot_sync(0xffffffffu, f >> (4 * i + 2 * e) & 1);
        const uint32_t down = __ballot_sync(0xffffffffu, f >> (4 * i + 2 * e + 1) & 1);
        if (seen) {
          marks->up[i][e] |= up;
          marks->down[i][e] |= down;
        }
      }
    }
  };
  constexpr uint32_t kAll = W == 1 ? 0xfu : 0xffu;
  bool full = false;  // every dim of the row is marked both ways: it cannot change any more
  for (int32_t key0 = ja * kKeys; key0 < jb * kKeys; key0 += kPage) {
    const bool none = full || lo >= key0 + kPage || hi < key0, whole = lo <= key0 && hi >= key0 + kPage - 1;
    if (__all_sync(0xffffffffu, none)) continue;
    const int32_t page = a.table[b * a.nb + key0 / kPage];
    if (page < 0 || page >= a.num_pages) continue;
    const uint32_t* v = reinterpret_cast<const uint32_t*>(a.v + ((int64_t)page * Hkv + h) * kPage * D) + lane;
    uint32_t f = 0;
    for (int k0 = 0; k0 < kPage && !__all_sync(0xffffffffu, f == kAll); k0 += kBatch) {
      uint32_t x[kBatch][W], odd = 0;
#pragma unroll
      for (int k = 0; k < kBatch; ++k)
#pragma unroll
        for (int i = 0; i < W; ++i) x[k][i] = v[(k0 + k) * (D / 2) + 32 * i];
#pragma unroll
      for (int k = 0; k < kBatch; ++k)
#pragma unroll
        for (int i = 0; i < W; ++i) odd |= (x[k][i] & 0x7fff7fffu) + 0x00800080u;  // a carry where all of an exponent is set
      if (!__any_sync(0xffffffffu, (odd & 0x80008000u) != 0)) continue;
#pragma unroll
      for (int k = 0; k < kBatch; ++k)
#pragma unroll
        for (int i = 0; i < W; ++i) f |= flags(x[k][i], i);
    }
    if (!__any_sync(0xffffffffu, f != 0)) continue;
    if (__all_sync(0xffffffffu, none || whole)) {
      note(f, whole);
    } else {
#pragma unroll 1
      for (int k = 0; k < kPage; ++k) {
        f = 0;
        for (int i = 0; i < W; ++i) f |= flags(v[k * (D / 2) + 32 * i], i);
        note(f, key0 + k >= lo && key0 + k <= hi);
      }
    }
    uint32_t both = 0xffffffffu;
    for (int i = 0; i < W; ++i)
      for (int e = 0; e < 2; ++e) both &= marks->up[i][e] & marks->down[i][e];
    full = both == 0xffffffffu;
  }
}

// The same for pages of e4m3, whose rows are finite or NaN throughout (scale
// 255): true for a lane that sees one of the latter.
__device__ __noinline__ bool sees_nan_row(const Args& a, int32_t Hkv, int32_t bh, int32_t ja, int32_t jb, int32_t lo,
                                          int32_t hi) {
  const int lane = threadIdx.x & 31;
  const int64_t b = (uint32_t)bh / (uint32_t)Hkv;
  const int64_t h = bh - b * Hkv;
  bool found = false;
  for (int32_t key0 = ja * kKeys; key0 < jb * kKeys; key0 += kPage) {
    const int32_t first = max(lo - key0, 0), last = min(hi - key0, kPage - 1);
    const bool none = found || first > last;
    if (__all_sync(0xffffffffu, none)) continue;
    const int32_t page = a.table[b * a.nb + key0 / kPage];
    if (page < 0 || page >= a.num_pages) continue;
    const uint8_t* s = a.vs + ((int64_t)page * Hkv + h) * kPage + lane;
    const uint32_t m0 = __ballot_sync(0xffffffffu, s[0] == 255), m1 = __ballot_sync(0xffffffffu, s[32] == 255);
    const uint64_t nan = (uint64_t)m1 << 32 | m0;
    if (!none) found = (nan >> first & ~0ull >> (kPage - 1 - (last - first))) != 0;
  }
  return found;
}

// Sets the marked outputs of the warp's rows: out + orow, or with splits the
// part at `at`.
template <int D>
__device__ __noinline__ void set_marked(const Args& a, bool row, int64_t orow, int64_t at, const Marks<D>* marks) {
  const int lane = threadIdx.x & 31;
  __syncwarp();  // the rows' stores come before those that replace them
  for (unsigned todo = __ballot_sync(0xffffffffu, row); todo; todo &= todo - 1) {
    const int x = __ffs(todo) - 1;
    const int64_t to = __shfl_sync(0xffffffffu, a.splits > 1 ? at * D : orow, x);
    for (int i = 0; i < D / 64; ++i) {
      for (int e = 0; e < 2; ++e) {
        const bool up = (__shfl_sync(0xffffffffu, marks->up[i][e], x) >> lane & 1) != 0;
        const bool down = (__shfl_sync(0xffffffffu, marks->down[i][e], x) >> lane & 1) != 0;
        if (!up && !down) continue;
        const float y = up && down ? NAN : (up ? INFINITY : -INFINITY);
        const int64_t dim = to + 64 * i + 2 * lane + e;
        if (a.splits > 1) a.part_o[dim] = y;
        else a.out[dim] = __bfloat16_as_ushort(__float2bfloat16(y));
      }
    }
  }
}

// MODE 0: scores are scale * q . k; 1: with a cap and / or a distance bias.
template <int D, int MODE, bool Q8>
__global__ void __launch_bounds__(Cfg<D, Q8>::kThreads, 1)
    paged_prefill_kernel(const __grid_constant__ Prob pr, const __grid_constant__ MaskArgs mk,
                         const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                         const __grid_constant__ CUtensorMap vmap, const __grid_constant__ Args a) {
  constexpr int kStages = Cfg<D, Q8>::kStages;
  constexpr uint32_t kTile = Cfg<D, Q8>::kTile;
  constexpr uint32_t kHalf = kKeys * 128;      // bytes of a tile's 64-column half
  constexpr uint32_t kPageHalf = kPage * 128;  // and of a page's
  constexpr uint32_t kIdescS = ptx::idesc_bf16_f32(kRows, kKeys);
  constexpr uint32_t kIdescO = ptx::idesc_bf16_f32(kRows, D) | (1u << 16);  // values MN-major
  extern __shared__ unsigned char smem_raw[];
  Smem<D, Q8>& sm =
      *reinterpret_cast<Smem<D, Q8>*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  volatile int32_t* abort = &sm.abort;

  if (warp == kLoadWarp && lane == 3) {  // the first item's lengths
    const int64_t b0 = (uint32_t)(blockIdx.x / a.splits) % (uint32_t)(pr.B * pr.Hkv) / (uint32_t)pr.Hkv;
    prefetch_l1(a.seq_lens + b0);
    if (a.new_lens) prefetch_l1(a.new_lens + b0);
  }
  if (threadIdx.x == 0) {
    for (int k = 0; k < kStages; ++k) {
      ptx::mbar_init(ptx::smem_u32(&sm.raw[k]), 1);
      ptx::mbar_init(ptx::smem_u32(&sm.full[k]), Q8 ? 4 : 1);
      ptx::mbar_init(ptx::smem_u32(&sm.empty[k]), 2);
    }
    for (int k = 0; k < kItems; ++k) {
      ptx::mbar_init(ptx::smem_u32(&sm.ifull[k]), 1);
      ptx::mbar_init(ptx::smem_u32(&sm.iempty[k]), Q8 ? 14 : 10);
    }
    ptx::mbar_init(ptx::smem_u32(&sm.scrub), 1);
    ptx::mbar_init(ptx::smem_u32(&sm.lent), 1);
    ptx::mbar_init(ptx::smem_u32(&sm.rows_out), 8);
    for (int v = 0; v < 2; ++v) {
      ptx::mbar_init(ptx::smem_u32(&sm.qfull[v]), 1);
      ptx::mbar_init(ptx::smem_u32(&sm.qempty[v]), 1);
      ptx::mbar_init(ptx::smem_u32(&sm.sfull[v]), 1);
      ptx::mbar_init(ptx::smem_u32(&sm.pfull[v][0]), 4);
      ptx::mbar_init(ptx::smem_u32(&sm.pfull[v][1]), 4);
      ptx::mbar_init(ptx::smem_u32(&sm.odone[v]), 1);
      ptx::mbar_init(ptx::smem_u32(&sm.done[v]), 1);
    }
    sm.abort = 0;
    sm.zero = 0;
    sm.bad_page = 0;
    for (int k = 0; k < kItems; ++k) sm.again[k] = 0;
    ptx::fence_mbar_init();
    ptx::fence_proxy_async_smem();
  }
  if (warp == kLoadWarp && lane < 3) ptx::prefetch_map(lane == 0 ? &qmap : (lane == 1 ? &kmap : &vmap));
  if (warp == kMmaWarp) {
    ptx::tmem_alloc(ptx::smem_u32(&sm.tmem), 512);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  pdl_wait();  // from here on the status word and the claims are clear
  // the joining kernel, where there is one, may be set up as CTAs of this one end
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const uint32_t tmem = sm.tmem;
  const int tokens = 1 << a.lg_tokens;  // of one row tile
  const uint32_t heads = (uint32_t)(pr.B * pr.Hkv);

  if (Q8 && warp >= kConvWarp) {
    // ----------------------------------------------------------- converters
    // Thread r turns row r of a tile into bf16, exactly (codes to numbers: see
    // row_factor), into the row's place of the MMAs' operand.  The 8 lanes of one pass over the banks have the 8 rows of a
    // swizzle: no two of their pieces share banks, read or written.
    asm volatile("setmaxnreg.dec.sync.aligned.u32 " PISA_CONVERT_REGS_Q8 ";");
    const int r = threadIdx.x & 127;
    bool ok = true;
    int st = 0, ph = 0;
    for (int items = 0;; ++items) {
      ok = ok && __all_sync(0xffffffffu, ptx::mbar_wait_fast(ptx::smem_u32(&sm.ifull[items % kItems]),
                                                             (items / kItems) & 1, abort)) != 0;
      if (!ok) break;
      const Item* ip = &sm.item[items % kItems];
      if (ip->bh < 0) break;
      const int ja = ip->ja, jb = ip->jb, klo = ip->klo, khi = ip->khi;
      const bool clean = ip->clean != 0;
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(&sm.iempty[items % kItems]));
      for (int f = 0; f < 2 * (jb - ja) && ok; ++f) {
        ok = __all_sync(0xffffffffu, ptx::mbar_wait_fast(ptx::smem_u32(&sm.raw[st]), ph, abort)) != 0;
        if (!ok) break;
        const uint8_t* from = (D == 64 ? sm.codes[D == 64 ? st : 0] : sm.kv[st] + kTile / 2) + r * D;
        const uint32_t scale = sm.scale[Q8 ? st : 0][r];
        // A value that no row of the item sees (behind the sequence's end among
        // them) may be anything, and a weight of zero does not undo a NaN: it
        // becomes zero; "clean", so does one that is not finite.
        const int32_t key = (ja + (f >> 1)) * kKeys + r;
        const bool zero = (f & 1) != 0 && (key < klo || key > khi || (sm.have[st] >> (r / kPage) & 1) == 0 ||
                                           (clean && scale == 255u));
        const uint32_t by = zero ? 0u : row_factor(scale), more = row_is_large(scale) ? row_factor_large(scale) : 0u;
        uint4 c[D / 16];
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
          c[i] = *reinterpret_cast<const uint4*>(from + ((i ^ (D == 128 ? r & 7 : (r >> 1) & 3)) << 4));
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          const uint32_t w[4] = {c[i].x, c[i].y, c[i].z, c[i].w};
          uint32_t x[8];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            x[2 * k] = mul_bf16x2(codes_lo(w[k]), by);
            x[2 * k + 1] = mul_bf16x2(codes_hi(w[k]), by);
          }
          if (more && !zero) {
#pragma unroll
            for (int k = 0; k < 8; ++k) x[k] = mul_bf16x2(x[k], more);
          }
          uint8_t* to = sm.kv[st] + (i >> 2) * kHalf + r * 128;
          *reinterpret_cast<uint4*>(to + (((2 * i & 7) ^ (r & 7)) << 4)) = make_uint4(x[0], x[1], x[2], x[3]);
          *reinterpret_cast<uint4*>(to + (((2 * i + 1 & 7) ^ (r & 7)) << 4)) = make_uint4(x[4], x[5], x[6], x[7]);
        }
        ptx::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(&sm.full[st]));
        if (++st == kStages) { st = 0; ph ^= 1; }
      }
      if (++st == kStages) { st = 0; ph ^= 1; }  // the stage that the rows go out through
    }
    if (!ok && lane == 0) *abort = 1;
  } else if (warp >= 8) {
    if constexpr (Q8) asm volatile("setmaxnreg.dec.sync.aligned.u32 " PISA_OTHER_REGS_Q8 ";");
    else asm volatile("setmaxnreg.dec.sync.aligned.u32 " PISA_OTHER_REGS ";");
    if (warp == kLoadWarp) {
      // ------------------------------------------------------------ loader
      bool ok = true;
      int fills = 0, scrubs = 0, items = 0, qfills[2] = {0, 0};
      int st = 0, ph = 0;  // stage and phase of the next fill
      auto advance = [&] {
        ++fills;
        if (++st == kStages) { st = 0; ph ^= 1; }
      };
      auto wait = [&](uint64_t* bar, int phase) {
        ok = ok && __all_sync(0xffffffffu, ptx::mbar_wait_fast(ptx::smem_u32(bar), phase & 1, abort)) != 0;
        return ok;
      };
      // the stage that an item's rows go out through, until they have
      int lent = -1, lendings = 0;
      auto take_back = [&] {
        if (lent >= 0) wait(&sm.rows_out, lendings++);
        lent = -1;
        return ok;
      };
      auto claim = [&] {
        int32_t k = 0;
        if (lane == 0) k = (int32_t)gridDim.x + atomicAdd(a.claimed, 1);
        return __shfl_sync(0xffffffffu, k, 0);
      };
      // the item that a slot held, where it has to be taken a second time (-1: not)
      auto to_repeat = [&](int slot) {
        if (*(volatile int32_t*)&sm.again[slot] == 0) return -1;
        const int32_t k = sm.item[slot].number;
        __syncwarp();
        if (lane == 0) sm.again[slot] = 0;
        __syncwarp();
        return k;
      };
      // the last tokens' items, which see the most keys, come first; a CTA
      // that has loaded what its item needs claims the next one
      int32_t now = blockIdx.x, next = 0;
      bool clean = false;  // `now` is taken a second time, and `next` follows it
      while (ok) {
        if (now >= a.items) {
          // none left, unless one of the last items, the older one first
          int32_t back = -1;
          for (int k = min(items, kItems); k > 0 && back < 0; --k) {
            const int n = items - k;
            if (wait(&sm.iempty[n % kItems], n / kItems)) back = to_repeat(n % kItems);
          }
          if (!ok || back < 0) break;
          next = now;
          now = back;
          clean = true;
        }
        uint32_t x = (uint32_t)now;
        Item it;
        it.number = now;
        it.clean = clean;
        it.split = (int32_t)(x % (uint32_t)a.splits);
        x /= (uint32_t)a.splits;
        it.bh = (int32_t)(x % heads);
        it.tile = a.tiles - 1 - (int32_t)(x / heads);
        const int64_t b = (uint32_t)it.bh / (uint32_t)pr.Hkv;
        const int h = it.bh - (int)b * pr.Hkv;
        const int64_t i0 = (int64_t)it.tile * 2 * tokens;
        int64_t len, cnt;
        it.fits = new_span(a.seq_lens, a.new_lens, b, a.n, pr.N, &len, &cnt);
        if (!it.fits && lane == 0) set_status(a.status, PISA_DEV_BAD_SEQ_LEN);
        if (i0 >= cnt) {
          now = claim();
          continue;
        }
        it.len = (int32_t)len;
        it.cnt = (int32_t)cnt;
        // keys that each row tile sees
        int32_t lo[2], hi[2];
#pragma unroll
        for (int v = 0; v < 2; ++v) {
          lo[v] = 0x7fffffff;
          hi[v] = -1;
          const int64_t r0 = i0 + v * tokens, r1 = min(cnt, r0 + tokens);  // its tokens
          if (!it.fits || r0 >= r1) continue;
          if (!mk.first_key) {  // both ends grow with the position
            int64_t l, u;
            key_span(mk, b, a.n, r0, len - cnt + r0, len, &l, &u);
            lo[v] = (int32_t)l;
            key_span(mk, b, a.n, r1 - 1, len - cnt + r1 - 1, len, &l, &u);
            hi[v] = (int32_t)u;
          } else {
            for (int64_t i = r0 + lane; i < r1; i += 32) {
              int64_t l, u;
              key_span(mk, b, a.n, i, len - cnt + i, len, &l, &u);
              if (l > u) continue;
              lo[v] = min(lo[v], (int32_t)l);
              hi[v] = max(hi[v], (int32_t)u);
            }
            lo[v] = __reduce_min_sync(0xffffffffu, lo[v]);
            hi[v] = __reduce_max_sync(0xffffffffu, hi[v]);
          }
        }
        const int32_t klo = min(lo[0], lo[1]), khi = max(hi[0], hi[1]);
        it.ja = it.jb = 0;
        if (khi >= 0) {
          const int j0 = klo / kKeys;
          const uint32_t cntj = (uint32_t)(khi / kKeys + 1 - j0);
          it.ja = j0 + (int)(a.splits == 1 ? 0 : (uint64_t)cntj * it.split / (uint32_t)a.splits);
          it.jb = j0 + (int)(a.splits == 1 ? cntj : (uint64_t)cntj * (it.split + 1) / (uint32_t)a.splits);
        }
#pragma unroll
        for (int v = 0; v < 2; ++v) {
          it.wa[v] = hi[v] < 0 ? it.jb : max(it.ja, lo[v] / kKeys);
          it.wb[v] = hi[v] < 0 ? it.jb : min(it.jb, hi[v] / kKeys + 1);
          if (it.wb[v] < it.wa[v]) it.wb[v] = it.wa[v];
        }
        it.klo = klo;
        it.khi = khi;
        it.fill = fills;
        // lane l: the page of block 2 j + l, -1: none of its keys is seen, -2: outside the pool
        const int32_t* trow = a.table + b * a.nb;
        auto look_up = [&](int j) {
          const int32_t blk = 2 * j + lane;
          int32_t e = -1;
          if ((int64_t)blk * kPage <= khi && (int64_t)blk * kPage + kPage > klo && blk < 2 * it.jb) {
            e = trow[blk];
            if (e < 0 || e >= a.num_pages) e = -2;
          }
          return e;
        };
        int32_t entry = look_up(it.ja);  // under way while the item is handed out
        const int is = items % kItems;
        if (items >= kItems) {
          if (!wait(&sm.iempty[is], (items / kItems) + 1)) break;
          const int32_t back = to_repeat(is);
          if (back >= 0) {
            next = now;
            now = back;
            clean = true;
            continue;
          }
        }
        if (lane == 0) {
          sm.item[is] = it;
          ptx::mbar_arrive(ptx::smem_u32(&sm.ifull[is]));
        }
        __syncwarp();
        ++items;
#pragma unroll
        for (int v = 0; v < 2; ++v) {
          if (it.wa[v] >= it.wb[v]) continue;
          if (qfills[v] && !wait(&sm.qempty[v], qfills[v] + 1)) break;
          ++qfills[v];
          if (lane == 0) {
            const uint32_t bar = ptx::smem_u32(&sm.qfull[v]);
            ptx::mbar_arrive_expect_tx(bar, kTile);
#pragma unroll
            for (int hh = 0; hh < D / 64; ++hh)
              tma_load_4d(ptx::smem_u32(sm.q[v]) + hh * kHalf, &qmap, 64 * hh, (int32_t)i0 + v * tokens, h * pr.G,
                          (int32_t)b, bar);
          }
          __syncwarp();
        }
        for (int j = it.ja; j < it.jb && ok; ++j) {
          const int at = (j - it.ja) & 15;
          if (at == 0) {
            if (j > it.ja) entry = look_up(j);
            if (entry == -2) {
              set_status(a.status, PISA_DEV_BAD_INDEX);
              *(volatile int32_t*)&sm.bad_page = 1;
            }
            __syncwarp();
          }
          const int32_t pg[2] = {__shfl_sync(0xffffffffu, entry, 2 * at), __shfl_sync(0xffffffffu, entry, 2 * at + 1)};
          const int pages = (pg[0] >= 0) + (pg[1] >= 0);
          // values that no row of the item sees (behind the sequence's end among
          // them) may be anything, and a weight of zero does not undo a NaN:
          // they are cleared before the MMA reads the tile
          const int32_t key0 = j * kKeys;
          const bool clear = key0 < klo || key0 + kKeys - 1 > khi || pages < 2;
#pragma unroll 1
          for (int kv = 0; kv < 2; ++kv) {
            if (fills >= kStages && !wait(&sm.empty[st], ph ^ 1)) break;  // the first round finds them empty
            if (lent == st && !take_back()) break;
            const uint32_t full = ptx::smem_u32(&sm.full[st]), dst = ptx::smem_u32(sm.kv[st]);
            const bool scrub = !Q8 && kv == 1 && (clear || clean);
            const uint32_t bar = Q8 ? ptx::smem_u32(&sm.raw[st]) : scrub ? ptx::smem_u32(&sm.scrub) : full;
            if (Q8 && lane == 0) {  // the converters do the rest
              sm.have[st] = (pg[0] >= 0 ? 1 : 0) | (pg[1] >= 0 ? 2 : 0);
              if (pages) ptx::mbar_arrive_expect_tx(bar, pages * kPage * (D + 1));
              else ptx::mbar_arrive(bar);
#pragma unroll
              for (int p = 0; p < 2; ++p) {
                if (pg[p] < 0) continue;
                const int32_t y = (int32_t)(((int64_t)pg[p] * pr.Hkv + h) * kPage);
                ptx::tma_load_2d(ptx::smem_u32(D == 64 ? sm.codes[D == 64 ? st : 0] : sm.kv[st] + kTile / 2) +
                                     p * (kPage * D),
                                 kv ? &vmap : &kmap, 0, y, bar);
                ptx::bulk_g2s(ptx::smem_u32(sm.scale[Q8 ? st : 0]) + p * kPage, (kv ? a.vs : a.ks) + y, kPage, bar);
              }
            } else if (!Q8 && lane == 0) {
              if (pages) ptx::mbar_arrive_expect_tx(bar, pages * (kTile / 2));
              else if (!scrub) ptx::mbar_arrive(bar);
#pragma unroll
              for (int p = 0; p < 2; ++p) {
                if (pg[p] < 0) continue;
                const int32_t y = (int32_t)(((int64_t)pg[p] * pr.Hkv + h) * kPage);
#pragma unroll
                for (int hh = 0; hh < D / 64; ++hh)
                  ptx::tma_load_2d(dst + hh * kHalf + p * kPageHalf, kv ? &vmap : &kmap, 64 * hh, y, bar);
              }
            }
            __syncwarp();
            if (scrub) {
              if (pages) {
                const bool got = ptx::mbar_wait_fast(bar, scrubs & 1, &sm.zero);
                ++scrubs;
                if (!(ok = __all_sync(0xffffffffu, got) != 0)) break;
              }
              for (int e = lane; e < kKeys * 8; e += 32) {
                const int rr = e >> 3;
                const int32_t key = key0 + rr;
                if (key < klo || key > khi || (rr < kPage ? pg[0] : pg[1]) < 0) {
#pragma unroll
                  for (int hh = 0; hh < D / 64; ++hh)
                    *reinterpret_cast<uint4*>(sm.kv[st] + hh * kHalf + rr * 128 + (e & 7) * 16) =
                        make_uint4(0, 0, 0, 0);
                }
              }
              if (clean) {
                __syncwarp();
                clean_tile<kTile>(sm.kv[st]);
              }
              ptx::fence_proxy_async_smem();
              __syncwarp();
              if (lane == 0) ptx::mbar_arrive(full);
            }
            advance();
          }
        }
        // one more stage, empty: the item's rows go out through it
        if (!take_back() || (fills >= kStages && !wait(&sm.empty[st], ph ^ 1))) break;
        lent = st;
        if (lane == 0) {
          ptx::mbar_arrive(ptx::smem_u32(&sm.lent));
          // nobody else sees it filled or releases it: rows_out says when it is free
          ptx::mbar_arrive(ptx::smem_u32(&sm.full[st]));
          if (Q8) {
            for (int k = 1; k < 4; ++k) ptx::mbar_arrive(ptx::smem_u32(&sm.full[st]));
            ptx::mbar_arrive(ptx::smem_u32(&sm.raw[st]));
          }
          ptx::mbar_arrive(ptx::smem_u32(&sm.empty[st]));
          ptx::mbar_arrive(ptx::smem_u32(&sm.empty[st]));
        }
        __syncwarp();
        advance();
        now = clean ? next : claim();
        clean = false;
      }
      if (ok && lane == 0) {  // (the slot is free: the last items have been waited for)
        sm.item[items % kItems].bh = -1;
        ptx::mbar_arrive(ptx::smem_u32(&sm.ifull[items % kItems]));
      }
      if (!ok && lane == 0) *abort = 1;
      // every issued load lands before the CTA can end, whoever gave up
      if (lane == 0) {
        for (int v = 0; v < 2; ++v)
          if (qfills[v]) ptx::mbar_wait_fast(ptx::smem_u32(&sm.qfull[v]), (qfills[v] - 1) & 1, &sm.zero);
        for (int f = max(0, fills - kStages); f < fills; ++f)
          ptx::mbar_wait_fast(ptx::smem_u32(Q8 ? &sm.raw[f % kStages] : &sm.full[f % kStages]), (f / kStages) & 1,
                              &sm.zero);
      }
      __syncwarp();
    } else if (warp < kLoadWarp) {
      // --------------------------------------------- the MMAs of row tile v
      // The tensor pipe takes few MMAs ahead and a wait on an mbarrier costs
      // some 300 cycles while the MMAs occupy shared memory, so each row tile
      // has a warp of its own: one waits while the other's MMAs run.  They
      // take turns (named barriers, which need no shared memory): a group -- O
      // of key tile j, then S of key tile j + 1 -- goes in whole, so that the
      // other tile's softmax runs beside it.  The softmax warps have seen V(j)
      // and K(j + 1) land before they hand over weights, so that only pfull is
      // waited for.  All lanes run the loop, and what it branches on is
      // broadcast, so that the descriptors stay in uniform registers (an MMA
      // then takes about 70 cycles to issue, not 100); one elected lane issues.
      const int v = warp - kMmaWarp;
      const uint32_t ut = __shfl_sync(0xffffffffu, tmem, 0);
      const uint32_t o = ut + 256 + v * D, sp = ut + v * 128, qb = ptx::smem_u32(sm.q[v]);
      bool ok = true;
      auto wait = [&](uint64_t* bar, int phase) {
        ok = ok && __all_sync(0xffffffffu, ptx::mbar_wait_fast(ptx::smem_u32(bar), phase & 1, abort)) != 0;
      };
      int st = 0, ph = 0;             // stage and phase of the next fill to release
      int tiles_done = 0, qfills = 0;  // key tiles of this row tile so far; query tiles
      for (int items = 0;; ++items) {
        const Item* ip = &sm.item[items % kItems];
        wait(&sm.ifull[items % kItems], items / kItems);
        // both warps go on, or neither: a turn is never waited for in vain
        if (!both_ok(ok)) break;
        if (__shfl_sync(0xffffffffu, ip->bh, 0) < 0) break;
        const int av = __shfl_sync(0xffffffffu, ip->wa[v], 0), bv = __shfl_sync(0xffffffffu, ip->wb[v], 0);
        const int uja = __shfl_sync(0xffffffffu, ip->ja, 0), ujb = __shfl_sync(0xffffffffu, ip->jb, 0);
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(&sm.iempty[items % kItems]));
        if (uja < ujb && av < bv) wait(&sm.qfull[v], qfills++);
        for (int j = uja - 1; j < ujb && uja < ujb; ++j) {
          const bool has_o = j >= av && j < bv, has_s = j + 1 >= av && j + 1 < bv;
          const int sv = st, pv = ph;  // V(j)
          if (j >= uja && ++st == kStages) { st = 0; ph ^= 1; }
          const int sk = st, pk = ph;  // K(j + 1)
          if (j + 1 < ujb && ++st == kStages) { st = 0; ph ^= 1; }
          const uint32_t vb = ptx::smem_u32(sm.kv[sv]), kb = ptx::smem_u32(sm.kv[sk]);
          if (!has_o || j == av) {  // (else a softmax warp has)
            if (j >= uja) wait(&sm.full[sv], pv);
            if (j + 1 < ujb) wait(&sm.full[sk], pk);
          }
          if (has_o) wait(&sm.pfull[v][0], tiles_done);
          if (v == 1 || j >= uja) turn_wait(v);
          if (has_o) {
            ptx::tc_fence_after();
            if (ok && elect_one()) {
#pragma unroll
              for (int k = 0; k < 4; ++k)
                mma_ts_bf16(o, sp + 8 * k, desc_mn_sw128(vb + k * 2048, kHalf), kIdescO, (j > av || k > 0) ? 1u : 0u);
            }
            wait(&sm.pfull[v][1], tiles_done);
            ptx::tc_fence_after();
            if (ok && elect_one()) {
#pragma unroll
              for (int k = 4; k < 8; ++k)
                mma_ts_bf16(o, sp + 8 * k, desc_mn_sw128(vb + k * 2048, kHalf), kIdescO, 1u);
            }
            ++tiles_done;
          }
          if (has_s && ok && elect_one()) {
            // over P of key tile j, which the MMAs above read: they run in order
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
              const uint32_t off = (k >> 2) * kHalf + (k & 3) * 32;
              ptx::mma_bf16(sp, ptx::desc_sw128(qb + off), ptx::desc_sw128(kb + off), kIdescS, k > 0 ? 1u : 0u);
            }
            ptx::mma_commit(ptx::smem_u32(&sm.sfull[v]));
          }
          __syncwarp();
          if (v == 0 || j + 1 < ujb) turn_pass(v);
          if (ok && elect_one()) {
            if (has_o && j + 1 == bv) ptx::mma_commit(ptx::smem_u32(&sm.odone[v]));
            if (has_s && j + 2 == bv) ptx::mma_commit(ptx::smem_u32(&sm.qempty[v]));
            if (j >= uja) ptx::mma_commit(ptx::smem_u32(&sm.empty[sv]));
            if (j + 1 < ujb) ptx::mma_commit(ptx::smem_u32(&sm.empty[sk]));
          }
          __syncwarp();
          if (!ok && lane == 0) *abort = 1;
        }
        if (++st == kStages) { st = 0; ph ^= 1; }  // the stage that the rows go out through
      }
      if (elect_one()) ptx::mma_commit(ptx::smem_u32(&sm.done[v]));
      __syncwarp();
      ptx::mbar_wait_fast(ptx::smem_u32(&sm.done[v]), 0, &sm.zero);
      __syncwarp();
    }
  } else {
    // ------------------------------------------------------------- softmax
    if constexpr (Q8) asm volatile("setmaxnreg.inc.sync.aligned.u32 " PISA_SOFTMAX_REGS_Q8 ";");
    else asm volatile("setmaxnreg.inc.sync.aligned.u32 " PISA_SOFTMAX_REGS ";");
    const int w = warp >> 2, r = threadIdx.x & 127;
    const uint32_t lane_base = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t s_at = lane_base + w * 128, o_at = lane_base + 256 + w * D;
    // MODE 0 keeps the dots and scales them inside the exponent
    const float sc = MODE == 0 ? pr.scale2 : 1.0f;
    const float slack = kSlack / sc;
    // A weight is 2^(s sc - m sc) by one FMA, with m sc rounded: a factor of the
    // whole row, unless |m sc| is so large (2^31) that it over- or underflows.
    // Scores beyond 2^28 lie 2^5 apart at least, so that their row takes the
    // power of two below sc: m sc is then exact, and as good as all of the
    // weight stays with the largest.
    const float pow2 = __uint_as_float(__float_as_uint(sc) & 0x7f800000u);
    bool ok = true;
    int tiles_done = 0, outs_done = 0;
    for (int items = 0;; ++items) {
      ok = ptx::mbar_wait_fast(ptx::smem_u32(&sm.ifull[items % kItems]), (items / kItems) & 1, abort);
      if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
      const Item* ip = &sm.item[items % kItems];
      if (ip->bh < 0) break;
      const int wa = ip->wa[w], wb = ip->wb[w], jb = ip->jb;
      // this thread's row and the keys that it sees; rows behind the new
      // tokens are computed as if they saw all, and not written
      int32_t lo = 0, hi = 0x7fffffff, t;
      float slope = 0.0f, lim = INFINITY;  // such a row has no say in the form of the cap
      {
        const int32_t b = (uint32_t)ip->bh / (uint32_t)pr.Hkv;
        const int32_t i = ip->tile * 2 * tokens + w * tokens + (r & (tokens - 1));
        t = ip->len - ip->cnt + i;
        if (i < ip->cnt && ip->fits) {
          int64_t l, u;
          key_span(mk, b, a.n, i, t, ip->len, &l, &u);
          lo = l <= u ? (int32_t)l : 0x7fffffff;
          hi = l <= u ? (int32_t)u : -1;
          lim = mk.by == 1.0f ? mk.lim : -1.0f;
        }
        if (MODE == 1 && mk.slopes)
          slope = mk.slopes[(ip->bh - b * pr.Hkv) * pr.G + (r >> a.lg_tokens)] * kLog2e;
      }
      const int f0 = ip->fill + 2 * (wa - ip->ja) + 3;  // the fill of the second V
      float m = -INFINITY, l = 0.0f, by = sc;
      int st = f0 % kStages, ph = (f0 / kStages) & 1;
      for (int j = wa; j < wb; ++j) {
        ok = true;
        if ((warp & 3) == 0 && j > wa) {
          // for the MMA warp: V(j) and K(j + 1) are there (as a rule they are by
          // now).  Not at an item's first tile: this warp has not followed the
          // ring up to it, and could take a phase for the one two fills earlier.
          ok = ptx::mbar_wait_fast(ptx::smem_u32(&sm.full[st]), ph, abort);
          if (++st == kStages) { st = 0; ph ^= 1; }
          if (j + 1 < jb) ok = ok && ptx::mbar_wait_fast(ptx::smem_u32(&sm.full[st]), ph, abort);
          if (++st == kStages) { st = 0; ph ^= 1; }
        }
        ok = ok && ptx::mbar_wait_fast(ptx::smem_u32(&sm.sfull[w]), tiles_done & 1, abort);
        if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
        ptx::tc_fence_after();
        float s[kKeys];
#pragma unroll
        for (int c = 0; c < kKeys; c += 32) ptx::tmem_ld32(s_at + c, *reinterpret_cast<uint32_t(*)[32]>(&s[c]));
        const int32_t key0 = j * kKeys;
        // keys clo .. chi of the tile are seen
        const int32_t clo = max(lo, key0) - key0, chi = min(hi, key0 + kKeys - 1) - key0;
        const bool bad = *(volatile int32_t*)&sm.bad_page != 0;
        const bool part = __any_sync(0xffffffffu, clo > 0 || chi < kKeys - 1) || bad;
        ptx::tmem_ld_wait();  // (all of the above in its shadow)
        bool late = false;  // the cap is applied on the way to the exponential
        if (MODE == 1) {
          if (mk.cap2 > 0.0f) {
            float big[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              big[k] = fmaxf(fabsf(s[32 * k]), fabsf(s[32 * k + 1]));
#pragma unroll
              for (int c = 2; c < 32; c += 2) big[k] = ptx::max3(big[k], fabsf(s[32 * k + c]), fabsf(s[32 * k + c + 1]));
            }
            // small scores: a polynomial on the FMA pipe, two at a time (the
            // exponential and the reciprocal of the other way take 12 cycles of
            // the SFU a warp, three times what the softmax takes itself).  What
            // stands at keys that are not seen may decide against it, and
            // changes no bit: a small score comes out the same both ways
            if (__all_sync(0xffffffffu, !(fmaxf(ptx::max3(big[0], big[1], big[2]), big[3]) > lim))) {
              late = !part && !mk.slopes;  // the cap is monotone: the largest score stays the largest
              if (!late) {
#pragma unroll
                for (int c = 0; c < kKeys; c += 2)
                  ptx::unpack2(mul2(ptx::pack2(s[c], s[c + 1]), cap_factor(mk, ptx::pack2(s[c], s[c + 1]))), s[c],
                               s[c + 1]);
              }
            } else {
              // cap_score(), two at a time: the small ones among them take the
              // polynomial too, since the other form's error is a part of the cap
              const uint64_t by2 = ptx::pack2(mk.by, mk.by);
              const float pre = mk.pre * (2.0f * kLog2e), cap = mk.cap2;
              auto large = [&](float x) { return fmaf(-2.0f * cap, rcp_approx(1.0f + ptx::ex2(x * pre)), cap); };
#pragma unroll
              for (int c = 0; c < kKeys; c += 2) {
                const uint64_t x2 = ptx::pack2(s[c], s[c + 1]);
                const uint64_t y2 = mul2(x2, by2);
                float a0, a1, y0, y1;
                ptx::unpack2(y2, y0, y1);
                ptx::unpack2(mul2(x2, cap_factor(mk, y2)), a0, a1);
                s[c] = within(y0, mk.lim, a0, large(s[c]));
                s[c + 1] = within(y1, mk.lim, a1, large(s[c + 1]));
              }
            }
          }
          if (mk.slopes) {
            // bias slope (j - t), j - t exact up to the fp32 product
            const float rel = (float)(int32_t)(key0 - t);
            const float by = mk.cap2 > 0.0f ? 1.0f : pr.scale2;
            const uint64_t by2 = ptx::pack2(by, by), slope2 = ptx::pack2(slope, slope), two = ptx::pack2(2.0f, 2.0f);
            uint64_t j2 = ptx::pack2(rel, rel + 1.0f);
#pragma unroll
            for (int c = 0; c < kKeys; c += 2) {
              ptx::unpack2(ptx::fma2(ptx::pack2(s[c], s[c + 1]), by2, mul2(slope2, j2)), s[c], s[c + 1]);
              j2 = ptx::add2(j2, two);
            }
          }
        }
        if (part) {
          // each side by itself: a tile rarely needs both
          if (__any_sync(0xffffffffu, clo > 0)) {
#pragma unroll
            for (int c = 0; c < kKeys; ++c)
              if (c < clo) s[c] = -INFINITY;
          }
          if (__any_sync(0xffffffffu, chi < kKeys - 1)) {
#pragma unroll
            for (int c = 0; c < kKeys; ++c)
              if (c > chi) s[c] = -INFINITY;
          }
        }
        if (bad) {
#pragma unroll
          for (int p = 0; p < 2; ++p) {
            const int64_t blk = 2 * (int64_t)j + p;
            if (blk * kPage > ip->khi) continue;
            const int32_t pg = a.table[(int64_t)((uint32_t)ip->bh / (uint32_t)pr.Hkv) * a.nb + blk];
            if (pg >= 0 && pg < a.num_pages) continue;
#pragma unroll
            for (int c = 0; c < kPage; ++c) s[p * kPage + c] = -INFINITY;
          }
        }
        float mx[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          mx[k] = fmaxf(s[32 * k], s[32 * k + 1]);
#pragma unroll
          for (int c = 2; c < 32; c += 2) mx[k] = ptx::max3(mx[k], s[32 * k + c], s[32 * k + c + 1]);
        }
        float top = fmaxf(ptx::max3(mx[0], mx[1], mx[2]), mx[3]);
        if (MODE == 1 && late) {
          float unused;
          ptx::unpack2(mul2(ptx::pack2(top, top), cap_factor(mk, ptx::pack2(top, top))), top, unused);
        }
        const bool grow = top > m + slack || (m == -INFINITY && top > -INFINITY);
        if (__any_sync(0xffffffffu, grow)) {
          const float f = grow && m > -INFINITY ? ptx::ex2((m - top) * sc) : 1.0f;
          if (grow) {
            m = top;
            if (MODE == 0) by = fabsf(top * sc) < 0x1p28f ? sc : pow2;
          }
          l *= f;
          if (j > wa && __any_sync(0xffffffffu, f != 1.0f)) {
            // the MMAs into O so far are done: S of this tile was issued after them
#pragma unroll 1
            for (int c = 0; c < D; c += 16) {
              uint32_t o[16];
              tmem_ld16(o_at + c, o);
              ptx::tmem_ld_wait();
#pragma unroll
              for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
              tmem_st16(o_at + c, o);
            }
          }
        }
        const float neg = m == -INFINITY ? 0.0f : -m * by;
        const uint64_t by2 = ptx::pack2(by, by), neg2 = ptx::pack2(neg, neg);
        uint64_t sum[2] = {0ull, 0ull};
        // weights of the row, 32 at a time, from the exponents of two scores
        auto weights = [&](auto exponents) {
#pragma unroll
          for (int c = 0; c < kKeys; c += 32) {
            uint32_t pk[16];
#pragma unroll
            for (int k = 0; k < 32; k += 2) {
              float p0, p1;
              ptx::unpack2(exponents(ptx::pack2(s[c + k], s[c + k + 1])), p0, p1);
              p0 = ptx::ex2(p0);
              p1 = ptx::ex2(p1);
              sum[(k >> 1) & 1] = ptx::add2(sum[(k >> 1) & 1], ptx::pack2(p0, p1));
              // P is rounded to bf16 for the MMA (2^-8 of each weight, the values' own step); l is not
              pk[k / 2] = pack_bf16(p0, p1);
            }
            tmem_st16(s_at + c / 2, pk);
            if (c & 32) {  // half of the weights: the MMAs may start on them
              tmem_st_wait();
              ptx::tc_fence_before();
              __syncwarp();
              if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(&sm.pfull[w][c >> 6]));
            }
          }
        };
        if (MODE == 1 && late) weights([&](uint64_t x2) { return ptx::fma2(x2, cap_factor(mk, x2), neg2); });
        else weights([&](uint64_t x2) { return ptx::fma2(x2, by2, neg2); });
        float s0, s1;
        ptx::unpack2(ptx::add2(sum[0], sum[1]), s0, s1);
        l += s0 + s1;
        ++tiles_done;
      }
      if (!ok) break;
      const bool any = wa < wb;
      if (any) {
        ok = ptx::mbar_wait_fast(ptx::smem_u32(&sm.odone[w]), outs_done & 1, abort);
        ++outs_done;
        if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
        ptx::tc_fence_after();
      }
      const int est = (ip->fill + 2 * (jb - ip->ja)) % kStages;  // the stage lent for the rows
      ok = ptx::mbar_wait_fast(ptx::smem_u32(&sm.lent), items & 1, abort);
      if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
      const int64_t b = (uint32_t)ip->bh / (uint32_t)pr.Hkv;
      const int32_t hq = (ip->bh - (int32_t)b * pr.Hkv) * pr.G + (r >> a.lg_tokens);
      const int32_t i = ip->tile * 2 * tokens + w * tokens + (r & (tokens - 1));
      const bool row = i < ip->cnt;
      const int64_t at =
          (((int64_t)ip->split * a.tiles + ip->tile) * heads + (uint32_t)ip->bh) * (2 * kRows) + w * kRows + r;
      // Rows go out through shared memory, a part of each at a time, so that
      // the stores cover whole lines (a row per thread would occupy the LSU,
      // and with it every barrier, for 4000 cycles).
      constexpr int kPart = D == 128 ? 128 : 64;  // bytes of a row at a time
      constexpr int kLines = kPart / 16;          // 16-byte pieces of that
      const uint32_t buf = ptx::smem_u32(sm.kv[est]) + w * (kTile / 2) + (warp & 3) * (32 * kPart);
      const int swz = kLines == 8 ? (lane & 7) : ((lane >> 1) & 3);
      auto pass = [&](const uint32_t (&x)[kPart / 4], char* dst) {
#pragma unroll
        for (int c = 0; c < kLines; ++c)
          asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(buf + lane * kPart + ((c ^ swz) << 4)),
                       "r"(x[4 * c]), "r"(x[4 * c + 1]), "r"(x[4 * c + 2]), "r"(x[4 * c + 3])
                       : "memory");
        __syncwarp();
        const int c = lane % kLines;
#pragma unroll
        for (int k = 0; k < kLines; ++k) {
          const int rr = (32 / kLines) * k + lane / kLines;
          const uint64_t dp = __shfl_sync(0xffffffffu, reinterpret_cast<uint64_t>(dst), rr);
          uint32_t a0, a1, a2, a3;
          asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                       : "=r"(a0), "=r"(a1), "=r"(a2), "=r"(a3)
                       : "r"(buf + rr * kPart + ((c ^ (kLines == 8 ? (rr & 7) : ((rr >> 1) & 3))) << 4))
                       : "memory");
          if (dp) reinterpret_cast<uint4*>(dp)[c] = make_uint4(a0, a1, a2, a3);
        }
        __syncwarp();
      };
      float finite = 0.0f;  // NaN once one of the row's outputs is not
      if (a.splits > 1) {
        // this part of the row: m in log2 units, l, and O as it is
        if (row) *reinterpret_cast<float2*>(a.part_ml + 2 * at) = make_float2(any ? m * sc : -INFINITY, any ? l : 0.0f);
        if (any) {
#pragma unroll 1
          for (int c = 0; c < D; c += kPart / 4) {
            uint32_t o[kPart / 4];
            if constexpr (kPart == 128) ptx::tmem_ld32(o_at + c, o);
            else tmem_ld16(o_at + c, o);
            ptx::tmem_ld_wait();
#pragma unroll
            for (int k = 0; k < kPart / 4; ++k) finite = fmaf(__uint_as_float(o[k]), 0.0f, finite);
            pass(o, row ? reinterpret_cast<char*>(a.part_o + at * D + c) : nullptr);
          }
        }
      } else {
        const float inv = 1.0f / l;
        const bool none = !any || l == 0.0f;
        char* dst = row ? reinterpret_cast<char*>(a.out + ((b * pr.Hq + hq) * a.n + i) * D) : nullptr;
#pragma unroll 1
        for (int c = 0; c < D; c += kPart / 2) {
          uint32_t pk[kPart / 4];
#pragma unroll
          for (int c2 = 0; c2 < kPart / 2; c2 += 32) {
            uint32_t o[32];
            if (any) {
              ptx::tmem_ld32(o_at + c + c2, o);
              ptx::tmem_ld_wait();
#pragma unroll
              for (int k = 0; k < 32; ++k) finite = fmaf(__uint_as_float(o[k]), 0.0f, finite);
            }
#pragma unroll
            for (int k = 0; k < 16; ++k)
              pk[c2 / 2 + k] =
                  none ? 0u : pack_bf16(__uint_as_float(o[2 * k]) * inv, __uint_as_float(o[2 * k + 1]) * inv);
          }
          pass(pk, dst ? dst + 2 * c : nullptr);
        }
      }
      if (ip->clean) {  // (a row of NaN scores is NaN already)
        Marks<D> marks = {};
        if constexpr (Q8) {
          if (sees_nan_row(a, pr.Hkv, ip->bh, wa, wb, lo, row ? hi : -1)) {
            for (int k = 0; k < D / 64; ++k)
              for (int e = 0; e < 2; ++e) marks.up[k][e] = marks.down[k][e] = 0xffffffffu;
          }
        } else {
          mark_tiles<D>(a, pr.Hkv, ip->bh, wa, wb, lo, row ? hi : -1, &marks);
        }
        set_marked<D>(a, row && any && l < INFINITY, ((b * pr.Hq + hq) * a.n + i) * D, at, &marks);
      } else if (__any_sync(0xffffffffu, row && finite != 0.0f)) {
        if (lane == 0) *(volatile int32_t*)&sm.again[items % kItems] = 1;
      }
      if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(&sm.iempty[items % kItems]));
      // the copy that fills the stage next comes after these accesses
      ptx::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(&sm.rows_out));
      ptx::tc_fence_before();  // the next item's weights, and so its first MMA into O, come after these reads
    }
    if (!ok) *abort = 1;
  }

  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  if (warp == kMmaWarp) ptx::tmem_dealloc(tmem, 512);
  if (threadIdx.x == 0 && sm.abort) set_status(a.status, PISA_DEV_TIMEOUT);
}

// The factor of x among values of weight f: an infinity keeps its own, where
// the weight came out as nothing too.
__device__ __forceinline__ float weight_of(float x, float f) { return fabsf(x) == INFINITY ? 1.0f : f; }

// Joins the parts of a row: one CTA per row, 8 dims x every 16th part a
// thread, so that all loads of a row are in flight at once.
template <int D>
__global__ void __launch_bounds__(D * 2, D == 128 ? 5 : 10) prefill_join_kernel(Prob pr, Args a) {
  constexpr int CH = D / 8, PL = 16;
  __shared__ float sm_m[PL], sm_l[PL];
  __shared__ float sm_o[PL][D];
  const int64_t rows = (int64_t)a.tiles * pr.B * pr.Hkv * (2 * kRows);
  const int64_t at = blockIdx.x;
  const int ch = threadIdx.x % CH, pl = threadIdx.x / CH;
  const int r = (int)(at & 127), w = (int)(at >> 7 & 1);
  const int64_t bh = (at >> 8) % (pr.B * pr.Hkv);
  const int64_t tile = (at >> 8) / (pr.B * pr.Hkv);
  const int64_t b = bh / pr.Hkv;
  const int tokens = 1 << a.lg_tokens;
  const int64_t i = tile * 2 * tokens + (int64_t)w * tokens + (r & (tokens - 1));
  int64_t len, cnt;
  new_span(a.seq_lens, a.new_lens, b, a.n, pr.N, &len, &cnt);
  // The lengths are the caller's, the parts the kernel's before.  A CTA without
  // a row need not wait for them, but the first one always does, so that this
  // grid, and what follows it in the stream, never ends before that kernel.
  if (i < cnt || at == 0) pdl_wait();
  if (i >= cnt) return;
  float M = -INFINITY, L = 0.0f, acc[8] = {};
  constexpr int kBatch = 2;
  for (int s0 = pl; s0 < a.splits; s0 += PL * kBatch) {
    float2 ml[kBatch];
    float4 o[kBatch][2];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      ml[k] = make_float2(-INFINITY, 0.0f);
      o[k][0] = o[k][1] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      if (s0 + PL * k < a.splits) {
        const int64_t p = (int64_t)(s0 + PL * k) * rows + at;
        ml[k] = *reinterpret_cast<const float2*>(a.part_ml + 2 * p);
        o[k][0] = *reinterpret_cast<const float4*>(a.part_o + p * D + 8 * ch);
        o[k][1] = *reinterpret_cast<const float4*>(a.part_o + p * D + 8 * ch + 4);
      }
    }
    float bm = M;
#pragma unroll
    for (int k = 0; k < kBatch; ++k) bm = fmaxf(bm, ml[k].x);
    if (bm > M) {
      const float f = M == -INFINITY ? 1.0f : ptx::ex2(M - bm);
      L *= f;
#pragma unroll
      for (int d = 0; d < 8; ++d) acc[d] *= weight_of(acc[d], f);
      M = bm;
    }
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      if (ml[k].y == 0.0f) continue;  // a part that saw no key wrote no output
      const float f = ml[k].x == -INFINITY ? 1.0f : ptx::ex2(ml[k].x - M);
      L = fmaf(ml[k].y, f, L);
      const float ov[8] = {o[k][0].x, o[k][0].y, o[k][0].z, o[k][0].w, o[k][1].x, o[k][1].y, o[k][1].z, o[k][1].w};
#pragma unroll
      for (int d = 0; d < 8; ++d) acc[d] = fmaf(ov[d], weight_of(ov[d], f), acc[d]);
    }
  }
  if (ch == 0) {
    sm_m[pl] = M;
    sm_l[pl] = L;
  }
#pragma unroll
  for (int d = 0; d < 8; ++d) sm_o[pl][8 * ch + d] = acc[d];
  __syncthreads();
  if (threadIdx.x >= D / 2) return;
  const int d = 2 * threadIdx.x;
  float top = -INFINITY, total = 0.0f, x = 0.0f, y = 0.0f;
#pragma unroll
  for (int k = 0; k < PL; ++k) top = fmaxf(top, sm_m[k]);
#pragma unroll
  for (int k = 0; k < PL; ++k) {
    if (sm_l[k] == 0.0f) continue;
    const float f = sm_m[k] == -INFINITY ? 1.0f : ptx::ex2(sm_m[k] - top);
    total = fmaf(sm_l[k], f, total);
    x = fmaf(sm_o[k][d], weight_of(sm_o[k][d], f), x);
    y = fmaf(sm_o[k][d + 1], weight_of(sm_o[k][d + 1], f), y);
  }
  const float inv = total == 0.0f ? 0.0f : 1.0f / total;
  const int64_t hq = (bh % pr.Hkv) * pr.G + (r >> a.lg_tokens);
  *reinterpret_cast<uint32_t*>(a.out + ((b * pr.Hq + hq) * a.n + i) * D + d) = pack_bf16(x * inv, y * inv);
}

// Grid of a call.  A GPU that has fewer CTAs than SMs gets the rows' keys
// split so that about one CTA per SM runs, each with four key tiles at least;
// the lengths are on the device, so the capacity stands for them.
constexpr int kSms = 152;
struct Plan {
  int32_t tiles, splits, lg_tokens;
  int64_t ctas;  // without the splits
  size_t ml, o, total;
};
void place_parts(const Prob& pr, int64_t parts, Plan* p) {  // of 256 rows each
  const size_t rows = (size_t)parts * 2 * kRows;
  size_t o = 256;
  p->ml = o; o = align_up(o + rows * 2 * 4, 256);
  p->o = o; o = align_up(o + rows * pr.d * 4, 256);
  p->total = o;
}
Plan make_plan(const Prob& pr, int64_t n) {
  Plan p;
  p.lg_tokens = pr.G == 1 ? 7 : (pr.G == 2 ? 6 : (pr.G == 4 ? 5 : 4));
  p.tiles = (int32_t)ceil_div64(n, (int64_t)2 << p.lg_tokens);
  p.ctas = p.tiles * pr.B * pr.Hkv;
  p.splits = 1;
  if (p.ctas > 0 && 2 * p.ctas <= kSms)
    p.splits = (int32_t)std::max<int64_t>(1, std::min(kSms / p.ctas, ceil_div64(pr.N, kKeys) / 4));
  place_parts(pr, p.splits > 1 ? p.splits * p.ctas : 0, &p);
  return p;
}

template <int D, int MODE, bool Q8>
cudaError_t launch_t(const Prob& pr, const MaskArgs& m, const Plan& pl, const CUtensorMap& qmap,
                     const CUtensorMap& kmap, const CUtensorMap& vmap, const Args& a, int num_sms, cudaStream_t st) {
  const size_t smem = sizeof(Smem<D, Q8>) + 1024;
  auto kern = paged_prefill_kernel<D, MODE, Q8>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  note_launch();
  e = launch_pdl(true, kern, dim3((unsigned)std::min<int64_t>(a.items, num_sms)), dim3(Cfg<D, Q8>::kThreads), smem,
                 st, pr, m,
                 qmap, kmap, vmap, a);
  if (e != cudaSuccess || pl.splits == 1) return e;
  note_launch();
  return launch_pdl(true, prefill_join_kernel<D>, dim3((unsigned)(pl.ctas * 2 * kRows)), dim3(D * 2), 0, st, pr, a);
}

}  // namespace

// What calls of up to n tokens need.  A call with fewer tokens may split its
// keys where one with more does not; splits x ctas is at most kSms, and at
// most the largest split times the most ctas that are split at all.
size_t paged_prefill_ws_bytes(const Prob& pr, int64_t n) {
  Plan p = make_plan(pr, n);
  const int64_t most = ceil_div64(pr.N, kKeys) / 4, heads = pr.B * pr.Hkv;
  const bool splits = p.ctas > 0 && 2 * heads <= kSms && most > 1;
  place_parts(pr, splits ? std::min<int64_t>(kSms, most * std::min<int64_t>(p.ctas, kSms / 2)) : 0, &p);
  return p.total;
}

// The bytes of e4m3 pages expanded to bf16 for calls of n tokens, and of the
// table of the expanded ones in front of them; 0: the call reads the codes
// itself.  Expanding moves the cache once (16384 positions of 4 heads 14 us),
// reading the codes costs every 256-row item about half its time again, since
// its converters share the shared memory's bandwidth with the MMAs.  Measured
// codes / expanded (us), one sequence behind 8192 (65536) cached tokens: 16 / 4
// heads of 128 with 5 items a key head 52 / 56 (196 / 189), with 8 73 / 72 (323 /
// 276), with 32 177 / 135 (1159 / 825); 32 / 8 heads of 64 with 8 86 / 87 (429 /
// 415), with 16 122 / 113 (807 / 732).  Without a cached part, which only the
// device knows of, it loses 5 to 9 us with few items: 16 / 4 heads of 128 with 8
// 21 / 26, with 16 64 / 70, with 32 46 / 45; 8 / 8 of 128 with 8 71 / 80, with 16
// 79 / 71; 32 / 8 of 64 with 16 25 / 31, with 32 38 / 43.  Not beyond 4 GiB.
size_t paged_prefill_scratch_bytes(const Prob& pr, int64_t n) {
  if (make_plan(pr, n).tiles < (pr.d == 128 ? 8 : 16) || pr.Hkv > 65535) return 0;  // (a grid's third dimension)
  const size_t pages = (size_t)pr.B * (size_t)ceil_div64(pr.N, kPage);
  const size_t total = align_up(pages * 4, 256) + pages * pr.Hkv * kPage * pr.d * 4;
  return total <= ((size_t)1 << 32) ? total : 0;
}

cudaError_t launch_paged_prefill(const Prob& pr, const MaskArgs& m, int64_t n, const void* q, const Pools& given,
                                 const int32_t* seq_lens, const int32_t* new_lens, char* ws, void* out,
                                 cudaStream_t st) {
  const Plan pl = make_plan(pr, n);
  Pools pools = given;
  const size_t scratch = pools.ks ? paged_prefill_scratch_bytes(pr, n) : 0;
  if (scratch > 0 && pools.scratch && pools.scratch_bytes >= scratch) {
    const int64_t pages = pr.B * pools.nb;
    char* at = (char*)pools.scratch + align_up((size_t)pages * 4, 256);
    Pools wide{at, at + (size_t)pages * pr.Hkv * kPage * pr.d * 2, (const int32_t*)pools.scratch, pages, pools.nb};
    const cudaError_t e = launch_expand_paged(pr, n, m.window, pools, wide, seq_lens, new_lens, st);
    if (e != cudaSuccess) return e;
    pools = wide;
  }
  CUtensorMap qmap, kmap, vmap;
  const int64_t rows = pools.num_pages * pr.Hkv * kPage;
  const bool in8 = pools.ks != nullptr;
  if (!(in8 ? make_tmap_codes : make_tmap_rows)(&kmap, pools.k, rows, pr.d, kPage) ||
      !(in8 ? make_tmap_codes : make_tmap_rows)(&vmap, pools.v, rows, pr.d, kPage) || !make_tmap_q(&qmap, q, pr.B, pr.Hq, n, pr.d, pr.G, 1 << pl.lg_tokens))
    return cudaErrorInvalidValue;
  cudaError_t e = launch_clear(ws, 256, st);
  if (e != cudaSuccess) return e;
  Args a{};
  a.n = n; a.nb = pools.nb; a.num_pages = pools.num_pages;
  a.q = (const uint16_t*)q; a.k = (const uint16_t*)pools.k; a.v = (const uint16_t*)pools.v;
  a.seq_lens = seq_lens; a.new_lens = new_lens; a.table = pools.table;
  a.ks = pools.ks; a.vs = pools.vs;
  a.status = (int32_t*)ws;
  a.claimed = (int32_t*)ws + 32;  // cleared with the status word
  a.out = (uint16_t*)out;
  a.part_ml = (float*)(ws + pl.ml);
  a.part_o = (float*)(ws + pl.o);
  a.items = (int32_t)(pl.ctas * pl.splits);
  int dev = 0;
  e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const int sms = sm_count(dev);
  if (sms < 1) return cudaErrorInvalidDevice;
  a.tiles = pl.tiles; a.splits = pl.splits; a.lg_tokens = pl.lg_tokens;
  const bool shaped = m.cap2 > 0.0f || m.slopes;  // scores that are more than scaled dots
  auto go = [&](auto dim) {
    constexpr int D = decltype(dim)::value;
    if (in8)
      return shaped ? launch_t<D, 1, true>(pr, m, pl, qmap, kmap, vmap, a, sms, st)
                    : launch_t<D, 0, true>(pr, m, pl, qmap, kmap, vmap, a, sms, st);
    return shaped ? launch_t<D, 1, false>(pr, m, pl, qmap, kmap, vmap, a, sms, st)
                  : launch_t<D, 0, false>(pr, m, pl, qmap, kmap, vmap, a, sms, st);
  };
  return pr.d == 128 ? go(std::integral_constant<int, 128>()) : go(std::integral_constant<int, 64>());
}

}  // namespace pisa
