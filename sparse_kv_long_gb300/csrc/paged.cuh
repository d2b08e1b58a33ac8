// paged.cuh -- attention of new tokens over a paged cache: a chunk of a
// prompt, a few drafted tokens or one token per request, causal, optionally
// through a sliding window with the first tokens kept visible.
//
// Token i of request b (n_b new tokens, T = lengths[b] in the cache, these
// included) stands at p = T - n_b + i and sees the keys t <= p that lie in the
// window (W == 0, or t > p - W) or among the first S:
//   out = sum_t softmax_t(scale q.k_t) v_t over the visible t; none: 0.
//
// One kernel on the tcgen05 tensor cores.  A query tile is 128 rows of one KV
// head per CTA, row = (token, query head of the group), so the group's heads
// share every K and V row read.  Keys come in tiles of KT; per tile
//   S = Q K^T   (M = 128 rows, N = KT, fp32 in tensor memory),
//   P = exp2(S scale log2e - m)  (one thread per row; bf16, written over S),
//   O += P V    (P from tensor memory, V from shared memory, fp32 in TMEM),
// with S double-buffered so that the softmax of one tile runs under the
// products of its neighbours.  m moves only when a row's maximum grows by
// more than 2^kLazy; then the row's O is rescaled.  P is bf16 because V is (or
// widens to it exactly) and a product takes one type; the row sum adds the
// weights as rounded, so that the weights applied sum to one.  What is left of
// that rounding (2^-9 of a weight, each on its own) takes the error against 64
// bits from the output's own (0.0017 of the values' size) to 0.0024.  What P
// leaves out as a second bf16 in a second product brings 0.0017, and was not
// taken for what it costs every kind of call: with shared prefixes, 8 single
// tokens behind 250000 int8 rows 143 us, then 162; 64 behind 131072 bf16 rows 102,
// 135; 80 drafts behind 60000 int8 rows 148, 173; 40 tokens behind five prefixes
// 57, 62 to 67; 5 chunks of 333 53, 57; 16 chunks of 256 behind 32768 1.26 ms, 1.78.
// Logits, O, m and the sums are fp32.
//
// What bounds it, and what it measured (bf16 product rate 1916 TFLOP/s, copy
// rate 6.79 TB/s):
//  - chunks of 256-dim bf16 rows: the products, and with calls back to back the
//    power limit.  2048 tokens at 65536 keys, 16 heads: 1.19 ms in bursts, 1.23
//    to 1.25 ms (1.7 PFLOP/s) held; 256 tokens at 262144 keys 0.58 and 0.66 to
//    0.67 ms.
//  - chunks of 128 dims: the softmax warps, whose chain per 128 keys (logits
//    from tensor memory, maximum, exponentials, weights back) takes 2.1 K clocks
//    against 1.0 K of products: 1.17 PFLOP/s; six prompts of up to 4096 tokens
//    247 us, 0.8 PFLOP/s with their masked tiles.
//  - int8 chunks: the same chain with scales and, beside it, the widening, which
//    every query tile does again for the keys it sees: the issue slots are 57 %
//    used.  4001 tokens in a window: 137 us.
//  - single tokens: reading the cache.  Four requests of 131072 tokens, bf16:
//    168 us, 94 % of the copy rate; 64 ragged int8 requests 115 us, 51 %: what
//    bounds them is the order of a tile's steps in the one CTA of an SM (copy,
//    widen, product, softmax), with no pipe full (issue 52 %, ALU 49 %, memory
//    44 %).  In a window of a thousand keys
//    (19.4 us) by what follows one another: launch, lengths, plan, table,
//    keys, two products, merge.
//
// Long prompts run as CTA pairs (cta_group::2, CTAS = 2): 256 query rows, 128
// keys a tile, each CTA holding half of the tile's keys (K) and half of its
// dims (V).  That halves the bytes that L2 has to hand to each SM: at M = 128
// a 256-dim tile needs 60 B per clock and SM, more than L2 gives.  Single
// tokens and drafts run as single CTAs with 64-key tiles; they are bound by
// reading the cache, and shared memory holds mostly the ring of K/V tiles.
//
// K and V tiles are 5-dimensional TMA boxes of whole pages (or the largest
// power-of-two part of one), laid out as [8-row group][64-column block][8 x
// 128 B], 128-byte swizzle: one box per page brings all dims.  int8 rows
// arrive in a staging ring and four warps (eight for few rows) widen them to
// bf16 (exact); the K scales multiply the logits, the V scales the weights.
//
// Work list: items (request, query tile, KV head), made on the device from the
// lengths.  Single CTAs share the batch's key tiles evenly; pairs cut items
// into pieces of about c tiles, c by the cost of a few candidates (see the
// plan).  Whole items write bf16 output, pieces write fp32 partials that
// merge_kernel joins in piece order.
//
// With prefixes that requests share (PRE; shared.cu) entries of the work list are
// groups over their prefixes, requests over their own keys, or requests over both;
// a piece's tiles up to nsink are then of a prefix.
#pragma once

#include <cuda.h>

#include "tc.cuh"
#include "worklist.cuh"

namespace skv {
namespace {

constexpr int kRows = 128;         // query rows per CTA (tensor-memory lanes)
constexpr int kMaxStages = 12;     // K/V ring
constexpr int kMaxStaging = 12;    // int8 staging ring
constexpr int kMaxPieces = 160;    // of an item; also the most CTAs of a launch
constexpr int kPieces = 4;         // piece descriptors in flight
constexpr int kTileInfo = 16;      // tiles whose page validity is kept (more than the ring holds)
constexpr int kScaleRing = 4;      // tiles whose int8 scales are kept
constexpr int kCand = 64;          // split candidates (pairs)
// Single CTAs.  Tiles that filling and draining a piece's pipeline is worth: 16
// drafts / 64 ragged requests took 64.8 / 133 us with 1, 52.5 / 128 with 3,
// 52.5 / 133 with 5, 52.0 / 139 with 8.  Tiles a CTA gets at least: eight tokens
// in a window of a thousand keys 19.5 us with 2 and 4, 22.7 with 8.
constexpr int kItem = 3;
constexpr int kMinStretch = 4;
// With prefixes, where each item's part counts less: eight agents behind 2000 tokens
// 17.3 us with 2, 18.5 with 4, 21.3 with 6.
constexpr int kMinShared = 2;
// The same for an item in the row of pairs with prefixes: 64 samples at 131072
// tokens took 131 us with 3, 100.7 with 5, 103.5 with 8, 112.7 with 12 (111 with all
// pieces dealt out).
constexpr int kRowItem = 5;
constexpr float kLazy = 8.f;       // log2 units a maximum may grow before O is rescaled
constexpr int kSplitPerPair = 8;   // pieces that write partials, per pair (single CTAs: two each)
constexpr uint32_t kGone = 0x7fc0dead;  // a NaN that no arithmetic gives
constexpr uint32_t kSCol = 256;    // tensor memory: O in [0, D), S/P buffers from here
constexpr int kMaxSmem = 227 * 1024;
constexpr int kOutBytes = 8 * 2048;

// Warp 0 copies, warp 1 issues products, warps 2 and 3 read int8 scales, two
// groups of four warps take the softmax of the two halves of a tile's keys,
// and for int8 rows four warps widen them.
template <bool INT8>
constexpr int kThreads = INT8 ? 512 : 384;
// Keys per tile.  Pairs: 128, what two logit buffers beside O leave room for at
// D = 256.  Single CTAs are bound by reading the cache, with 32 KB stages.
__host__ __device__ constexpr int keys_per_tile(int d, int ctas) { return ctas == 2 ? 128 : 64 * (256 / d); }

// Whether the tensor cores add up the rows' weights, as a product with ones
// beside O (int8 rows: with the reciprocals of the value scales, each as the
// sum of two bf16), where tensor memory has columns for it.  The additions and
// the unpacking of the rounded weights were a third of the softmax warps'
// exponential loop: 2048 tokens at 65536 keys of 128 dims took 289 us, now 257;
// int8 rows at 16384 keys 397, now 363, single tokens 129.7, now 127.2 (64
// requests, 256 dims).  Single bf16 tokens of 256 dims wait for memory and
// gained nothing (170.5 against 172), so theirs are added up by the warps.
__host__ __device__ constexpr bool row_sums(int d, int ctas, bool int8) { return d == 128 || (ctas == 1 && int8); }
// Their first column: beside O, or beside the 64 keys' logits of single CTAs.
__host__ __device__ constexpr uint32_t sum_col(int d) { return d == 128 ? 128 : kSCol + 64; }

constexpr int kDense = -2;
constexpr int kHasPrefix = 1 << 16;  // beside the number of a token's rows: it has a prefix, too

struct Piece {
  int tok0, toks;     // first token, tokens of the whole tile
  int pos0;           // position of the first token
  int b, h;           // request; with prefixes: -1 for a group's tokens over its prefix
  int lo, nsink;      // first window tile, sink tiles before it; with prefixes: the prefix's keys, its tiles before the request's
  int j0, n;          // this piece's tiles: j0 .. j0 + n of the item's list
  int slot;           // partial slot, -1: whole item, kDense: whole, but joined with its prefix or its own keys;
                      // with prefixes as slot_of and group_of read it: a field more cost the kernels without
                      // them registers (windowed int8 chunk 139.5 -> 141.5 us)
  int last;           // no piece follows
};

template <bool PRE>
struct Maps {
  CUtensorMap k, v, q;
};
template <>
struct Maps<true> {
  CUtensorMap k, v, q, q_own;  // queries of a group, of a request
};

struct alignas(16) Aux {
  uint64_t kv_full[kMaxStages], kv_empty[kMaxStages];
  // Two barriers where a waiter may skip tiles: when S(t + 1) is there, O of
  // t - 1 is done and of t may not be, and one parity could not tell them apart.
  uint64_t s_full[2], p_full[2], pv_done[2], q_full, q_free, mma_idle;
  uint64_t pc_full[kPieces], pc_empty[kPieces];
  Piece pc[kPieces];
  uint32_t tile_bad[kTileInfo];  // bit i: rows [8 i, 8 i + 8) of the tile have no page
  union {
    float2 cand[16];       // while planning: each warp's best cost and candidate
    float x[2][2][kRows];  // [exchange parity][group][row]: maxima of a tile, at a piece's end sums
  };
  int nmax, items;
  int rest;      // pairs, with prefixes: the row's length
  int disorder;  // some request's offsets descend or leave [0, n_tok]
  uint32_t tmem_base;
  alignas(16) uint16_t ones[256];  // 16 rows of 16 ones
  int dirty;  // a value that only some queries of a tile see was not finite
  int abort;
};

template <int KT>
struct alignas(16) Aux8 {  // int8 rows only
  uint64_t st_full[kMaxStaging], st_empty[kMaxStaging];
  uint64_t sc_full[kScaleRing], sc_empty[kScaleRing];
  alignas(16) float ks[kScaleRing][KT], vs[kScaleRing][KT];
  int wild[kScaleRing];  // a value scale of the tile is not finite
  union {  // 1 / vs
    float rs[kScaleRing][KT];
    // for the sums' products: of every eight keys eight rows of 16 bytes, row 0
    // the reciprocals as bf16, row 1 what is left of them, the others zero
    alignas(16) uint16_t rsum[kScaleRing][KT * 8];
  };
};

static_assert(kMaxStages == kMaxStaging && kScaleRing <= kPieces, "one thread sets up a barrier of each");
static_assert(sizeof(Aux) <= 4 * 1024, "room beside the query tile, the stages and the output rows");

// ---- work list -------------------------------------------------------------------

// Pairs, with prefixes: which stretch of the row each takes.  Dealing leaves some
// with a piece less; they come last and take as much more of the row, so that all end
// together, as far as it goes.  Stretches of less than kMinStretch go to fewer pairs.
struct Stretches {
  int n, o0, r;         // pairs; the first with a share; the first with a longer one
  int64_t short_, long_;  // shares, in 2^-16 tiles
  int total;
  __device__ __forceinline__ void plan(int units, int pieces, int tiles, int row) {
    const int rounds = (pieces + units - 1) / units;
    const int64_t a = pieces > 0 ? (static_cast<int64_t>(tiles) + static_cast<int64_t>(pieces) * kItem) * 65536 / pieces : 0;
    const int64_t w = static_cast<int64_t>(row) * 65536, least = static_cast<int64_t>(kMinStretch) * 65536;
    n = units;
    total = row;
    o0 = 0;
    r = pieces > 0 ? pieces - (rounds - 1) * units : units;
    const int64_t less = (units - r) * a;
    short_ = w > less ? (w - less) / units : 0;
    long_ = short_ + a;
    if (short_ < least && r < units) {
      o0 = r;
      long_ = w / (units - r);
    }
    if ((o0 == r && r < units ? long_ : short_) < least) {
      const int used = max(1, min(units, row / kMinStretch));
      o0 = r = units - used;
      long_ = w / used;
    }
  }
  __device__ __forceinline__ int begin(int o) const {
    if (o >= n) return total;
    const int64_t at = o <= o0 ? 0 : o <= r ? (o - o0) * short_ : max(r - o0, 0) * short_ + (o - max(r, o0)) * long_;
    return static_cast<int>(at >> 16);
  }
  __device__ __forceinline__ int owner(int at) const {
    const int64_t x = static_cast<int64_t>(at) * 65536, split = max(r - o0, 0) * short_;
    int o = x < split && short_ > 0 ? o0 + static_cast<int>(x / short_) : max(r, o0) + static_cast<int>((x - split) / max(long_, static_cast<int64_t>(1)));
    o = min(max(o, o0), n - 1);
    while (o + 1 < n && begin(o + 1) <= at) o++;
    while (o > o0 && begin(o) > at) o--;
    return o;
  }
};

__device__ __forceinline__ int pieces_of(int ntmax, int c) { return c > 0 && ntmax > c ? (ntmax + c - 1) / c : 1; }

// ---- helpers ---------------------------------------------------------------------

// Page of key t < 2^31; a general division would cost the copying warp as much as the copy's issue.
__device__ __forceinline__ int page_of(const PagedArgs& a, int t) {
  return static_cast<int>((__umulhi(a.page_mul, static_cast<uint32_t>(t)) + static_cast<uint32_t>(t)) >> a.page_shift);
}

template <int CTAS>
__device__ __forceinline__ uint32_t leader_addr(uint64_t* bar) {
  const uint32_t l = tc::smem_addr(bar);
  if (CTAS == 1) return l;
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(l));
  return r;
}

// Bounded wait for the phase of the given parity: gives up after kSpins looks
// (each sleeps for 230 to 2900 clocks, so half a second to six), or when
// another role has; sets *abort and returns false.  Half a dozen waits
// follow one another per tile, so this is as short as it can be: a clock in
// the loop, a call, or one lane asking for the warp each cost 5 to 20 % of a
// whole call.  Built with another SKV_PAGED_LOOKS (0: waits give up at once),
// the tests take the paths behind a wait that has given up.
#ifndef SKV_PAGED_LOOKS
#define SKV_PAGED_LOOKS 4000000
#endif
constexpr uint32_t kSpins = SKV_PAGED_LOOKS;
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, volatile int* abort) {
  if (tc::bar_test(bar, parity, false)) return true;
#pragma unroll 1
  for (uint32_t it = 0; it != kSpins; it++) {
    if (tc::bar_test(bar, parity, false)) return true;
    if ((it & 255) == 255 && *abort) return false;
  }
  *abort = 1;
  return false;
}

// One lane of a whole warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n.reg .pred p;\nelect.sync _|p, 0xffffffff;\nselp.u32 %0, 1, 0, p;\n}\n" : "=r"(r));
  return r != 0;
}

// A whole warp waits; false in every lane if one gave up.
__device__ __forceinline__ bool wait_all(uint64_t* bar, uint32_t parity, volatile int* abort) {
  return __all_sync(0xffffffffu, wait(bar, parity, abort));
}

// Arrive on the leader CTA's barrier.  Default (CTA) scope: what the leader's
// products read of this CTA is its own tensor and shared memory, ordered by
// the tcgen05 and proxy fences before the arrival; a release at cluster scope
// would wait here for every earlier access of the thread, each tile.
template <int CTAS>
__device__ __forceinline__ void arrive_leader(uint64_t* bar) {
  if (CTAS == 1)
    tc::bar_arrive(bar);
  else
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(leader_addr<CTAS>(bar))
                 : "memory");
}

// A box of the pool to this CTA's shared memory.
__device__ __forceinline__ void tma_rows(uint32_t dst, const CUtensorMap* map, int sub, int rg, int h, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(dst),
      "l"(map), "r"(0), "r"(0), "r"(sub), "r"(rg), "r"(h), "r"(tc::smem_addr(bar))
      : "memory");
}

// Shared-memory matrix descriptor (128-byte swizzle, as tc::sw128_desc) from
// its low word, which holds the address, and its constant high word.
__device__ __forceinline__ uint32_t desc_lo(uint32_t addr, uint32_t lbo) { return (addr >> 4) | ((lbo >> 4) << 16); }
__device__ __forceinline__ uint64_t desc(uint32_t lo, uint32_t sbo) {
  return (static_cast<uint64_t>((sbo >> 4) | (1u << 14) | (2u << 29)) << 32) | lo;
}

// One 64-column block of a query tile: rows (token, head of the group).
__device__ __forceinline__ void tma_query(uint32_t dst, const CUtensorMap* map, int head, int tok, int sub,
                                          uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
      "l"(map), "r"(0), "r"(head), "r"(tok), "r"(sub), "r"(tc::smem_addr(bar))
      : "memory");
}

__host__ __device__ constexpr uint32_t idesc_bf16(int M, int N, int b_mn) {
  return tc::idesc_f16(M, N, b_mn) | (1u << 7) | (1u << 10);  // A and B bf16
}

template <int CTAS>
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool acc) {
  if (CTAS == 1)
    asm volatile(
        "{\n.reg .pred p;\nsetp.ne.b32 p, %4, 0;\n"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(acc ? 1 : 0));
  else
    asm volatile(
        "{\n.reg .pred p;\nsetp.ne.b32 p, %4, 0;\n"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(acc ? 1 : 0));
}

template <int CTAS>
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool acc) {
  if (CTAS == 1)
    asm volatile(
        "{\n.reg .pred p;\nsetp.ne.b32 p, %4, 0;\n"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(acc ? 1 : 0));
  else
    asm volatile(
        "{\n.reg .pred p;\nsetp.ne.b32 p, %4, 0;\n"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(acc ? 1 : 0));
}

// Completion of this thread's earlier products, signalled on the barrier of every CTA of the pair.
template <int CTAS>
__device__ __forceinline__ void commit(uint64_t* bar) {
  if (CTAS == 1)
    asm volatile(
        "{\ntcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(tc::smem_addr(bar))
        : "memory");
  else
    asm volatile(
        "{\ntcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n}\n" ::"r"(
            tc::smem_addr(bar)),
        "h"(static_cast<uint16_t>(3))
        : "memory");
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
          taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]));
}


// Two columns of the warp's 32 rows.
__device__ __forceinline__ float2 tmem_ld2(uint32_t taddr) {
  float2 r;
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x2.b32 {%0, %1}, [%2];\ntcgen05.wait::ld.sync.aligned;"
               : "=f"(r.x), "=f"(r.y)
               : "r"(taddr)
               : "memory");
  return r;
}
__device__ __forceinline__ void tmem_st2(uint32_t taddr, float2 r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x2.b32 [%0], {%1, %2};" ::"r"(taddr), "f"(r.x), "f"(r.y) : "memory");
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// Two int8 codes (bytes 0 and 1, or 2 and 3, of x) -> two bf16, exact: a
// byte's low 7 bits under the exponent of 128 give 128 + low7, its sign bit
// there gives 128 or 256, and their difference is the code.
template <int HI>
__device__ __forceinline__ uint32_t int8_to_bf16x2(uint32_t x) {
  const uint32_t w = prmt(x, 0x43434343u, HI ? 0x4342u : 0x4140u);
  const uint32_t lo = w & 0xff7fff7fu, sg = w & 0xff80ff80u;
  const __nv_bfloat162 r =
      __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&lo), *reinterpret_cast<const __nv_bfloat162*>(&sg));
  return *reinterpret_cast<const uint32_t*>(&r);
}

// Copies and products take the K and V tiles of a piece in the order K0, K1,
// V0, K2, V1, ..., V(n-1); this is the place of V(j) in it.
__device__ __forceinline__ uint32_t fill_v(int j, int n) { return j + 1 < n ? 2u * j + 2u : 2u * n - 1u; }

struct Ring {  // a stage index and the parity of its current use
  int s = 0;
  uint32_t ph = 0;
  __device__ __forceinline__ void next(int depth) {
    if (++s == depth) {
      s = 0;
      ph ^= 1;
    }
  }
};

constexpr int kSlotBits = 12;
__device__ __forceinline__ int slot_and_group(int slot, int g) { return (slot - kDense) | g << kSlotBits; }
template <bool PRE>
__device__ __forceinline__ int slot_of(const Piece& pc) {
  return PRE ? (pc.slot & ((1 << kSlotBits) - 1)) + kDense : pc.slot;
}
__device__ __forceinline__ int group_of(const Piece& pc) { return pc.slot >> kSlotBits; }
static_assert(2 + (kSplitPerPair + 2) * kMaxPieces / 2 + 2 < 1 << kSlotBits && 2 + 2 * kMaxPieces + 2 < 1 << kSlotBits, "slots fit");

// Whether tile j of a piece is of a prefix, which every row sees all of.
template <bool PRE>
__device__ __forceinline__ bool of_prefix(const Piece& pc, int j) {
  return PRE && pc.j0 + j < pc.nsink;
}
// The last key of tile j's part that the row of position `pos` (of the request's own keys) sees.
template <bool PRE>
__device__ __forceinline__ int seen(const Piece& pc, int j, int pos) {
  return of_prefix<PRE>(pc, j) ? pc.lo - 1 : pos;
}
template <bool PRE>
__device__ __forceinline__ int last_seen(const Piece& pc, int j) {
  return seen<PRE>(pc, j, pc.pos0 + pc.toks - 1);
}
// Tile j's row of the block table, and its length.
template <bool PRE>
__device__ __forceinline__ const int32_t* pages_of(const PagedArgs& a, const Piece& pc, int j, int64_t& n) {
  if (of_prefix<PRE>(pc, j)) {
    n = a.n_prefix_pages;
    return a.prefix_table + group_of(pc) * n;
  }
  n = a.n_pages;
  return a.block_table + pc.b * n;
}

// Bits 0 .. n - 1.
__device__ __forceinline__ uint32_t bits_below(int n) {
  return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u;
}

// A warp writes 64 bytes of each lane's row: through shared memory, so that a
// store covers eight rows of 64 consecutive bytes (32 rows of 16 bytes take
// the store unit 32 lines each, and ran 3 to 7 K clocks per piece).  Lane i
// stores piece i % 4 of rows i / 4 + 8 k, at to[k] (null: no such row).
__device__ __forceinline__ void put_rows(unsigned char* buf, int lane, const uint32_t (&w)[16], char* const (&to)[4],
                                         int at) {
#pragma unroll
  for (int c = 0; c < 4; c++)
    *reinterpret_cast<uint4*>(buf + lane * 64 + ((c ^ ((lane >> 1) & 3)) << 4)) =
        make_uint4(w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]);
  __syncwarp();
  uint4 v[4];
#pragma unroll
  for (int k = 0; k < 4; k++) {
    const int row = 8 * k + (lane >> 2), c = lane & 3;
    v[k] = *reinterpret_cast<const uint4*>(buf + row * 64 + ((c ^ ((row >> 1) & 3)) << 4));
  }
#pragma unroll
  for (int k = 0; k < 4; k++)
    if (to[k]) *reinterpret_cast<uint4*>(to[k] + at) = v[k];
  __syncwarp();
}

// Key tile j of a piece.
template <bool PRE>
__device__ __forceinline__ int tile_of(const Piece& pc, int j) {
  j += pc.j0;
  return j < pc.nsink ? j : (PRE ? 0 : pc.lo) + j - pc.nsink;
}

// A lane's box of tile j of a piece (lanes past the tile's boxes: none).
struct Box {
  int rg;     // its first 8-row group in the pool; -1: no such page
  bool want;  // some query of the piece sees a key of it
};
struct BoxLoad {  // the table entry in flight
  int blk, t, pg;
};
template <int KT, bool PRE>
__device__ __forceinline__ BoxLoad box_load(const PagedArgs& a, const Piece& pc, int j, int lane) {
  BoxLoad x{-1, 0, 0};
  if (j < pc.n && lane * a.rb < KT) {
    x.t = tile_of<PRE>(pc, j) * KT + lane * a.rb;
    x.pg = page_of(a, x.t);
    int64_t n_pages;
    const int32_t* pages = pages_of<PRE>(a, pc, j, n_pages);
    if (x.pg < n_pages) x.blk = pages[x.pg];
  }
  return x;
}
template <int KT>
__device__ __forceinline__ Box box_of(const PagedArgs& a, const Piece& pc, const BoxLoad& x, int p_hi, int lane) {
  Box r;
  r.want = lane * a.rb < KT && x.t <= p_hi && (a.W == 0 || x.t + a.rb - 1 > pc.pos0 - a.W || x.t < a.S);
  r.rg = x.blk >= 0 && x.blk < a.n_blocks ? x.blk * (a.page >> 3) + ((x.t - x.pg * a.page) >> 3) : -1;
  return r;
}

// Values that are not finite were zeroed in the tiles that only some queries
// of the query tile see; this adds up those in columns [c0, c0 + 32) that a
// query at position p sees.
template <int D, int KT, bool PRE>
__device__ __noinline__ void add_nonfinite(const PagedArgs& a, const Piece& pc, int p, int p_last, int c0,
                                           float (&sum)[32]) {
#pragma unroll 1
  for (int j = 0; j < pc.n; j++) {
    int64_t n_pages;
    const int32_t* pages = pages_of<PRE>(a, pc, j, n_pages);
    const int t0 = tile_of<PRE>(pc, j) * KT, last = seen<PRE>(pc, j, p);
    bool masked = t0 + KT - 1 > seen<PRE>(pc, j, pc.pos0) || (a.W > 0 && t0 <= p_last - a.W && t0 + KT > a.S);
#pragma unroll 1
    for (int x = 0; x < KT && !masked; x += 8) {  // or a row without a page
      const int pg = page_of(a, t0 + x);
      const int blk = pg < n_pages ? pages[pg] : -1;
      masked = blk < 0 || blk >= a.n_blocks;
    }
    if (!masked) continue;  // every query sees the whole tile: its values went through the products as they are
#pragma unroll 1
    for (int x = 0; x < KT; x++) {
      const int key = t0 + x;
      if (key > last || !(a.W == 0 || key > p - a.W || key < a.S)) continue;
      const int pg = page_of(a, key);
      const int blk = pg < n_pages ? pages[pg] : -1;
      if (blk < 0 || blk >= a.n_blocks) continue;
      const uint16_t* v = a.v_pool + ((static_cast<int64_t>(blk) * a.page + (key - pg * a.page)) * a.Hkv + pc.h) * D + c0;
#pragma unroll 1
      for (int i = 0; i < 32; i++)
        if ((v[i] & 0x7f80u) == 0x7f80u)
          sum[i] += bf16_bits_to_f32(v[i]);
    }
  }
}

// PRE: with prefixes that requests share.
template <int D, int CTAS, bool INT8, bool PRE>
__global__ void __launch_bounds__(kThreads<INT8>, 1)
    paged_kernel(const __grid_constant__ Maps<PRE> maps, const PagedArgs a) {
  using Req = ReqOf<PRE>;
  const CUtensorMap &k_map = maps.k, &v_map = maps.v, &q_map = maps.q;
  const int n_req = PRE ? a.n_groups + a.B : a.B;
  constexpr int KT = keys_per_tile(D, CTAS);
  constexpr int KR = KT / CTAS;          // of them, this CTA's rows of K
  constexpr int NSUB = D / 64;           // 64-column blocks of a row
  constexpr int VSUB = NSUB / CTAS;      // those of this CTA's part of V
  constexpr int STAGE = KR * D * 2;      // bytes of a K or V stage (this CTA's part)
  constexpr int THREADS = kThreads<INT8>;
  constexpr bool SUM = row_sums(D, CTAS, INT8);
  constexpr uint32_t LCOL = sum_col(D);
  constexpr uint32_t SBO_K = NSUB * 1024, SBO_V = VSUB * 1024;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* sQ = smem_raw;  // 1024-byte aligned, as the swizzled tiles need (checked below)
  unsigned char* sKV = sQ + a.q_bytes;
  unsigned char* sI8 = sKV + a.stages * STAGE;
  unsigned char* sOut = sI8 + (INT8 ? a.staging * (STAGE / 2) : 0);  // 2 KB per softmax warp
  Aux* ax = reinterpret_cast<Aux*>(sOut + kOutBytes);
  Aux8<KT>* a8 = reinterpret_cast<Aux8<KT>*>(ax + 1);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = CTAS == 1 ? 0u : tc::cluster_rank();
  // Softmax warps and widening warps: with at most 32 rows a tile, as single
  // tokens have, warps 4 and 8 do the softmax and 5, 6, 7, 11 join the widening (9 and
  // 10 rest: at most two widen per scheduler that has other work).  64 ragged
  // requests took 190 us with four widening warps, 166 with these eight.  With
  // prefixes also at most 64 rows: 4, 5, 8 and 9, and 6, 7, 10 and 11.
  const bool thin = INT8 && CTAS == 1 && a.thin;
  const bool half = PRE && thin && a.thin == 2;
  const uint32_t n_soft = half ? 4 : thin ? 2 : 8, n_wide = thin ? 8 : 4;
  const bool softer = warp >= 4 && warp < 12 && (!thin || (warp & 3) <= (half ? 1 : 0));
  const int unit = blockIdx.x / CTAS, n_units = gridDim.x / CTAS;
  volatile int* abort = &ax->abort;

  allow_dependent_launch();  // the merge may be scheduled as SMs come free; it waits for this grid
  if (tid < kMaxStages) {  // a thread per barrier: one after the other they took a microsecond
    // int8: the widening warps of both CTAs; bf16: the copies, and on the leader a note from the peer's
    tc::bar_init(&ax->kv_full[tid], INT8 ? n_wide * CTAS : (rank == 0 ? CTAS : 1));
    tc::bar_init(&ax->kv_empty[tid], 1);
    if (INT8) {
      tc::bar_init(&a8->st_full[tid], 1);
      tc::bar_init(&a8->st_empty[tid], n_wide);
    }
  } else if (tid >= 32 && tid < 34) {
    tc::bar_init(&ax->s_full[tid - 32], 1);
    tc::bar_init(&ax->p_full[tid - 32], n_soft * CTAS);
    tc::bar_init(&ax->pv_done[tid - 32], 1);
  } else if (tid >= 64 && tid < 64 + kPieces) {
    tc::bar_init(&ax->pc_full[tid - 64], 1);
    tc::bar_init(&ax->pc_empty[tid - 64], 1 + n_soft + (INT8 ? 2 + n_wide : 0));  // products, softmax, scales, widening
    if (INT8 && tid - 64 < kScaleRing) {
      tc::bar_init(&a8->sc_full[tid - 64], 1);
      tc::bar_init(&a8->sc_empty[tid - 64], n_soft + (SUM ? 1 : 0));  // softmax, the sums' products
    }
  } else if (tid == 96) {
    tc::bar_init(&ax->q_full, rank == 0 ? CTAS : 1);  // the copy, and on the leader a note from the peer's
    tc::bar_init(&ax->q_free, 1);
    tc::bar_init(&ax->mma_idle, 1);
    ax->abort = (tc::smem_addr(smem_raw) & 1023u) != 0;  // every wait would give up at once
    ax->dirty = 0;
    ax->disorder = 0;
    ax->nmax = 0;
    ax->items = 0;
    ax->rest = 0;
  }
  if (SUM) {
    if (INT8) {
      for (int i = tid; i < kScaleRing * KT; i += THREADS)
        *reinterpret_cast<uint4*>(&a8->rsum[0][8 * i]) = make_uint4(0u, 0u, 0u, 0u);
    } else {
      for (int i = tid; i < 256; i += THREADS) ax->ones[i] = 0x3f80u;  // 1
    }
    tc::fence_async_smem();
  }
  if (tid < 128) asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  if (warp == 1) {
    if (CTAS == 1) {
      tc::tmem_alloc<512>(&ax->tmem_base);
    } else {
      asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(
          tc::smem_addr(&ax->tmem_base)));
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
    }
  }
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  // Launched early, too: barriers and tensor memory are set up while the
  // previous kernel ends (eight tokens in a window 19.5 -> 19.2 us); from here on
  // what it wrote is there.
  grid_dependency_wait();

  // ---- plan ------------------------------------------------------------------------
  // Single CTAs: the items' key tiles, each item preceded by kItem tiles' worth
  // of filling and draining its pipeline, lie in one row and every CTA takes an
  // equal stretch of it, whatever the requests' lengths (64 ragged requests: the
  // busiest CTA had 2.2 times the idlest's work when whole pieces were dealt
  // out).  An item's stretches are its pieces; a CTA has at most two that are
  // not whole, its first and its last.  Fewer CTAs when a stretch would be
  // shorter than kMinStretch.
  //
  // Pairs: queries of one request read the same keys, and those that run at the
  // same time should be at the same place, so pieces are equal cuts of items
  // instead.  Candidate k cuts the longest item into k pieces of c = ceil(nmax /
  // k) tiles and every other one into ceil(tiles / c): all items, or those past
  // the last full round over the pairs.  Its cost is the number of rounds times
  // a piece (the last at full length); a piece pays kOvh tiles for filling and
  // draining its pipeline, a split kJoin tiles once and part_cost per piece
  // for its partials.  Each warp weighs every NW-th candidate, a lane per
  // request; the batch waits in shared memory that the ring will take over.
  int split_c = 1, split_from = 0;
  int total = 0, n_used = n_units;  // single CTAs: the row's length, the CTAs that share it
  Stretches row;                    // pairs, with prefixes (warp 0)
  int n_dealt = 0;
  Req mine;                         // warp 0: the first 32 requests
  mine.start = mine.nq = mine.T = mine.nqt = mine.ntmax = 0;
  auto again = [&]() {  // offsets out of order: the batch is gone through again, without the requests that overlap
    __syncthreads();
    if (tid == 0) ax->nmax = ax->items = ax->rest = 0;
    __syncthreads();
  };
  if (CTAS == 1) {
#pragma unroll 1
    for (bool known = false;; known = true) {
      int sum = 0, rows = 0;
#pragma unroll 1
      for (int b = tid; b < n_req; b += THREADS) {
        const Req r = request_of<KT, PRE>(a, b, unit == 0, &ax->disorder, known);
        if (b < 32) mine = r;
        sum += r.nqt * a.Hkv * (r.ntmax + kItem);
        rows = max(rows, min(a.tpt, r.nq) * a.G);
      }
      if (warp * 32 < n_req) {
        sum = __reduce_add_sync(0xffffffffu, sum);
        rows = __reduce_max_sync(0xffffffffu, rows);
        if (lane == 0 && sum > 0) {
          atomicAdd(&ax->items, sum);
          atomicMax(&ax->nmax, rows);
        }
      }
      __syncthreads();
      if ((!PRE && !a.q_start) || known || !ax->disorder) break;
      again();
    }
    total = ax->items;
    n_used = min(n_units, max(1, total / (PRE ? kMinShared : kMinStretch)));
    if (!PRE && tid == 0 && unit == 0) {
      a.ws_head[0] = n_units;
      a.ws_head[1] = ax->nmax;
      a.ws_head[2] = 1;
    }
  } else {
    constexpr float kOvh = 3.f, kJoin = 3.f;
    constexpr int NW = THREADS / 32;
    int2* req = reinterpret_cast<int2*>(sKV);  // (query tiles, key tiles of the longest)
#pragma unroll 1
    for (bool known = false;; known = true) {
      int longest = 0, tiles = 0, in_row = 0;
#pragma unroll 1
      for (int b = tid; b < n_req; b += THREADS) {
        const Req r = request_of<KT, PRE>(a, b, unit == 0 && rank == 0, &ax->disorder, known);
        if (b < 32) mine = r;
        if (PRE && !dealt(r)) {
          req[b] = make_int2(0, 0);
          in_row += r.nqt * a.Hkv * (r.ntmax + kRowItem);
          continue;
        }
        req[b] = make_int2(r.nqt, r.ntmax);
        longest = max(longest, r.ntmax);
        tiles += r.nqt;
      }
      if (warp * 32 < n_req) {
        longest = __reduce_max_sync(0xffffffffu, longest);
        tiles = __reduce_add_sync(0xffffffffu, tiles);
        if (PRE) in_row = __reduce_add_sync(0xffffffffu, in_row);
        if (PRE && lane == 0 && in_row > 0) atomicAdd(&ax->rest, in_row);
        if (lane == 0 && tiles > 0) {
          atomicMax(&ax->nmax, longest);
          atomicAdd(&ax->items, tiles);
        }
      }
      __syncthreads();
      if ((!PRE && !a.q_start) || known || !ax->disorder) break;
      again();
    }
    const int nmax = ax->nmax, items = ax->items * a.Hkv;
    // Items kept whole in the second half of the candidates: the full rounds,
    // in the work list's order; only a batch that one warp holds is looked at
    // this way.
    const int x1 = !PRE && n_req <= 32 && items > n_units ? items / n_units * n_units : 0;
    const int nk = min(nmax, n_req > 512 ? 8 : PRE ? n_units : kCand);
    float best = 3e38f;
    int pick = 0;
#pragma unroll 1
    for (int i = warp; i < nk * (x1 > 0 ? 2 : 1); i += NW) {
      const bool rest = i >= nk;
      const int k = rest ? i - nk + 1 : i + 1;
      const int c = (nmax + k - 1) / k;
      const float rc = 1.f / c;
      int P = 0, S = 0, u = 0, main_u = 0;  // pieces, those of cut items, tiles of the items looked at, of the others
      int PL = 0, uL = 0;                   // with prefixes: long pieces, their tiles
#pragma unroll 1
      for (int b0 = 0; b0 < n_req; b0 += 32) {
        const int2 r = b0 + lane < n_req ? req[b0 + lane] : make_int2(0, 0);
        const int all = r.x * a.Hkv;
        int n = all;  // items that may be cut
        if (rest) {
          int sum = all;
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, sum, o);
            if (lane >= o) sum += y;
          }
          n = max(0, sum - max(sum - all, x1));
        }
        // ceil(tiles / c): the quotient is half a c-th away from every integer, its error below 65 * 2^-23
        const int ps = nmax < (1 << 15) ? max(1, static_cast<int>((r.y + c - 0.5f) * rc)) : pieces_of(r.y, c);
        P += n * ps;
        S += ps > 1 ? n * ps : 0;
        u += n * r.y;
        main_u += (all - n) * r.y;
        if (PRE && 2 * r.y >= c) {
          PL += n * ps;
          uL += n * r.y;
        }
      }
      P = __reduce_add_sync(0xffffffffu, P);
      S = __reduce_add_sync(0xffffffffu, S);
      u = __reduce_add_sync(0xffffffffu, u);
      if (rest) main_u = __reduce_add_sync(0xffffffffu, main_u);
      if (S <= (PRE ? kSplitPerPair * n_units : a.max_split)) {
        float cost = rest ? static_cast<float>(main_u) / n_units + x1 / n_units * kOvh : 0.f;
        if (PRE) {
          // Long pieces and short ones are dealt out in rounds of their own; the row evens
          // out what these leave, as far as it goes.
          PL = __reduce_add_sync(0xffffffffu, PL);
          uL = __reduce_add_sync(0xffffffffu, uL);
          const int rounds = (P + n_units - 1) / n_units, long_rounds = (PL + n_units - 1) / n_units;
          if (PL > 0) cost = long_rounds * (static_cast<float>(uL) / PL + kOvh);
          if (rounds > long_rounds) cost += (rounds - long_rounds) * (static_cast<float>(u - uL) / (P - PL) + kOvh);
          cost = fmaxf(cost, (u + P * kOvh + ax->rest) / n_units) + (S > 0 ? kJoin + S * a.part_cost : 0.f);
        } else if (P > 0)
          cost += static_cast<float>((P - 1) / n_units) * (static_cast<float>(u) / P + kOvh) + c + kOvh +
                  (S > 0 ? kJoin + S * a.part_cost : 0.f);
        if (cost < best) {
          best = cost;
          pick = i;
        }
      }
    }
    if (lane == 0) ax->cand[warp] = make_float2(best, __int_as_float(pick));
    __syncthreads();
    {
      const float2 o = ax->cand[min(lane, NW - 1)];
      best = o.x;
      pick = __float_as_int(o.y);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      const float ob = __shfl_xor_sync(0xffffffffu, best, o);
      const int oi = __shfl_xor_sync(0xffffffffu, pick, o);
      if (ob < best || (ob == best && oi < pick)) {
        best = ob;
        pick = oi;
      }
    }
    split_from = pick >= nk && nk > 0 ? x1 : 0;
    const int k = pick >= nk && nk > 0 ? pick - nk + 1 : pick + 1;
    split_c = max(1, (nmax + k - 1) / k);
    if (PRE && warp == 0) {
      int P = 0, u = 0;
#pragma unroll 1
      for (int b0 = 0; b0 < n_req; b0 += 32) {
        const int2 r = b0 + lane < n_req ? req[b0 + lane] : make_int2(0, 0);
        P += r.x * a.Hkv * pieces_of(r.y, split_c);
        u += r.x * a.Hkv * r.y;
      }
      row.plan(n_units, __reduce_add_sync(0xffffffffu, P), __reduce_add_sync(0xffffffffu, u), ax->rest);
      n_dealt = __reduce_add_sync(0xffffffffu, P);
    }
    tc::fence_async_smem();  // the copies write where the batch was
    tc::cluster_sync();  // also: the peer's barriers exist before any remote access
  }
  const int c = split_c, whole = split_from;  // tiles per piece; items before this one are not cut
  if (tid == 0 && ax->tmem_base != 0) *abort = 1;
  if (PRE && tid == 0 && unit == 0 && rank == 0) a.ws_head[0] = ax->disorder;  // the merge then writes nothing
  // All 512 columns are this CTA's, so they start at 0: a constant keeps the
  // products' addresses out of registers.
  constexpr uint32_t tm = 0;

  if (warp == 0) {
    // ---------------- pieces and copies ----------------
    // The requests are walked 32 at a time, a lane each.  Pairs: request b's
    // pieces are first those of its items that are kept whole, then the cut
    // items'.  Single CTAs: `pp` is the requests' length in the row.
    int b32 = 0, base = 0, ibase = 0, sbase = 0, seen = 0;  // first request of the window; pieces, split items, slots, items before it
    Req r = mine;
    int pp, ii = 0, ss = 0, tt = 0, ns = 1, nw = 0;  // inclusive sums over the window's requests; pieces per cut item, items kept whole
    constexpr int OVH = CTAS == 1 ? kItem : kRowItem;
    bool stretch = CTAS == 1;  // walking the row; pairs, with prefixes: once the pieces are dealt out
    auto scan = [&]() {
      const int items = !PRE || CTAS == 1 || dealt(r) != stretch ? r.nqt * a.Hkv : 0;
      if (stretch) {
        ii = ss = tt = 0;
        pp = items * (r.ntmax + OVH);
      } else {
        ns = pieces_of(r.ntmax, c);
        tt = items;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int x = __shfl_up_sync(0xffffffffu, tt, o);
          if (lane >= o) tt += x;
        }
        nw = min(items, max(0, whole - (seen + tt - items)));
        if (ns == 1) nw = items;
        pp = nw + (items - nw) * ns;
        ii = items - nw;
        ss = ii * ns;
      }
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, pp, o), y = CTAS == 1 ? 0 : __shfl_up_sync(0xffffffffu, ii, o),
                  z = CTAS == 1 ? 0 : __shfl_up_sync(0xffffffffu, ss, o);
        if (lane >= o) {
          pp += x;
          ii += y;
          ss += z;
        }
      }
    };
    scan();
    // single CTAs: this one's stretch, and the CTA that has a place of the row; of
    // pairs with prefixes, their places in the order of shares
    int x = 0, x_end = 0, me = unit, slots = 0;  // slots: before the row's
    bool listed = false;  // a split item begins here
    if (CTAS == 1 && unit < n_used) {
      x = static_cast<int>(static_cast<int64_t>(total) * unit / n_used);
      x_end = static_cast<int>(static_cast<int64_t>(total) * (unit + 1) / n_used);
    }
    if (PRE && CTAS == 2) {
      const int last_round = n_dealt > 0 ? (n_dealt - 1) / n_units : 0;
      me = (last_round & 1) ? n_units - 1 - unit : unit;
      x = row.begin(me);
      x_end = row.begin(me + 1);
      slots = kSplitPerPair * n_units;
    }
    const int x_begin = x;
    auto owner = [&](int at) {
      if (PRE && CTAS == 2) return row.owner(at);
      return static_cast<int>((static_cast<int64_t>(at + 1) * n_used - 1) / total);
    };
    const uint32_t full = 0xffffffffu;
    // boxes of a tile: this CTA copies boxes_k of them for K, all for V
    const int boxes_k = KR / a.rb, rb_log = 31 - __clz(a.rb);
    const uint32_t box_k = static_cast<uint32_t>(a.rb) * D * (INT8 ? 1 : 2), box_v = box_k / CTAS;
    Ring st;  // K/V stage (bf16) or staging slot (int8)
    const int depth = INT8 ? a.staging : a.stages;
    uint64_t* fulls = INT8 ? a8->st_full : ax->kv_full;
    uint64_t* empties = INT8 ? a8->st_empty : ax->kv_empty;
    const uint32_t ring0 = tc::smem_addr(INT8 ? sI8 : sKV);
    constexpr int SLOT = INT8 ? STAGE / 2 : STAGE;
    uint32_t uses = 0, tile_no = 0, qn = 0;  // copies, tiles, query tiles so far
    bool ok = true;
    // A warp that has given up walks on without copies: the merge reads the
    // descriptor of every split item, and one that this call did not write
    // would be an earlier call's, or no descriptor at all.
#pragma unroll 1
    for (int k = 0;; k++) {
      Piece pc;
      pc.last = 1;
      pc.n = 0;
      pc.toks = 0;
      pc.slot = -1;
      // every other round backwards: pieces come longest first, so this evens the pairs' shares
      const int id = CTAS == 1 ? 0 : k * n_units + ((k & 1) ? n_units - 1 - unit : unit);
#pragma unroll 1
      while (pc.last) {
        if (PRE && CTAS == 2 && !stretch && id >= n_dealt) {
          stretch = true;
          b32 = base = 0;
          r = request_of<KT, PRE>(a, lane, false, &ax->disorder, true);
          scan();
        }
        const int at = stretch ? x : id;
        if (stretch && x >= x_end) break;
#pragma unroll 1
        while (b32 < n_req && at >= base + __shfl_sync(full, pp, 31)) {
          base += __shfl_sync(full, pp, 31);
          ibase += __shfl_sync(full, ii, 31);
          sbase += __shfl_sync(full, ss, 31);
          seen += __shfl_sync(full, tt, 31);
          b32 += 32;
          r = request_of<KT, PRE>(a, b32 + lane, false, &ax->disorder, true);
          scan();
        }
        if (b32 >= n_req) break;
        const int w = __ffs(__ballot_sync(full, at < base + pp)) - 1;
        Req q;
        q.start = __shfl_sync(full, r.start, w);
        q.nq = __shfl_sync(full, r.nq, w);
        q.T = __shfl_sync(full, r.T, w);
        q.nqt = __shfl_sync(full, r.nqt, w);
        q.ntmax = __shfl_sync(full, r.ntmax, w);
        if constexpr (PRE) {
          q.kind = __shfl_sync(full, r.kind, w);
          q.g = __shfl_sync(full, r.g, w);
          q.plen = __shfl_sync(full, r.plen, w);
          pc.slot = -1;  // (an item passed over has left its own)
        }
        const int before = __shfl_sync(full, pp, w);
        int item, nt, first = 0, n_seg = 1, seg = 0, list = 0;  // of a split item: pieces, this one's number, its place in the list
        if (stretch) {
          const int len = q.ntmax + OVH;
          const int start = base + before - q.nqt * a.Hkv * len;
          item = (x - start) / len;
          first = start + item * len;  // the item's place in the row
        } else {
          const int nsw = __shfl_sync(full, ns, w), kept = __shfl_sync(full, nw, w);
          const int cut = q.nqt * a.Hkv - kept;
          item = id - base - (before - kept - cut * nsw);
          if (item >= kept) {  // piece-major, so that neighbours in time read the same part of the keys
            const int idx = item - kept;
            seg = idx / cut;
            item = kept + idx % cut;
            n_seg = nsw;
            list = ibase + __shfl_sync(full, ii, w) - cut + item - kept;
            pc.slot = sbase + __shfl_sync(full, ss, w) - cut * nsw + (item - kept) * nsw + seg;
          }
        }
        pc.h = item % a.Hkv;
        const int qt = q.nqt - 1 - item / a.Hkv;  // longest first
        pc.b = b32 + w;
        pc.tok0 = q.start + qt * a.tpt;
        pc.toks = min(a.tpt, q.nq - qt * a.tpt);
        pc.pos0 = q.T - q.nq + qt * a.tpt;
        pc.last = 0;
        if constexpr (PRE) {
          int own = 0, none;
          if (q.kind != kPrefix) tile_range<KT>(a, q, qt, none, none, own);
          // the longest list has every prefix tile and the request's
          pc.nsink = q.kind == kPrefix ? q.ntmax
                     : q.kind == kFull ? static_cast<int>((min(static_cast<int64_t>(q.plen), a.n_prefix_pages * a.page) + KT - 1) / KT)
                                       : 0;
          nt = pc.nsink + own;
          pc.b = q.kind == kPrefix ? -1 : pc.b - a.n_groups;
          pc.lo = q.plen;
          if (pc.slot < 0 && (q.kind == kPrefix || q.kind == kBehind)) pc.slot = kDense;
        } else {
          tile_range<KT>(a, q, qt, pc.lo, pc.nsink, nt);
        }
        if (stretch) {
          // Tiles of the item lie at [first + kItem, first + len), fewer than
          // ntmax of them spread evenly; the CTAs that share these have its pieces.
          const int len = q.ntmax + OVH, lo = max(0, x - first - OVH), hi = max(0, min(len, x_end - first) - OVH);
          int f = me, l = me;
          if (q.ntmax == 0) {
            f = l = owner(first);
          } else if (first + OVH < x_begin || first + len > x_end) {
            f = owner(first + OVH);
            l = owner(first + len - 1);
          }
          x = min(x_end, first + len);
          pc.j0 = 0;
          pc.n = nt;
          if (me < f || me > l) {
            pc.last = 1;  // nothing of it but the part that stands for its pipeline
          } else if (f < l) {
            pc.j0 = nt == q.ntmax ? lo : static_cast<int>(static_cast<int64_t>(lo) * nt / q.ntmax);
            pc.n = (nt == q.ntmax ? hi : static_cast<int>(static_cast<int64_t>(hi) * nt / q.ntmax)) - pc.j0;
            n_seg = l - f + 1;
            seg = me - f;
            list = unit;
            pc.slot = slots + (seg == 0 ? 2 * me + 1 : 2 * me);
            listed |= seg == 0;
          }
        } else {
          const int each = nt / n_seg, more = nt % n_seg;  // the first `more` pieces take a tile more
          pc.j0 = seg * each + min(seg, more);
          pc.n = each + (seg < more ? 1 : 0);
        }
        if constexpr (PRE) {
          if (!pc.last && seg == 0 && rank == 0) {  // where the merge finds the item's rows
            const bool prefix = q.kind == kPrefix;
            const int dense = ((prefix ? a.n_tok : 0) + pc.tok0) * (a.Hkv * a.G) + pc.h * a.G;
            const int one = pc.slot >= 0 ? a.n_dense + pc.slot * a.part_rows : dense;
            const int two = stretch ? a.n_dense + (slots + 2 * me + 2) * a.part_rows : one + a.part_rows;
            const int n = (pc.slot == -1 ? 0 : n_seg) | (q.kind == kBehind ? kHasPrefix : 0);
            const int pitch = pc.slot >= 0 ? a.G : a.Hkv * a.G;  // from token to token
#pragma unroll 1
            for (int i = lane; i < pc.toks; i += 32)
              a.ws_rows[(static_cast<int64_t>(prefix ? a.n_tok : 0) + pc.tok0 + i) * a.Hkv + pc.h] =
                  make_int4(n, one + i * pitch, two + i * a.G, (stretch ? 2 : 1) * a.part_rows);
          }
          pc.slot = slot_and_group(pc.slot, q.g);
        } else if (!pc.last && n_seg > 1 && seg == 0 && rank == 0 && lane == 0) {
          a.ws_item[2 * list] = make_int4(pc.tok0, pc.toks * a.G, pc.h, pc.slot);
          // pieces; the slots of the second and of each further one
          a.ws_item[2 * list + 1] = CTAS == 1 ? make_int4(n_seg, 2 * unit + 2, 2, 0) : make_int4(n_seg, pc.slot + 1, 1, 0);
        }
      }
      if (pc.last) {
        pc.n = 0;
        pc.toks = 0;
        pc.slot = -1;
      }
      const int slot = k % kPieces;
      if (ok && k >= kPieces) ok = wait_all(&ax->pc_empty[slot], ((k / kPieces) - 1) & 1, abort);
      if (ok && lane == 0) {
        ax->pc[slot] = pc;
        tc::bar_arrive(&ax->pc_full[slot]);
      }
      if (pc.last) break;
      if (!ok) continue;
      // Copies, in the order the products take them.  Lane i holds the box of
      // rows [i rb, i rb + rb) of a tile; table entries are read two tiles ahead.
      BoxLoad l0 = box_load<KT, PRE>(a, pc, 0, lane), l1 = box_load<KT, PRE>(a, pc, 1, lane);
      Box cur{-1, false}, prev;
#pragma unroll 1
      for (int j = 0; ok && pc.n > 0 && j <= pc.n; j++) {
        const BoxLoad l2 = box_load<KT, PRE>(a, pc, j + 2, lane);
        prev = cur;
        cur = box_of<KT>(a, pc, l0, last_seen<PRE>(pc, j), lane);  // keys past it are not copied
        l0 = l1;
        l1 = l2;
        if (j < pc.n) {  // which 8-row groups have no page
          const uint32_t none = __ballot_sync(full, cur.want && cur.rg < 0);
          uint32_t m = 0;
          if (none) {
            if (lane == 0 && rank == 0) set_status(a.status, SKV_DEV_RANGE);
#pragma unroll 1
            for (int g = 0; g < KT / 8; g++) m |= ((none >> ((8 * g) >> rb_log)) & 1u) << g;
          }
          if (lane == 0) ax->tile_bad[tile_no % kTileInfo] = m;
          tile_no++;
        }
#pragma unroll 1
        for (int v = j < pc.n ? 0 : 1; v < (j == 0 ? 1 : 2); v++) {  // K(j), then V(j - 1)
          const Box x = v ? prev : cur;
          const int at = v ? lane : lane - static_cast<int>(rank) * boxes_k;
          const bool mine = x.want && x.rg >= 0 && (v || (at >= 0 && at < boxes_k));
          if (uses >= static_cast<uint32_t>(depth) && !(ok = wait_all(&empties[st.s], st.ph ^ 1, abort))) break;
          const uint32_t bytes = v ? box_v : box_k;
          const uint32_t cnt = __popc(__ballot_sync(full, mine));
          if (lane == 0) tc::bar_arrive_expect_tx(&fulls[st.s], cnt * bytes);
          __syncwarp();
          if (mine) {
            constexpr int kSubV = INT8 ? (D / CTAS >= 128 ? D / CTAS / 128 : 1) : VSUB;  // column blocks of the V box
            tma_rows(ring0 + st.s * SLOT + at * bytes, v ? &v_map : &k_map, v ? static_cast<int>(rank) * kSubV : 0,
                     x.rg, pc.h, &fulls[st.s]);
          }
          uses++;
          st.next(depth);
        }
        if (ok && j == 0) {  // the query tile, behind the first keys: it is free once the last piece's logits are done
          if (qn > 0 && !(ok = wait_all(&ax->q_free, (qn - 1) & 1, abort))) break;
          qn++;
          const CUtensorMap* map = &q_map;
          int box = a.q_box;
          if constexpr (PRE) {
            if (pc.b >= 0) {
              map = &maps.q_own;
              box = a.q_box_own;
            }
          }
          if (lane == 0) tc::bar_arrive_expect_tx(&ax->q_full, NSUB * box);
          __syncwarp();
          if (lane < NSUB)
            tma_query(tc::smem_addr(sQ) + lane * a.q_sub, map, pc.h * a.G, pc.tok0 + static_cast<int>(rank) * a.tpc,
                      lane, &ax->q_full);
        }
      }
    }
    if (!ok) {
      if (lane == 0) set_status(a.status, SKV_DEV_TIMEOUT);
      // Its own copies land while it waits here.  (They are waited for at the
      // end, too, whoever gave up; with that wait alone the compiler's int8
      // loops came out slower: 64 ragged requests 119.9 against 117.0 us, the
      // windowed chunk 142.4 against 139.3.)
      const uint64_t t0 = tc::global_ns();
      for (int i = 0; i < 1000000 && tc::global_ns() - t0 < 20000000ull; i++) __nanosleep(1000);
    }
    // split items of this call, for the merge
    if (PRE) {
      // (their rows were listed on the way)
    } else if (CTAS == 1) {
      if (!listed && lane == 0) a.ws_item[2 * unit + 1] = make_int4(0, 0, 0, 0);
    } else if (unit == 0 && rank == 0) {
      int cut = 0, before = 0, rows = 0;
#pragma unroll 1
      for (int b0 = 0; b0 < a.B; b0 += 32) {
        const auto x = request_of<KT, PRE>(a, b0 + lane, false, &ax->disorder, true);
        const int items = x.nqt * a.Hkv;
        int sum = items;
#pragma unroll 1
        for (int o = 1; o < 32; o <<= 1) {
          const int y = __shfl_up_sync(full, sum, o);
          if (lane >= o) sum += y;
        }
        if (pieces_of(x.ntmax, c) > 1) {
          const int n = items - min(items, max(0, whole - (before + sum - items)));
          cut += n;
          if (n > 0) rows = max(rows, min(a.tpt, x.nq) * a.G);
        }
        before += __shfl_sync(full, sum, 31);
      }
      cut = __reduce_add_sync(full, cut);
      rows = __reduce_max_sync(full, rows);
      if (lane == 0) {
        a.ws_head[0] = cut;
        a.ws_head[1] = rows;
        a.ws_head[2] = 0;
      }
    }
  } else if (warp == 1) {
    // ---------------- products (one thread of the leader) ----------------
    // elect.sync and not lane == 0: the compiler then knows that one thread is
    // left and issues the products with less around them (chunks of 2048 tokens
    // at 65536 keys: 1193 -> 1142 us).
    if (elect_one()) {
      constexpr uint32_t id_qk = idesc_bf16(kRows * CTAS, KT, 0), id_pv = idesc_bf16(kRows * CTAS, D, 1),
                         id_sum = idesc_bf16(kRows * CTAS, 16 * CTAS, 0);
      // K-major without a swizzle: eight rows of 16 bytes follow one another, 128
      // bytes on come the next eight keys; int8: rows 8 on repeat the first eight
      const uint64_t ones =
          (static_cast<uint64_t>(((INT8 ? 0 : 256) >> 4) | (1u << 14)) << 32) |
          desc_lo(INT8 ? tc::smem_addr(a8->rsum) : tc::smem_addr(ax->ones), 128);
      const uint32_t dQ = desc_lo(tc::smem_addr(sQ), 16), dK = desc_lo(tc::smem_addr(sKV), 16),
                     dV = desc_lo(tc::smem_addr(sKV), 1024);
      const uint32_t q_step = CTAS == 2 ? kRows * 128 >> 4 : a.q_sub >> 4;
      Ring st;
      uint32_t g = 0, np = 0;  // tiles, pieces with work so far
      bool ok = true;
#pragma unroll 1
      for (int k = 0; ok; k++) {
        const int slot = k % kPieces;
        ok = wait(&ax->pc_full[slot], (k / kPieces) & 1, abort);
        if (!ok) break;
        const int n = ax->pc[slot].n, last = ax->pc[slot].last;
        tc::bar_arrive(&ax->pc_empty[slot]);
        if (last) break;
        if (rank != 0) {  // the peer passes on to the leader that its query tile and its stages are full
          if (n > 0 && (ok = wait(&ax->q_full, np & 1, abort))) arrive_leader<CTAS>(&ax->q_full);
          np += n > 0;
#pragma unroll 1
          for (int f = 0; !INT8 && ok && f < 2 * n; f++) {
            ok = wait(&ax->kv_full[st.s], st.ph, abort);
            if (ok) arrive_leader<CTAS>(&ax->kv_full[st.s]);
            st.next(a.stages);
          }
          continue;
        }
        if (n == 0) continue;
        ok = wait(&ax->q_full, np & 1, abort);
#pragma unroll 1
        for (int j = 0; ok && j <= n; j++) {
          if (j < n) {
            ok = wait(&ax->kv_full[st.s], st.ph, abort);
            if (!ok) break;
            tc::tc_fence_after();
            const uint32_t kv = dK + st.s * (STAGE >> 4);
            const uint32_t d = tm + kSCol + ((g + j) & 1) * 128;
            {
#pragma unroll
              for (int x = 0; x < D / 16; x++) {
                const uint32_t off = ((x >> 2) * 1024 + (x & 3) * 32) >> 4;
                mma_ss<CTAS>(d, desc(dQ + (x >> 2) * q_step + (x & 3) * 2, 1024), desc(kv + off, SBO_K), id_qk, x > 0);
              }
              commit<CTAS>(&ax->kv_empty[st.s]);
              commit<CTAS>(&ax->s_full[(g + j) & 1]);
              if (j == n - 1) commit<CTAS>(&ax->q_free);
            }
            st.next(a.stages);
          }
          if (j >= 1) {
            const uint32_t t = g + j - 1;
            ok = wait(&ax->p_full[t & 1], (t >> 1) & 1, abort);
            ok = ok && wait(&ax->kv_full[st.s], st.ph, abort);
            if (!ok) break;
            tc::tc_fence_after();
            const uint32_t kv = dV + st.s * (STAGE >> 4);
            const uint32_t p = tm + kSCol + (t & 1) * 128;  // each half's weights start where its logits did
            {
#pragma unroll
              for (int x = 0; x < KT / 16; x++)
                mma_ts<CTAS>(tm, p + 8 * x + (x >= KT / 32 ? KT / 4 : 0), desc(kv + x * (2 * SBO_V >> 4), SBO_V), id_pv,
                             j > 1 || x > 0);
              commit<CTAS>(&ax->kv_empty[st.s]);
              if (SUM) {
#pragma unroll
                for (int x = 0; x < KT / 16; x++)
                  mma_ts<CTAS>(tm + LCOL, p + 8 * x + (x >= KT / 32 ? KT / 4 : 0),
                               INT8 ? ones + ((t % kScaleRing * KT + x * 16) * 16 >> 4) : ones, id_sum, j > 1 || x > 0);
                if (INT8) commit<CTAS>(&a8->sc_empty[t % kScaleRing]);
              }
              commit<CTAS>(&ax->pv_done[t & 1]);
            }
            st.next(a.stages);
          }
        }
        g += n;
        np++;
      }
      if (!ok) set_status(a.status, SKV_DEV_TIMEOUT);
      if (rank == 0) commit<CTAS>(&ax->mma_idle);  // nothing of this thread's may run when tensor memory is released
      if (!tc::bar_drain(&ax->mma_idle, 0, 4000000000ull)) set_status(a.status, SKV_DEV_TIMEOUT);
    }
    __syncwarp();
  } else if (warp < 4) {
    // ---------------- int8: row scales (warp 2 even tiles, warp 3 odd) ----------------
    if (INT8) {
      uint32_t g = 0;  // tiles so far
      bool ok = true;
#pragma unroll 1
      for (int k = 0; ok; k++) {
        const int slot = k % kPieces;
        ok = wait_all(&ax->pc_full[slot], (k / kPieces) & 1, abort);
        if (!ok) break;
        const Piece pc = ax->pc[slot];
        __syncwarp();
        if (lane == 0) tc::bar_arrive(&ax->pc_empty[slot]);
        if (pc.last) break;
        const int rb_log = 31 - __clz(a.rb);
        int j = static_cast<int>((g ^ (warp & 1)) & 1);  // first tile of this warp's parity
        BoxLoad l0 = box_load<KT, PRE>(a, pc, j, lane);
#pragma unroll 1
        for (; j < pc.n; j += 2) {
          const Box box = box_of<KT>(a, pc, l0, last_seen<PRE>(pc, j), lane);
          const int rg = box.want ? box.rg : -1;
          float ks[KT / 32], vs[KT / 32];
#pragma unroll
          for (int e = 0; e < KT / 32; e++) {  // key lane + 32 e: its box's group, its place in the box
            const int key = lane + 32 * e;
            const int kg = __shfl_sync(0xffffffffu, rg, key >> rb_log);
            const int64_t vec = (static_cast<int64_t>(kg) * 8 + (key & (a.rb - 1))) * a.Hkv + pc.h;
            ks[e] = kg >= 0 ? __half2float(a.k_scale[vec]) * a.scale_log2 : 0.f;
            vs[e] = kg >= 0 ? __half2float(a.v_scale[vec]) : 0.f;
          }
          l0 = box_load<KT, PRE>(a, pc, j + 2, lane);
          const uint32_t t = g + j, s = t % kScaleRing;
          if (t >= kScaleRing && !(ok = wait_all(&a8->sc_empty[s], (t / kScaleRing - 1) & 1, abort))) break;
          bool wild = false;
#pragma unroll
          for (int e = 0; e < KT / 32; e++) {
            a8->ks[s][lane + 32 * e] = ks[e];
            // A zero scale would leave the sum without the row's weight: 2^-100 keeps
            // it, and the values at zero.  A scale that is not finite has no reciprocal.
            const float v = vs[e] == 0.f ? 7.888609e-31f : vs[e];
            a8->vs[s][lane + 32 * e] = v;
            const bool finite = fabsf(v) <= 65504.f;
            wild |= !finite;
            const float r = finite ? 1.f / v : 0.f;
            if (SUM) {
              const int key = lane + 32 * e;
              uint16_t* to = &a8->rsum[s][(key >> 3) * 64 + (key & 7)];
              const uint32_t hi = pack_bf16(r, 0.f) & 0xffffu;
              to[0] = static_cast<uint16_t>(hi);
              to[8] = static_cast<uint16_t>(pack_bf16(r - __uint_as_float(hi << 16), 0.f));
            } else {
              a8->rs[s][lane + 32 * e] = r;
            }
          }
          if (SUM) tc::fence_async_smem();
          wild = __any_sync(0xffffffffu, wild);
          __syncwarp();
          if (lane == 0) {
            a8->wild[s] = wild;
            tc::bar_arrive(&a8->sc_full[s]);
          }
        }
        g += pc.n;
      }
    }
  } else if (softer) {
    // ---------------- softmax and output: thread = row, two groups ----------------
    // Group `wg` takes half of every tile's keys and half of the output's
    // columns: the logits-to-weights time stands between two products of the
    // same tile, so it is halved by two warps per 32 rows rather than spread
    // over two tiles (3.4K against 2.5K clocks a tile).  The two agree on the
    // tile's maximum through shared memory, so both hold the same running
    // maximum, and add up their sums at a piece's end.
    const int wg = (warp - 4) >> 2, quad = warp & 3;
    const int r = 32 * quad + lane;                     // row within this CTA
    const int tok_r = r / a.G, head_r = r % a.G;        // its token within the CTA's part of the tile, its head
    const uint32_t lane_base = static_cast<uint32_t>(32 * quad) << 16;
    uint32_t g = 0, fills = 0, xc = 0;  // tiles, ring fills, exchanges so far
    bool ok = true;

    // This thread's value and its partner's (the other group's, same row), over
    // a named barrier of the two warps (an mbarrier took 100 clocks more).  Such
    // a barrier has no bound of its own: each warp, done or given up, goes on
    // exchanging kGone until it gets kGone back, so neither is left waiting.
    auto exchange = [&](float v, float& other) {
      ax->x[xc & 1][wg][r] = v;
      asm volatile("bar.sync %0, 64;" ::"r"(1 + quad) : "memory");
      other = ax->x[xc & 1][wg ^ 1][r];
      xc++;
    };

    auto get = [&](int k, Piece& pc) -> bool {  // descriptor k
      const int slot = k % kPieces;
      if (!wait_all(&ax->pc_full[slot], (k / kPieces) & 1, abort)) return false;
      pc = ax->pc[slot];
      __syncwarp();
      if (lane == 0) tc::bar_arrive(&ax->pc_empty[slot]);
      return true;
    };

    Piece pc;
    bool ready = false;  // the next tile's logits (and scales) are known to be there
    ok = get(0, pc);
#pragma unroll 1
    for (int k = 0; ok && !pc.last; k++) {
      const int tok_i = static_cast<int>(rank) * a.tpc + tok_r;  // this row's token within the tile
      const bool live = tok_r < a.tpc && tok_i < pc.toks;
      const int pos = live ? pc.pos0 + tok_i : -1;  // this row's position: keys 0 .. pos
      // some row of the warp is used
      const bool warp_live = 32 * quad < min(a.tpc, pc.toks - static_cast<int>(rank) * a.tpc) * a.G;
      float m_ref = -INFINITY, l = 0.f;           // the maximum that l is relative to
      const int pos_last = pc.pos0 + pc.toks - 1;
#pragma unroll 1
      for (int j = 0; j < pc.n; j++) {
        const uint32_t t = g + j;
        const int t0 = tile_of<PRE>(pc, j) * KT;
        const int p = PRE && !live ? -1 : seen<PRE>(pc, j, pos), p_last = seen<PRE>(pc, j, pos_last);
        // every row of the tile sees every key unless one of these holds, or a page is missing
        const bool edge = t0 + KT - 1 > seen<PRE>(pc, j, pc.pos0) || (a.W > 0 && t0 <= p_last - a.W && t0 + KT > a.S);
        constexpr int HC = KT / 2;  // this group's keys of the tile
        const uint32_t scol = tm + lane_base + kSCol + (t & 1) * 128 + wg * HC;
        const uint32_t sc = t % kScaleRing;
        if (!(PRE && INT8) || !__all_sync(0xffffffffu, ready)) {
          if (INT8 && !(ok = wait_all(&a8->sc_full[sc], (t / kScaleRing) & 1, abort))) break;
          if (!(ok = wait_all(&ax->s_full[t & 1], (t >> 1) & 1, abort))) break;
        }
        ready = false;
        tc::tc_fence_after();
        const uint32_t bad = ax->tile_bad[t % kTileInfo];
        const bool masked = edge || bad != 0;
        const bool wild = INT8 && masked && a8->wild[sc];
        if (warp_live) {
          uint32_t s[HC / 32][32];
#pragma unroll
          for (int c = 0; c < HC / 32; c++) tc::tmem_ld32(scol + 32 * c, s[c]);
          tc::tmem_wait_ld();
          F2 x[HC / 2];
#pragma unroll
          for (int i = 0; i < HC / 2; i++)
            x[i] = f2(__uint_as_float(s[i / 16][2 * i % 32]), __uint_as_float(s[i / 16][2 * i % 32 + 1]));
          if (INT8) {
#pragma unroll
            for (int i = 0; i < HC / 2; i += 2) {
              const ulonglong2 f = *reinterpret_cast<const ulonglong2*>(&a8->ks[sc][wg * HC + 2 * i]);
              x[i] = f2_mul(x[i], F2{f.x});
              x[i + 1] = f2_mul(x[i + 1], F2{f.y});
            }
          }
          uint32_t vis[HC / 32];  // bit i: key 32 c + i of this group is visible
          if (masked) {
            const int f0 = t0 + wg * HC;  // first key of this group
#pragma unroll
            for (int c = 0; c < HC / 32; c++) {
              const int f = f0 + 32 * c;
              vis[c] = bits_below(p + 1 - f);
              if (a.W > 0) vis[c] &= ~bits_below(p - a.W + 1 - f) | bits_below(a.S - f);
              if (bad) {
                const uint32_t b4 = bad >> ((f - t0) >> 3);
                vis[c] &= ~((b4 & 1 ? 0xffu : 0u) | (b4 & 2 ? 0xff00u : 0u) | (b4 & 4 ? 0xff0000u : 0u) |
                            (b4 & 8 ? 0xff000000u : 0u));
              }
            }
#pragma unroll
            for (int i = 0; i < HC / 2; i++) {
              const float2 v = f2_out(x[i]);
              x[i] = f2((vis[i / 16] >> (2 * i % 32)) & 1u ? v.x : -INFINITY,
                        (vis[i / 16] >> (2 * i % 32 + 1)) & 1u ? v.y : -INFINITY);
            }
          }
          float mp[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int i = 0; i < HC / 2; i++) {
            const float2 v = f2_out(x[i]);
            mp[i & 3] = max3(mp[i & 3], v.x, v.y);
          }
          const float f = INT8 ? 1.f : a.scale_log2;
          float mc = fmaxf(max3(mp[0], mp[1], mp[2]), mp[3]) * f, mo;
          if (!live) mc = -INFINITY;  // a row without a query holds anything: it must not call for a rescale
          exchange(mc, mo);
          mc = fmaxf(mc, mo);
          const float m_new = mc > m_ref + kLazy || m_ref == -INFINITY ? fmaxf(mc, m_ref) : m_ref;
          if (__any_sync(0xffffffffu, m_new != m_ref)) {
            const float alpha = m_new == m_ref ? 1.f : tc::ex2_approx(m_ref - m_new);
            if (j > 0) {
              if (!(ok = wait_all(&ax->pv_done[(t - 1) & 1], ((t - 1) >> 1) & 1, abort))) break;
              tc::tc_fence_after();
#pragma unroll 1
              for (int c0 = wg * (D / 2); c0 < (wg + 1) * (D / 2); c0 += 32) {
                uint32_t o[32];
                tc::tmem_ld32(tm + lane_base + c0, o);
                tc::tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 32; i++) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
                tc::tmem_st32(tm + lane_base + c0, o);
              }
              if (SUM && wg == 0) {
                const float2 s2 = tmem_ld2(tm + lane_base + LCOL);
                tmem_st2(tm + lane_base + LCOL, make_float2(s2.x * alpha, s2.y * alpha));
              }
            }
            l = m_ref == -INFINITY ? 0.f : l * alpha;
            m_ref = m_new;
          }
          // Asked for under the exponentials, the next tile's logits and scales mostly
          // cost no wait: 80 drafts 155 -> 148 us (with 3 wide stages), eight agents
          // 144.7 -> 143.4.  Without prefixes the windowed chunk lost (136.4, 139.7),
          // and bf16 rows (57.0, 59.1 for 40 tokens behind five prefixes).
          if (PRE && INT8) {
            ready = tc::bar_poll(&ax->s_full[(t + 1) & 1], ((t + 1) >> 1) & 1);
            ready &= tc::bar_poll(&a8->sc_full[(t + 1) % kScaleRing], ((t + 1) / kScaleRing) & 1);
          }
          const float m_use = m_ref == -INFINITY ? 0.f : m_ref;
          const F2 ff = f2(f, f), mm = f2(-m_use, -m_use);
          F2 ls[2] = {f2(0.f, 0.f), f2(0.f, 0.f)};
#pragma unroll
          for (int c = 0; c < HC / 32; c++) {
            uint32_t pk[16];
#pragma unroll
            for (int y = 0; y < 16; y += 2) {
              const int i = 16 * c + y;
              float2 e[2];
#pragma unroll
              for (int z = 0; z < 2; z++) {
                e[z] = f2_out(INT8 ? f2_add(x[i + z], mm) : f2_fma(x[i + z], ff, mm));
                e[z].x = tc::ex2_approx(e[z].x);
                e[z].y = tc::ex2_approx(e[z].y);
              }
              if (INT8) {
                const ulonglong2 v = *reinterpret_cast<const ulonglong2*>(&a8->vs[sc][wg * HC + 2 * i]);
                e[0] = f2_out(f2_mul(f2(e[0].x, e[0].y), F2{v.x}));
                e[1] = f2_out(f2_mul(f2(e[1].x, e[1].y), F2{v.y}));
              }
#pragma unroll
              for (int z = 0; z < 2; z++) {
                const uint32_t w = pack_bf16(e[z].x, e[z].y);
                pk[y + z] = w;
                // The sum takes the weights as they are rounded, so that the weights
                // applied add up to one: with few keys their errors cancel.
                if (!INT8 && !SUM) ls[z] = f2_add(ls[z], f2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u)));
              }
            }
            // A scale that this row does not see may be anything.  (Asked of each weight,
            // its mask was a tenth of the kernel's instructions: 80 drafts behind 60000
            // keys 167 us, now 154.)
            if (wild) {
#pragma unroll
              for (int y = 0; y < 16; y++)
                pk[y] &= (vis[c] >> (2 * y) & 1u ? 0xffffu : 0u) | (vis[c] >> (2 * y + 1) & 1u ? 0xffff0000u : 0u);
            }
            if (INT8 && !SUM) {
#pragma unroll
              for (int y = 0; y < 16; y += 2) {
                const ulonglong2 r = *reinterpret_cast<const ulonglong2*>(&a8->rs[sc][wg * HC + 32 * c + 2 * y]);
                ls[0] = f2_fma(f2(__uint_as_float(pk[y] << 16), __uint_as_float(pk[y] & 0xffff0000u)), F2{r.x}, ls[0]);
                ls[1] = f2_fma(f2(__uint_as_float(pk[y + 1] << 16), __uint_as_float(pk[y + 1] & 0xffff0000u)), F2{r.y},
                               ls[1]);
              }
            }
            tmem_st16(scol + 16 * c, pk);
          }
          const float2 l0 = f2_out(f2_add(ls[0], ls[1]));
          l += l0.x + l0.y;
          tc::tmem_wait_st();
        }  // a warp without rows leaves S as its weights: rows are independent, and its are not used
        if (!INT8 && masked) {
          // Zero weights do not stop a NaN: rows of V that no query of the tile
          // sees become zero, and so does every value that is not finite (put
          // back for the queries that see it when the output is written).
          const uint32_t fv = fills + fill_v(j, pc.n);
          const uint32_t vs = fv % a.stages;
          if (!(ok = wait_all(&ax->kv_full[vs], (fv / a.stages) & 1, abort))) break;
          unsigned char* V = sKV + vs * STAGE;
          bool found = false;
          // A single token's keys, and a prefix's, every query of the tile sees or none
          // does: there is nothing to look for, and nothing before the first unseen row.
          const bool alike = PRE && (pc.toks == 1 || of_prefix<PRE>(pc, j));
          const int skip = alike && bad == 0 ? (max(p_last + 1 - t0, 0) >> 3) * (VSUB * 64) : 0;
#pragma unroll 1
          for (int i = skip + tid - 128; i < STAGE / 16; i += 256) {
            const int grp = i / (VSUB * 64), row = grp * 8 + ((i >> 3) & 7);  // 64 16-byte pieces per 1024 B block
            uint4* at = reinterpret_cast<uint4*>(V + i * 16);
            const int key = t0 + row;  // seen by no query of the tile: its page may not have been read
            const bool dead = key > p_last || (a.W > 0 && key <= pc.pos0 - a.W && key >= a.S) || ((bad >> grp) & 1u);
            if (alike) {
              if (dead) *at = make_uint4(0u, 0u, 0u, 0u);
              continue;
            }
            uint4 w = dead ? make_uint4(0u, 0u, 0u, 0u) : *at;
            uint32_t* e = reinterpret_cast<uint32_t*>(&w);
            bool change = dead;
#pragma unroll
            for (int y = 0; y < 4; y++) {
              if ((e[y] & 0x7f80u) == 0x7f80u) {
                e[y] &= 0xffff0000u;
                change = found = true;
              }
              if ((e[y] & 0x7f800000u) == 0x7f800000u) {
                e[y] &= 0x0000ffffu;
                change = found = true;
              }
            }
            if (change) *at = w;
          }
          if (found) {
            *reinterpret_cast<volatile int*>(&ax->dirty) = 1;
            if (CTAS == 2)
              asm volatile(
                  "{\n.reg .b32 ra;\nmapa.shared::cluster.u32 ra, %0, %1;\nst.shared::cluster.u32 [ra], %2;\n}\n" ::"r"(
                      tc::smem_addr(&ax->dirty)),
                  "r"(rank ^ 1u), "r"(1)
                  : "memory");
            __threadfence();  // the peer reads it after this tile's products
          }
          tc::fence_async_smem();
        }
        tc::tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if (INT8) tc::bar_arrive(&a8->sc_empty[sc]);
          arrive_leader<CTAS>(&ax->p_full[t & 1]);
        }
      }
      if (!ok) break;
      const uint32_t t_last = g + pc.n - 1;
      if (pc.n > 0) {
        if (!SUM && warp_live) {
          float lo;
          exchange(l, lo);
          l += lo;  // a sum of two: the same in both
        }
        if (!(ok = wait_all(&ax->pv_done[t_last & 1], (t_last >> 1) & 1, abort))) break;
        tc::tc_fence_after();
      }
      // ---- output: this group's half of the columns ----
      if (warp_live) {
        const int part = slot_of<PRE>(pc);
        const bool whole = PRE ? part == -1 : part < 0;
        if (SUM && pc.n > 0) {
          const float2 s2 = tmem_ld2(tm + lane_base + LCOL);
          l = INT8 ? s2.x + s2.y : s2.x;
        }
        const float inv = whole ? (l != 0.f ? 1.f / l : 0.f) : 1.f;
        const bool dirty = !INT8 && *reinterpret_cast<volatile int*>(&ax->dirty) != 0;
        const int64_t tok = static_cast<int64_t>(pc.tok0) + tok_i;
        int64_t prow = static_cast<int64_t>(part) * a.part_rows + tok_i * a.G + head_r;
        if (PRE)
          prow = part == kDense ? ((pc.b < 0 ? a.n_tok : 0) + tok) * (a.Hkv * a.G) + pc.h * a.G + head_r
                                   : prow + a.n_dense;
        unsigned char* buf = sOut + (warp - 4) * 2048;
        const int id = !live ? -1 : whole ? static_cast<int>(tok * (a.Hkv * a.G)) + pc.h * a.G + head_r : static_cast<int>(prow);
        char* base = whole ? reinterpret_cast<char*>(a.out) : reinterpret_cast<char*>(a.ws_o);
        const int pitch = whole ? 2 * D : 4 * D;
        // With a few rows each lane writes its own (a window's single tokens 19.7 ->
        // 19.3 us; with 32 rows that took 4 to 7 % of a chunk).
        const bool few = (CTAS == 1 || PRE) && __popc(__ballot_sync(0xffffffffu, live)) <= 8;
        char* to[4];
#pragma unroll
        for (int x = 0; x < 4; x++) {
          const int row = few ? id : __shfl_sync(0xffffffffu, id, 8 * x + (lane >> 2));
          to[x] = row < 0 ? nullptr : base + static_cast<int64_t>(row) * pitch + (few ? 0 : 16 * (lane & 3));
        }
        auto put = [&](const uint32_t (&w)[16], int at) {  // 64 bytes of each row
          if (!few) {
            put_rows(buf, lane, w, to, at);
          } else if (live) {
#pragma unroll
            for (int i = 0; i < 4; i++)
              *reinterpret_cast<uint4*>(to[0] + at + 16 * i) = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
          }
        };
#pragma unroll 1
        for (int c0 = wg * (D / 2); c0 < (wg + 1) * (D / 2); c0 += 32) {
          uint32_t o[32];
          if (pc.n > 0) {
            tc::tmem_ld32(tm + lane_base + c0, o);
            tc::tmem_wait_ld();
          } else {
#pragma unroll
            for (int i = 0; i < 32; i++) o[i] = 0u;
          }
          if (dirty) {
            float y[32];
#pragma unroll 1
            for (int i = 0; i < 32; i++) y[i] = 0.f;
            if (live) add_nonfinite<D, KT, PRE>(a, pc, pos, pos_last, c0, y);
#pragma unroll
            for (int i = 0; i < 32; i++) o[i] = __float_as_uint(__uint_as_float(o[i]) + y[i]);
            __syncwarp();
          }
          uint32_t w[16];
          if (whole) {
#pragma unroll
            for (int i = 0; i < 16; i++)
              w[i] = pack_bf16(__uint_as_float(o[2 * i]) * inv, __uint_as_float(o[2 * i + 1]) * inv);
            put(w, 2 * c0);
          } else if (pc.n > 0) {
#pragma unroll
            for (int y = 0; y < 2; y++) {
#pragma unroll
              for (int i = 0; i < 16; i++) w[i] = o[16 * y + i];
              put(w, 4 * (c0 + 16 * y));
            }
          }
        }
        if (!whole && live && wg == 0) a.ws_ml[prow] = make_float2(m_ref, l);
      }
      tc::tc_fence_before();  // the next piece's weights also say that this one's O has been read
      g += pc.n;
      fills += 2 * pc.n;
      ok = get(k + 1, pc);
    }
    if (!ok) {
      if (lane == 0) set_status(a.status, SKV_DEV_TIMEOUT);
      __syncwarp();
      tc::tmem_wait_ld();
    }
    for (float other = 0.f; __float_as_uint(other) != kGone;) exchange(__uint_as_float(kGone), other);
  } else if (INT8 && (warp >= 12 || warp < 8 || warp == 11 || half)) {
    // ---------------- int8 -> bf16 (warps 12-15, and where they are free 5, 6, 7, 11) ----------------
    const int extra = half ? (warp >= 10 ? warp - 8 : warp - 6) : warp == 11 ? 3 : warp - 5;
    const int ct = warp >= 12 ? tid - 384 : 128 + 32 * extra + lane;
    // Thread -> 16 codes of one row, a few times a stage: ct % 8 is the row
    // of its 8-row group, so eight lanes read eight rows' swizzled pieces
    // (distinct banks) and write them the same way.  Piece `pce` of a row is
    // bytes 16 pce of the staged row and the 32 bytes at 32 pce of the wide
    // one; a step of 128 threads is 2048 staged bytes, 4096 wide ones.
    constexpr int kSteps = STAGE / 4096;
    const int jump = thin ? 2 : 1;
    auto offsets = [&](int row_bytes, uint32_t& s, uint32_t& d) {
      const int pcs = row_bytes / 16, row = ct & 7, grp = (ct >> 3) / pcs, pce = (ct >> 3) % pcs;
      if (row_bytes == 64)  // 64-byte rows, 64-byte swizzle
        s = grp * 512 + row * 64 + ((pce ^ (row >> 1)) << 4 & 0x30);
      else  // [8-row group][128-byte block][8 rows], 128-byte swizzle
        s = grp * (row_bytes * 8) + (pce >> 3) * 1024 + row * 128 + (((pce & 7) ^ row) << 4);
      d = grp * (row_bytes * 16) + (pce >> 2) * 1024 + row * 128 + ((((pce & 3) * 2) ^ row) << 4);
    };
    uint32_t sk, dk, sv, dv;
    offsets(D, sk, dk);
    offsets(D / CTAS, sv, dv);
    Ring st, sg;
    uint32_t uses = 0;
    bool ok = true;
#pragma unroll 1
    for (int k = 0; ok; k++) {
      const int slot = k % kPieces;
      ok = wait_all(&ax->pc_full[slot], (k / kPieces) & 1, abort);
      if (!ok) break;
      const int n = ax->pc[slot].n, last = ax->pc[slot].last;
      __syncwarp();
      if (lane == 0) tc::bar_arrive(&ax->pc_empty[slot]);
      if (last) break;
#pragma unroll 1
      for (int f = 0; f < 2 * n; f++) {
        const bool is_v = !(f == 0 || ((f & 1) && f != 2 * n - 1));
        ok = wait_all(&a8->st_full[sg.s], sg.ph, abort);
        if (ok && uses >= static_cast<uint32_t>(a.stages))
          ok = wait_all(&ax->kv_empty[st.s], st.ph ^ 1, abort);
        if (!ok) break;
        const unsigned char* src = sI8 + sg.s * (STAGE / 2);
        unsigned char* dst = sKV + st.s * STAGE;
        const uint32_t s0 = is_v ? sv : sk, d0 = is_v ? dv : dk;
#pragma unroll 1
        for (int y0 = 0; y0 < kSteps; y0 += 4 * jump) {
          uint4 w[4];
#pragma unroll
          for (int y = 0; y < 4; y++) w[y] = *reinterpret_cast<const uint4*>(src + s0 + (y0 + y * jump) * 2048);
#pragma unroll
          for (int y = 0; y < 4; y++) {
            unsigned char* d = dst + (y0 + y * jump) * 4096;
            *reinterpret_cast<uint4*>(d + d0) = make_uint4(int8_to_bf16x2<0>(w[y].x), int8_to_bf16x2<1>(w[y].x),
                                                           int8_to_bf16x2<0>(w[y].y), int8_to_bf16x2<1>(w[y].y));
            *reinterpret_cast<uint4*>(d + (d0 ^ 16)) = make_uint4(int8_to_bf16x2<0>(w[y].z), int8_to_bf16x2<1>(w[y].z),
                                                                  int8_to_bf16x2<0>(w[y].w), int8_to_bf16x2<1>(w[y].w));
          }
        }
        tc::fence_async_smem();
        __syncwarp();
        if (lane == 0) {
          tc::bar_arrive(&a8->st_empty[sg.s]);
          arrive_leader<CTAS>(&ax->kv_full[st.s]);
        }
        uses++;
        st.next(a.stages);
        sg.next(a.staging);
      }
    }
    if (!ok && lane == 0) set_status(a.status, SKV_DEV_TIMEOUT);
  }

  __syncwarp();
  tc::tc_fence_before();
  if (CTAS == 2)
    tc::cluster_sync();  // no CTA leaves while its peer may still signal it
  else
    __syncthreads();
  // Whichever role gave up, copies that none has waited for may be in flight,
  // also where the copying warp had issued its last: they land before the CTA
  // leaves.  (Where none gave up, each has been waited for by who used it: the
  // products, the peer's notes to the leader or the widening warps.)
  if (warp == 0 && *abort) {
    const uint64_t t0 = tc::global_ns();
    for (int i = 0; i < 1000000 && tc::global_ns() - t0 < 20000000ull; i++) __nanosleep(1000);
    __syncwarp();
  }
  if (warp == 1) {
    tc::tc_fence_after();
    if (CTAS == 1)
      tc::tmem_dealloc<512>(tm);
    else
      asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tm));
  }
  if (CTAS == 2) tc::cluster_sync();
}

// ---- host ------------------------------------------------------------------------

using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                              const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                              CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encode_fn() {
  static std::atomic<EncodeFn> fn{nullptr};
  EncodeFn f = fn.load(std::memory_order_acquire);
  if (f) return f;
  void* p = nullptr;
  cudaDriverEntryPointQueryResult res;
  if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &res) != cudaSuccess ||
      res != cudaDriverEntryPointSuccess) {
    cudaGetLastError();
    return nullptr;
  }
  f = reinterpret_cast<EncodeFn>(p);
  fn.store(f, std::memory_order_release);
  return f;
}

// Rows as [KV head][8-row group][column block][8 rows][column block's values]:
// a box of `rows` rows and `subs` column blocks lands as the tensor cores read it.
bool encode_rows(CUtensorMap* map, const void* pool, bool int8, int Hkv, int d, int64_t n_rows, int block, int subs,
                 int rows) {
  const int es = int8 ? 1 : 2;
  const cuuint64_t pitch = static_cast<cuuint64_t>(Hkv) * d * es;
  const cuuint64_t dims[5] = {static_cast<cuuint64_t>(block), 8, static_cast<cuuint64_t>(d / block),
                              static_cast<cuuint64_t>(n_rows / 8), static_cast<cuuint64_t>(Hkv)};
  const cuuint64_t strides[4] = {pitch, static_cast<cuuint64_t>(block) * es, 8 * pitch,
                                 static_cast<cuuint64_t>(d) * es};
  const cuuint32_t box[5] = {static_cast<cuuint32_t>(block), 8, static_cast<cuuint32_t>(subs),
                             static_cast<cuuint32_t>(rows / 8), 1};
  const cuuint32_t ones[5] = {1, 1, 1, 1, 1};
  return encode_fn()(map, int8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5,
                     const_cast<void*>(pool), dims, strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
                     block * es == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
                     CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <bool PRE>
bool encode_pools(Maps<PRE>& maps, const void* k, const void* v, bool int8, int Hkv, int d, int64_t n_rows, int ctas,
                  int rows) {
  const int block = int8 ? 128 : 64;  // columns of a 128-byte block
  const int vcols = d / ctas, vblock = vcols < block ? vcols : block;
  return encode_rows(&maps.k, k, int8, Hkv, d, n_rows, block, d / block, rows) &&
         encode_rows(&maps.v, v, int8, Hkv, d, n_rows, vblock, vcols / vblock, rows);
}

// Queries as [column block][token][head][64]: a box holds a group's heads of
// `toks` tokens; tokens past the last read as zeros.
bool encode_query(CUtensorMap* map, const uint16_t* q, int64_t q_stride, int n_tok, int Hq, int G, int d, int toks) {
  const cuuint64_t dims[4] = {64, static_cast<cuuint64_t>(Hq), static_cast<cuuint64_t>(n_tok),
                              static_cast<cuuint64_t>(d / 64)};
  const cuuint64_t strides[3] = {static_cast<cuuint64_t>(d) * 2, static_cast<cuuint64_t>(q_stride) * 2, 128};
  const cuuint32_t box[4] = {64, static_cast<cuuint32_t>(G), static_cast<cuuint32_t>(toks), 1};
  const cuuint32_t ones[4] = {1, 1, 1, 1};
  return encode_fn()(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<uint16_t*>(q), dims, strides, box, ones,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

void set_page(PagedArgs& a, int page) {
  a.page = page;
  a.rb = 8;  // rows per box: the largest power of two up to 64 that divides the page
  while (a.rb < 64 && page % (2 * a.rb) == 0) a.rb *= 2;
  while ((1u << a.page_shift) < static_cast<uint32_t>(page)) a.page_shift++;
  a.page_mul = static_cast<uint32_t>(((((static_cast<uint64_t>(1) << a.page_shift) - page) << 32) / page) + 1);
}

// A partial row is 4 d bytes out and back through L2 by all SMs (0.3 ns at
// d = 256), a tile about 0.75 us (64 keys) or 1.2 us (128).
float part_cost(int rows, int d, int ctas) {
  return static_cast<float>(rows) * d / 256.f * (ctas == 2 ? 1.5e-4f : 2e-4f);
}

// Rows of a query tile that can hold a token: the tile's tokens, or all there are.
int tile_rows(int n_tok, int G, int ctas) {
  const int tpt = ctas * (kRows / G);
  return (n_tok < tpt ? n_tok : tpt) * G;
}

// Shared memory of a CTA: the query tile (q_sub bytes per 64 columns), then as
// many stages as fit.  int8 rows: four wide stages (pairs three, six of half
// the size at 128 dims), the rest staging; where that would leave fewer than
// two staging slots (128 dims: three), as beside a full query tile, a wide stage
// makes room (64 ragged requests: 3 and 6 slots 130.2 us, 4 and 4 129.3, 5 and
// 2 156; 128 dims, 80 drafts behind a shared prefix of 60000: 4 and 2 155, 3 and 4
// 148, 16 x 5 drafts with 60000 keys each 702 and 648, 8 x 32 tokens at 30000 201 and
// 181, 64 ragged single tokens 174 and 173, 16 x 20 in a window of 1024 34.5 and 34.6,
// 64 x 2 ragged tokens of 8 heads a KV head 83.7 and 84.2).  With
// q_start the tokens of a request are not known here, so a batch of single tokens
// gets a full tile's layout: the same requests take 153 us with q_start, 118
// without (bf16 rows 134 either way).
struct Shared {
  int q_bytes, stages, staging, total;
};
constexpr Shared shared_layout(int d, int ctas, bool int8, int q_sub) {
  Shared s{};
  const int stage = keys_per_tile(d, ctas) / ctas * d * 2;
  const int aux8 = static_cast<int>(keys_per_tile(d, ctas) == 64 ? sizeof(Aux8<64>) : sizeof(Aux8<128>));
  const int aux = static_cast<int>(sizeof(Aux)) + (int8 ? aux8 : 0);
  s.q_bytes = q_sub * (d / 64);
  const int room = kMaxSmem - kOutBytes - aux - s.q_bytes;
  if (int8) {
    s.stages = ctas == 1 ? 4 : d == 128 ? 6 : 3;
    while (s.stages > 1 && (room - s.stages * stage) / (stage / 2) < (d == 128 ? 3 : 2)) s.stages--;
    s.staging = (room - s.stages * stage) / (stage / 2);
    if (s.staging > kMaxStaging) s.staging = kMaxStaging;
  } else {
    s.stages = room / stage;
    if (s.stages > kMaxStages) s.stages = kMaxStages;
  }
  s.total = s.q_bytes + s.stages * stage + s.staging * (stage / 2) + kOutBytes + aux;
  return s;
}
// A full query tile leaves the least room: two keys' tiles and the values
// between them, and int8 rows two slots to arrive in.
constexpr bool fits(int d, int ctas, bool int8) {
  const Shared s = shared_layout(d, ctas, int8, kRows * 128);
  return s.stages >= 3 && (!int8 || s.staging >= 2) && s.total <= kMaxSmem;
}
static_assert(fits(128, 1, false) && fits(128, 2, false) && fits(256, 1, false) && fits(256, 2, false) &&
                  fits(128, 1, true) && fits(128, 2, true) && fits(256, 1, true) && fits(256, 2, true),
              "every kind of call has its stages");
// The ring that the batch waits in while pairs plan.
constexpr int ring_bytes(int d, bool int8) {
  return shared_layout(d, 2, int8, kRows * 128).stages * (keys_per_tile(d, 2) / 2 * d * 2);
}
constexpr int kMaxEntries = 8192;  // requests and groups
static_assert(ring_bytes(128, false) >= 8 * kMaxEntries && ring_bytes(128, true) >= 8 * kMaxEntries &&
                  ring_bytes(256, false) >= 8 * kMaxEntries && ring_bytes(256, true) >= 8 * kMaxEntries,
              "eight bytes for each");

}  // namespace
}  // namespace skv
