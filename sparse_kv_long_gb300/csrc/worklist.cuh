// worklist.cuh -- the entries of the paged attention's work list: which new tokens
// a request or a group of requests has, how many query tiles and how many key
// tiles these are, from offsets and lengths on the device that may be anything.
// Nothing here reads outside the arrays that the call names.
#pragma once

#include <type_traits>

#include "common.cuh"

namespace skv {
namespace {

struct PagedArgs {
  int B, n_tok, Hkv, G, tpc, tpt;  // tokens per CTA's 128 rows, and per query tile
  const uint16_t* v_pool;     // bf16 rows, for the non-finite pass only
  const __half *k_scale, *v_scale;
  int64_t n_blocks;
  int page, rb;               // rows per TMA box
  uint32_t page_mul, page_shift;  // t / page = (umulhi(page_mul, t) + t) >> page_shift for t < 2^31
  const int32_t* block_table;
  int64_t n_pages;
  const int32_t *q_start, *lengths;
  int S, W;
  float scale_log2;
  uint16_t* out;
  int32_t* status;
  int stages, staging;        // ring depths
  int thin;                   // int8: query tiles of at most 32 rows (2: 64); the other rows' softmax warps widen instead
  int q_bytes;                // shared memory of the query tile: D / 64 column blocks of q_sub bytes
  int q_sub, q_box;           // (128 per row, rounded up to 1024; pairs: 128 rows); bytes a copy of one brings
  int part_rows;              // rows of a partial slot
  int max_split;              // partial slots
  float part_cost;            // tiles' worth of writing and joining a partial
  int* ws_head;               // listed split items of this call, the most rows one has, whether the list has gaps
  int4* ws_item;              // per split item: (tok0, rows, h, first slot), (pieces, 0, 0, 0)
  float2* ws_ml;              // [slot][row]: running max (log2 units), row sum
  float* ws_o;                // [slot][row][D]
  // With prefixes (shared.cu) a work list of n_groups + B: the groups' tokens
  // over their prefixes, which all of them see, then the requests over their own
  // keys.  Every row of a partial is a state row: whole items' first, then the
  // slots' rows from n_dense on.
  int n_groups;
  const int32_t *group_start, *prefix_table, *prefix_lengths;
  int64_t n_prefix_pages;
  int q_box_own;              // bytes a copy of one column block brings of a request's queries
  int n_dense;                // 2 * n_tok * Hq: [own keys, prefix][token][head]
  int4* ws_rows;              // [own keys, prefix][token][KV head]: a token's state rows, see the copying warp
};

struct Req {
  int start, nq, T;  // first token, new tokens, cached tokens
  int nqt, ntmax;    // query tiles, key tiles of the last one
};
struct PreReq : Req {
  int kind = 0;
  int g = 0, plen = 0;  // group, keys of its prefix
};
constexpr int kPrefix = 1;  // the tokens of a group over its prefix
constexpr int kBehind = 2;  // a request's own keys, behind a prefix that its group's tokens share
constexpr int kFull = 3;    // a request's keys, those of its prefix before its own
// Pairs, with prefixes: whether an entry's pieces are dealt out (several query tiles
// or a group's tokens read the same keys, at the same time if they can) or its items
// lie in the row of which each pair takes a stretch.
__device__ __forceinline__ bool dealt(const PreReq& r) { return r.kind == kPrefix || r.kind == kFull || r.nqt > 1; }
__device__ __forceinline__ bool dealt(const Req&) { return true; }
template <bool PRE>
using ReqOf = std::conditional_t<PRE, PreReq, Req>;

// Key tiles of query tile qt of a request: window tiles [lo, lo + n - nsink) after the sink tiles [0, nsink).
template <int KT>
__device__ __forceinline__ void tile_range(const PagedArgs& a, const Req& r, int qt, int& lo, int& nsink, int& n) {
  const int first = qt * a.tpt, m = min(a.tpt, r.nq - first);
  const int p_lo = max(0, r.T - r.nq + first);
  int p_hi = r.T - r.nq + first + m - 1;
  const int64_t cap = a.n_pages * a.page;
  if (p_hi >= cap) p_hi = static_cast<int>(cap) - 1;
  lo = nsink = n = 0;
  if (p_hi < 0 || m <= 0) return;
  if (a.W > 0) {
    lo = max(0, p_lo - a.W + 1) / KT;
    nsink = min((min(a.S, p_hi + 1) + KT - 1) / KT, lo);
  }
  n = nsink + max(0, p_hi / KT - lo + 1);
}

// Whether an earlier request has tokens past the first of request b; only
// possible where some request's offsets are not in order.
__device__ __noinline__ bool taken(const int32_t* q_start, int n_tok, int b, int first) {
  bool hit = false;
#pragma unroll 1
  for (int i = 0, s = q_start[0]; i < b; i++) {
    const int e = q_start[i + 1];
    hit |= s >= 0 && e > s && e <= n_tok && e > first;
    s = e;
  }
  return hit;
}

// A request whose offsets are not in order, or (looked for once *disorder is
// known) whose tokens an earlier one has, has none: the requests left are
// disjoint, so none writes another's rows and 32 bits count their work.
template <int KT>
__device__ __noinline__ Req request(const PagedArgs& a, int b, bool report, int* disorder, bool known) {
  Req r;
  if (b >= a.B) return Req{0, 0, 0, 0, 0};
  r.T = max(0, a.lengths[b]);
  if (a.q_start) {
    const int s = a.q_start[b], e = a.q_start[b + 1];
    bool bad = s < 0 || e < s || e > a.n_tok;
    if (bad) {
      *disorder = 1;  // (every writer's value)
      if (report) set_status(a.status, SKV_DEV_RANGE);
    }
    if (known && !bad && e > s && *disorder) bad = taken(a.q_start, a.n_tok, b, s);
    r.start = s;
    r.nq = bad ? 0 : e - s;
  } else {
    r.start = b;
    r.nq = 1;
  }
  if (r.nq > 0 && r.T > a.n_pages * a.page && report) set_status(a.status, SKV_DEV_RANGE);
  r.nqt = (r.nq + a.tpt - 1) / a.tpt;
  r.ntmax = 0;
  if (r.nqt > 0) {
    int lo, ns;
    tile_range<KT>(a, r, r.nqt - 1, lo, ns, r.ntmax);
    if (r.nqt > 1) {  // the last tile may hold fewer tokens, and so a tile less
      int n2;
      tile_range<KT>(a, r, r.nqt - 2, lo, ns, n2);
      r.ntmax = max(r.ntmax, n2);
    }
  }
  return r;
}

// Whether the requests [lo, hi) of a group go through the prefix each for itself:
// their query tiles then see the prefix's keys and their own in one pass, with no
// state rows to write and to join, but a request's last tile may be part empty
// where the group's tokens together would fill it.  Those tiles cost the prefix's
// key tiles; the state rows and the second pass over a query tile, about nine.
__device__ __noinline__ bool one_by_one(const PagedArgs& a, int lo, int hi, int key_tiles) {
  const int n = hi - lo;
  if (n <= 1) return true;
  if (!a.q_start) return false;
  const int first = a.q_start[lo], tiles = (a.q_start[hi] - first + a.tpt - 1) / a.tpt;
  if (2 * tiles < n) return false;  // (also many requests of few tokens)
  int each = 0;
  if (n <= 32) {
#pragma unroll 1
    for (int i = lo, s = first; i < hi; i++) {
      const int e = a.q_start[i + 1];
      each += (e - s + a.tpt - 1) / a.tpt;
      s = e;
    }
  } else {
    each = tiles + n / 2;
  }
  return static_cast<int64_t>(each - tiles) * key_tiles <= static_cast<int64_t>(9) * tiles;
}

// Entry i of a call with prefixes: group i's tokens over its prefix, or request
// i - n_groups over its own keys or, where its group's requests go one by one, the
// prefix and its own.  Where any offset or group boundary is out of order there are
// none (*disorder, once known).
template <int KT>
__device__ __noinline__ PreReq pre_request(const PagedArgs& a, int i, bool report, int* disorder, bool known) {
  PreReq r;
  r.start = r.nq = r.T = r.nqt = r.ntmax = 0;
  if (i >= a.n_groups + a.B) return r;
  const bool prefix = i < a.n_groups;
  const int b = i - a.n_groups;
  int lo = prefix ? a.group_start[i] : b, hi = prefix ? a.group_start[i + 1] : b + 1;  // requests
  bool bad = lo < 0 || hi < lo || hi > a.B;
  if (bad) lo = hi = 0;
  int s = lo, e = hi;
  if (a.q_start) {
    s = a.q_start[lo];
    e = a.q_start[hi];
    bad |= s < 0 || e < s || e > a.n_tok;
  }
  if (bad) {
    *disorder = 1;  // (every writer's value)
    if (report) set_status(a.status, SKV_DEV_RANGE);
  }
  if (bad || (known && *disorder)) return r;
  const int64_t cap = (prefix ? a.n_prefix_pages : a.n_pages) * a.page;
  r.T = max(0, prefix ? a.prefix_lengths[i] : a.lengths[b]);
  r.start = s;
  r.nq = e - s;
  if (r.nq > 0 && r.T > cap && report) set_status(a.status, SKV_DEV_RANGE);
  r.nqt = (r.nq + a.tpt - 1) / a.tpt;
  // every query tile sees a whole prefix; of its own keys a request's last tile the most
  r.ntmax = static_cast<int>((min(static_cast<int64_t>(r.T), cap) + KT - 1) / KT);
  if (prefix) {
    r.kind = kPrefix;
    r.g = i;
    r.plen = r.T;
    if (r.T == 0 || one_by_one(a, lo, hi, r.ntmax)) r.nq = r.nqt = 0;
  } else if (a.n_groups > 0) {  // the last group that begins at b or before
    int g = 0, end = a.n_groups;
    while (end - g > 1) {
      const int mid = (g + end) / 2;
      (a.group_start[mid] <= b ? g : end) = mid;
    }
    const int from = a.group_start[g], to = a.group_start[g + 1];
    // The group's boundaries index the offsets below, and nobody may have looked at
    // them yet: one outside [0, B] leaves the request without a prefix (the group's
    // own entry flags it).
    if (from >= 0 && from <= b && b < to && to <= a.B) {
      const int64_t pcap = a.n_prefix_pages * a.page;
      r.g = g;
      r.plen = max(0, a.prefix_lengths[g]);
      const int tiles = static_cast<int>((min(static_cast<int64_t>(r.plen), pcap) + KT - 1) / KT);
      if (r.plen > 0) r.kind = one_by_one(a, from, to, tiles) ? kFull : kBehind;
      if (r.kind == kFull) r.ntmax += tiles;
    }
  }
  if (r.nqt == 0) r.ntmax = 0;
  return r;
}

template <int KT, bool PRE>
__device__ __forceinline__ ReqOf<PRE> request_of(const PagedArgs& a, int b, bool report, int* disorder, bool known) {
  if constexpr (PRE)
    return pre_request<KT>(a, b, report, disorder, known);
  else
    return request<KT>(a, b, report, disorder, known);
}

}  // namespace
}  // namespace skv
