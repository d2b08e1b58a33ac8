// shared.cu -- attention of new tokens of a batch whose requests share long
// prefixes: the tokens of all requests of a group attend to the group's prefix
// together, so that its rows are read once for all of them.
//
// Token i of request b, of group g with a prefix of P_g tokens, sees the whole
// prefix and of its request's own keys those up to its place.  The softmax over
// both falls into the parts' maxima m, sums l and weighted values o:
//   M = max(m_p, m_o),  out = (2^(m_p - M) o_p + 2^(m_o - M) o_o)
//                           / (2^(m_p - M) l_p + 2^(m_o - M) l_o).
//
// Both parts run in one launch of the kernel of paged.cuh, as one work list:
// first the groups, each a request whose tokens all see every key of the
// prefix, then the requests over their own keys.  Pieces and whole items leave
// fp32 state rows (m, l, o) that merge_kernel joins, the prefix's first; a
// request without a prefix whose keys are not cut writes its output directly.
// Chunks fill query tiles by themselves: their requests take the prefix's keys
// before their own, one by one (see there), and leave nothing to join.
//
// What bounds it, and what it measured (bf16 product rate 1916 TFLOP/s, copy rate
// 6.79 TB/s):
//  - eight tokens behind 250000, int8 rows of 256 dims (528 MB): 143 us, 54 % of the
//    copy rate.  No pipe is full (issue 60 %, ALU 53 %, tensor 42 %): the widening of
//    a tile, its products from shared memory and its softmax take some 2 K clocks
//    each and are handed from one to the next.  With the widening cut to a move the
//    call takes 129 us, with neither widening nor softmax 122.
//  - 80 drafts behind 60000, int8 rows of 128 dims: 148 us.  The widening warps' chain
//    (alone 118 us) and the softmax warps' (alone 134) share issue slots, and a step
//    of one that gets shorter is mostly hidden by the other.
//  - 64 tokens behind 131072, bf16 rows of 256 dims: 102 us, 1.35 PFLOP/s, of one batch
//    again and again, 112 us (1.23) of another batch each call; long tiles take 2.3 K
//    clocks where the products take 2.0 K, the requests' own keys and the merge the
//    rest.
//  - 16 chunks of 256 tokens behind 32768: 1.26 to 1.29 ms, 1.71 to 1.76 PFLOP/s, the
//    power limit.
//  - 40 tokens, 5 prefixes, bf16 rows of 128 dims (236 MB): 57 to 63 us; memory, behind
//    the launch, the plan and the merge.
//  - small calls (eight tokens behind 2000: 17 us): what follows one another.
// Where it pays: what it saves is the reading of a prefix once per request, what it
// costs a second item and a merge of state rows per request.  40 single tokens in
// five groups, up to 5000 keys of their own, int8 rows of 256 dims, against the paged
// attention with the prefixes' pages in every table: behind 500 keys 46.5 / 45.8 us,
// 5000 64 / 134, 50000 207 / 990; 64 in pairs behind 500 74 / 63, 5000 163 / 199.
// (Several groups get the layout of a full query tile, as q_start does.)
#include "paged.cuh"

namespace skv {
namespace {

// Joins the state rows of each token and head, the prefix's first.  Launched
// early, as the merge of paged.cu, and for the same reasons nothing here is
// declared read-only and nothing starts early behind it.
//
// Bound by what follows one another: descriptors, maxima and sums, values.  A block
// takes every gridDim-th row, reads their descriptors at once, lists those that are
// to be joined (most of a chunk's were written directly, and the others lie side by
// side) and shares its warps out among them: 5 questions of up to 333 tokens 53 us,
// with warps shared out among all rows 62.5; 64 samples 102, with a warp per row 110.
constexpr int kMergeWarps = 16;
constexpr int kMergeRows = 128;  // listed at once
template <int D>
__global__ void __launch_bounds__(32 * kMergeWarps, 2)
    merge_kernel(const int* head, const int4* rows, const float2* ml, const float* o, const int32_t* q_start, int B,
                 int n_tok, int Hkv, int G, uint16_t* out) {
  constexpr int E = D / 32;  // columns per lane: float4 f at 4 (lane + 32 f)
  constexpr int Q = 2 * kMaxPieces / 32;
  __shared__ __align__(16) float red[kMergeWarps][D];
  __shared__ float weight[kMergeWarps][2 * kMaxPieces];
  __shared__ int4 own[kMergeRows], pre[kMergeRows];
  __shared__ int row[kMergeRows], listed[kMergeRows / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  grid_dependency_wait();
  const int Hq = Hkv * G, tasks = n_tok * Hq;
  const int disorder = head[0];
  const int first_tok = q_start ? q_start[0] : 0, end_tok = q_start ? q_start[B] : n_tok;
#pragma unroll 1
  for (int64_t i0 = blockIdx.x; i0 < tasks; i0 += static_cast<int64_t>(kMergeRows) * gridDim.x) {
    int4 x = make_int4(0, 0, 0, 0), y = x;
    const int64_t at = i0 + static_cast<int64_t>(threadIdx.x) * gridDim.x;
    if (threadIdx.x < kMergeRows && at < tasks) {
      const int tok = static_cast<int>(at) / Hq, h = (static_cast<int>(at) - tok * Hq) / G;
      x = rows[static_cast<int64_t>(tok) * Hkv + h];
      y = rows[(static_cast<int64_t>(n_tok) + tok) * Hkv + h];
      if (disorder || tok < first_tok || tok >= end_tok) x.x = 0;  // padding: its rows were not listed
    }
    const uint32_t live = __ballot_sync(0xffffffffu, (x.x & (kHasPrefix - 1)) > 0);  // the others were written directly
    if (lane == 0 && warp < kMergeRows / 32) listed[warp] = __popc(live);
    __syncthreads();
    int n_rows = 0, mine = 0;
#pragma unroll
    for (int i = 0; i < kMergeRows / 32; i++) {
      mine += i < warp ? listed[i] : 0;
      n_rows += listed[i];
    }
    if (live >> lane & 1u) {
      mine += __popc(live & ((1u << lane) - 1u));
      own[mine] = x;
      pre[mine] = y;
      row[mine] = static_cast<int>(at);
    }
    __syncthreads();
    int team = kMergeWarps;  // warps to a row
    while (team > 1 && n_rows * team > kMergeWarps) team >>= 1;
    const int s0 = warp & (team - 1);
#pragma unroll 1
    for (int r = warp / team; r < n_rows || team > 1; r += kMergeWarps / team) {
      const bool there = r < n_rows;
      x = there ? own[r] : make_int4(0, 0, 0, 0);
      y = there ? pre[r] : x;
      const int w = there ? row[r] : 0, g = w % G;
      const int n_own = min(x.x & (kHasPrefix - 1), kMaxPieces), n_pre = x.x & kHasPrefix ? min(y.x, kMaxPieces) : 0;
      const int n = n_pre + n_own;
      auto row_of = [&](int s) -> int64_t {
        if (s < n_pre) return g + (s == 0 ? y.y : y.z + (s - 1) * y.w);
        s -= n_pre;
        return g + (s == 0 ? x.y : x.z + (s - 1) * x.w);
      };
      float2 v[Q];
      float m = -INFINITY;
#pragma unroll
      for (int i = 0; i < Q; i++) {
        v[i] = make_float2(-INFINITY, 0.f);
        if (lane + 32 * i < n) v[i] = ml[row_of(lane + 32 * i)];
        m = fmaxf(m, v[i].x);
      }
#pragma unroll
      for (int i = 16; i; i >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, i));
      // One without a visible key takes no part, and its o may be unwritten:
      // marked with a weight of -1.  One whose weight vanishes beside another's
      // does take part: what is not finite in it reaches the output.
      float den = 0.f;
      __syncwarp();
#pragma unroll
      for (int i = 0; i < Q; i++) {
        const bool none = v[i].x == -INFINITY && v[i].y == 0.f;
        const float f = none ? 0.f : exp2f(v[i].x - m);
        den += none ? 0.f : f * v[i].y;
        if (32 * i < n) weight[warp][lane + 32 * i] = none ? -1.f : f;
      }
      __syncwarp();
#pragma unroll
      for (int i = 16; i; i >>= 1) den += __shfl_xor_sync(0xffffffffu, den, i);
      float acc[E];
#pragma unroll
      for (int e = 0; e < E; e++) acc[e] = 0.f;
#pragma unroll 8
      for (int s = s0; s < n; s += team) {
        const float f = weight[warp][s];
        if (f < 0.f) continue;
        const float* src = o + row_of(s) * D + 4 * lane;
#pragma unroll
        for (int e = 0; e < E; e += 4) {
          const float4 z = *reinterpret_cast<const float4*>(src + 32 * e);
          acc[e] += f * z.x;
          acc[e + 1] += f * z.y;
          acc[e + 2] += f * z.z;
          acc[e + 3] += f * z.w;
        }
      }
      const float inv = den != 0.f ? 1.f / den : 0.f;
      uint16_t* dst = out + static_cast<int64_t>(w) * D;
      if (team == 1) {
#pragma unroll
        for (int e = 0; e < E; e += 4)
          *reinterpret_cast<uint2*>(dst + 4 * lane + 32 * e) =
              make_uint2(pack_bf16(acc[e] * inv, acc[e + 1] * inv), pack_bf16(acc[e + 2] * inv, acc[e + 3] * inv));
        continue;
      }
#pragma unroll
      for (int e = 0; e < E; e += 4)
        *reinterpret_cast<float4*>(&red[warp][4 * lane + 32 * e]) = make_float4(acc[e], acc[e + 1], acc[e + 2], acc[e + 3]);
      __syncthreads();
      for (int c = 32 * s0 + lane; there && c < D / 2; c += 32 * team) {
        float2 sum = make_float2(0.f, 0.f);
        for (int i = 0; i < team; i++) {
          const float2 r2 = *reinterpret_cast<const float2*>(&red[warp - s0 + i][2 * c]);
          sum.x += r2.x;
          sum.y += r2.y;
        }
        *reinterpret_cast<uint32_t*>(dst + 2 * c) = pack_bf16(sum.x * inv, sum.y * inv);
      }
      break;  // a team has one row at most
    }
    __syncthreads();
  }
}

// ---- host ------------------------------------------------------------------------

struct Layout {  // workspace
  int max_split, part_rows;
  int64_t n_dense;  // state rows before the slots'
  size_t rows, ml, o, total;
};

Layout layout(int n_tok, int Hkv, int G, int d, int ctas, int sms) {
  Layout w;
  if (sms > kMaxPieces) sms = kMaxPieces;
  w.max_split = ctas == 1 ? 2 * sms : (kSplitPerPair + 2) * (sms / 2);  // (pieces dealt out, and cut by stretches)
  w.part_rows = tile_rows(n_tok, G, ctas);
  w.n_dense = static_cast<int64_t>(2) * n_tok * Hkv * G;
  const size_t state = static_cast<size_t>(w.n_dense) + static_cast<size_t>(w.max_split) * w.part_rows;
  auto up = [](size_t x) { return (x + 255) & ~static_cast<size_t>(255); };
  w.rows = 256;
  w.ml = w.rows + up(static_cast<size_t>(2) * n_tok * Hkv * sizeof(int4));
  w.o = w.ml + up(state * sizeof(float2));
  w.total = w.o + state * d * sizeof(float);
  return w;
}

// CTA pairs or single CTAs.  Requests of few tokens: a pair spends as long on
// their own keys as a single CTA, so pairs pay only where long prefixes outweigh
// that and a single CTA's tile of 256 dims asks more of L2 than it gives.  64
// tokens of 16 / 2 heads of 256, 100 keys of their own, single against pairs, behind
// 8000 / 32000 / 100000 tokens: bf16 28 / 47 / 139 us against 35 / 49 / 84, int8 33 /
// 64 / 157 against 42 / 62 / 120; of 32 / 8 heads of 128 behind 32000: bf16 63 against
// 81, int8 91 against 120.  The prefixes' lengths are on the device; their table's
// width stands for them.
// The rule for 128 dims leaves long prefixes to single CTAs, too: 64 requests of 1 / 5 /
// 16 tokens of 32 / 8 heads, single against pairs, bf16 behind 8000 39 / 80 / 179 us
// against 64 / 99 / 181, behind 32000 69 / 182 / 540 against 90 / 196 / 497, behind
// 100000 140 / 546 / 1880 against 142 / 465 / 1355.
// Else by the query tiles of an average group (without groups, request) that each
// CTA takes, a pair's being two, weighed by what they cost: 192 rows, two tiles or a
// pair, over 30000 keys took 185 / 119 us (bf16 rows of 256 dims), 205 / 157 (int8),
// 112 / 96 and 134 / 123 (128 dims).  All tokens count as the groups', so a batch of
// which few requests are in a group may run as pairs where single CTAs would do: 2
// requests behind 8000 and 62 alone with 4000 keys, 20 tokens each of 32 / 8 heads of
// 128, single against pairs 199 / 264 us (bf16), 237 / 358 (int8); 40 tokens each 373 /
// 280 and 440 / 380.
int ctas_for(int B, int n_groups, int n_tok, int d, int G, bool int8, bool single, int64_t prefix_keys) {
  if (n_groups == 0 && single) return 1;
  const bool few = static_cast<int64_t>(n_tok) * G <= static_cast<int64_t>(B) * (kRows / 2);
  if (n_groups > 0 && few && (d == 128 || prefix_keys < 32768)) return 1;
  const int n = n_groups > 0 ? n_groups : B, toks = (n_tok + n - 1) / n, tpc = kRows / G;
  const float one = static_cast<float>((toks + tpc - 1) / tpc), two = 2.f * ((toks + 2 * tpc - 1) / (2 * tpc));
  return one * (d == 256 ? (int8 ? 1.3f : 1.55f) : int8 ? 1.09f : 1.17f) <= two ? 1 : 2;
}

template <int D, int CTAS, bool INT8>
int launch(const PagedArgs& a, const Maps<true>& maps, int smem, int sms, cudaStream_t st) {
  static std::atomic<int> configured[kMaxDevices];
  auto kernel = paged_kernel<D, CTAS, INT8, true>;
  if (smem_limit_once(configured, kernel, kMaxSmem) != SKV_OK) return SKV_ECUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((sms < kMaxPieces ? sms : kMaxPieces) / CTAS * CTAS, 1, 1);
  cfg.blockDim = dim3(kThreads<INT8>, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = CTAS;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  if (cudaLaunchKernelEx(&cfg, kernel, maps, a) != cudaSuccess) {
    cudaGetLastError();
    return SKV_ECUDA;
  }
  cfg.gridDim = dim3(2 * sms, 1, 1);
  cfg.blockDim = dim3(32 * kMergeWarps, 1, 1);
  cfg.dynamicSmemBytes = 0;
  cfg.numAttrs = 1;
  const int* head = a.ws_head;
  const int4* rows = a.ws_rows;
  const float2* ml = a.ws_ml;
  const float* o = a.ws_o;
  if (cudaLaunchKernelEx(&cfg, merge_kernel<D>, head, rows, ml, o, a.q_start, a.B, a.n_tok, a.Hkv, a.G, a.out) !=
      cudaSuccess) {
    cudaGetLastError();
    return SKV_ECUDA;
  }
  return SKV_OK;
}

template <int D, int CTAS>
int launch_kind(const PagedArgs& a, const Maps<true>& maps, bool int8, int smem, int sms, cudaStream_t st) {
  return int8 ? launch<D, CTAS, true>(a, maps, smem, sms, st) : launch<D, CTAS, false>(a, maps, smem, sms, st);
}

}  // namespace
}  // namespace skv

using namespace skv;

SKV_EXPORT size_t skv_shared_attend_workspace_size(int B, int n_groups, int n_tok, int Hq, int Hkv, int d) {
  if (B < 1 || n_groups < 0 || n_tok < 1 || Hkv < 1 || Hq < 1 || Hq % Hkv || Hq / Hkv > 128 || (d != 128 && d != 256) ||
      static_cast<int64_t>(n_tok) * Hq >= 1 << 29)
    return 0;
  const int sms = sm_count() > 0 ? sm_count() : 152;
  const int G = Hq / Hkv;
  // Enough for every call of up to n_tok tokens: by the number of groups one
  // runs as pairs or not, but never with so few rows (ctas_for).
  const size_t one = layout(n_tok, Hkv, G, d, 1, sms).total;
  if (static_cast<int64_t>(n_tok) * G <= kRows) return one;
  const size_t two = layout(n_tok, Hkv, G, d, 2, sms).total;
  return one > two ? one : two;
}

SKV_EXPORT int skv_shared_attend(int kv_kind, int B, int n_tok, int Hq, int Hkv, int d, const uint16_t* q,
                                 int64_t q_stride, const void* k_pool, const void* v_pool, const uint16_t* k_scale,
                                 const uint16_t* v_scale, int64_t n_pool_rows, int page, int n_groups,
                                 const int32_t* group_start, const int32_t* prefix_table, int64_t n_prefix_pages,
                                 const int32_t* prefix_lengths, const int32_t* block_table, int64_t n_pages,
                                 const int32_t* q_start, const int32_t* lengths, float softmax_scale, uint16_t* out,
                                 void* workspace, size_t workspace_bytes, int32_t* dev_status, void* stream) {
  if (kv_kind != SKV_KV_BF16 && kv_kind != SKV_KV_INT8) return SKV_EINVAL;
  static_assert(kMaxEntries >= 2 * 4096, "requests and groups");
  if (B < 0 || B > 4096 || n_tok < 0 || Hkv < 1 || Hq < 1 || Hq % Hkv || n_groups < 0 || n_groups > 4096 || n_pages < 0 ||
      n_prefix_pages < 0)
    return SKV_EINVAL;
  if ((d != 128 && d != 256) || Hq / Hkv > 128 || page < 8 || page % 8) return SKV_EUNSUPPORTED;
  if (B == 0 || n_tok == 0) return SKV_OK;
  if (!q || !k_pool || !v_pool || !block_table || !lengths || !out || n_pages < 1 || n_pool_rows < page)
    return SKV_EINVAL;
  if (n_groups > 0 && (!group_start || !prefix_table || !prefix_lengths || n_prefix_pages < 1)) return SKV_EINVAL;
  const bool int8 = kv_kind == SKV_KV_INT8;
  if (int8 && (!k_scale || !v_scale)) return SKV_EINVAL;
  if (!q_start && n_tok != B) return SKV_EINVAL;
  if (!aligned16(q) || !aligned16(k_pool) || !aligned16(v_pool) || !aligned16(out) || q_stride % 8 ||
      q_stride < static_cast<int64_t>(Hq) * d)
    return SKV_EINVAL;
  if (!(softmax_scale > 0.f) || softmax_scale > 2.0e38f) return SKV_EINVAL;  // in log2 units it is finite, too
  // 32-bit positions, tile coordinates, state rows and work-list counts
  const int64_t most_pages = n_groups > 0 && n_prefix_pages > n_pages ? n_prefix_pages : n_pages;
  if (most_pages > INT32_MAX / page || most_pages * page > INT32_MAX - 1024 ||
      static_cast<int64_t>(n_tok) * Hq >= 1 << 29 || n_pool_rows > (static_cast<int64_t>(1) << 33))
    return SKV_EINVAL;
  const int G = Hq / Hkv;
  const int ctas = ctas_for(B, n_groups, n_tok, d, G, int8, !q_start, n_groups > 0 ? n_prefix_pages * page : 0);
  const int tpt = ctas * (kRows / G);  // tokens per query tile
  const int kt = keys_per_tile(d, ctas);
  const int64_t pre_tiles = n_groups > 0 ? n_prefix_pages * page / kt + 1 + kRowItem : 0;
  const int64_t own_tiles = pre_tiles + n_pages * page / kt + 1 + kRowItem;  // a request's with its prefix before them
  const int64_t own_items = (static_cast<int64_t>(B) + n_tok / tpt) * Hkv;
  const int64_t pre_items = n_groups > 0 ? (static_cast<int64_t>(n_groups) + n_tok / tpt) * Hkv : 0;
  if (own_tiles > INT32_MAX / own_items || (pre_items > 0 && pre_tiles > (INT32_MAX - own_tiles * own_items) / pre_items))
    return SKV_EINVAL;
  if (!workspace || !aligned16(workspace) ||
      workspace_bytes < skv_shared_attend_workspace_size(B, n_groups, n_tok, Hq, Hkv, d))
    return SKV_ENOMEM;
  const int sms = sm_count();
  if (sms <= 1 || !encode_fn()) return SKV_ECUDA;

  PagedArgs a{};
  a.B = B;
  a.n_tok = n_tok;
  a.Hkv = Hkv;
  a.G = G;
  a.tpc = kRows / G;
  a.tpt = tpt;
  a.v_pool = int8 ? nullptr : static_cast<const uint16_t*>(v_pool);
  a.k_scale = reinterpret_cast<const __half*>(k_scale);
  a.v_scale = reinterpret_cast<const __half*>(v_scale);
  a.n_blocks = n_pool_rows / page;
  set_page(a, page);
  a.block_table = block_table;
  a.n_pages = n_pages;
  a.q_start = q_start;
  a.lengths = lengths;
  a.n_groups = n_groups;
  a.group_start = group_start;
  a.prefix_table = prefix_table;
  a.prefix_lengths = prefix_lengths;
  a.n_prefix_pages = n_prefix_pages;
  a.scale_log2 = softmax_scale * kLog2e;
  a.out = out;
  a.status = dev_status;
  const Layout w = layout(n_tok, Hkv, G, d, ctas, sms);
  if (w.n_dense + static_cast<int64_t>(w.max_split + 2) * w.part_rows > INT32_MAX) return SKV_EINVAL;
  unsigned char* ws = static_cast<unsigned char*>(workspace);
  a.n_dense = static_cast<int>(w.n_dense);
  a.part_rows = w.part_rows;
  a.max_split = w.max_split;
  a.part_cost = part_cost(w.part_rows, d, ctas);
  a.ws_head = reinterpret_cast<int*>(ws);
  a.ws_rows = reinterpret_cast<int4*>(ws + w.rows);
  a.ws_ml = reinterpret_cast<float2*>(ws + w.ml);
  a.ws_o = reinterpret_cast<float*>(ws + w.o);

  // The query rows that can hold a token: of a group, and of a request.
  const int toks = n_tok < a.tpc ? n_tok : a.tpc, own_toks = q_start ? toks : 1;
  const int most_toks = n_groups > 0 ? toks : own_toks;  // per CTA
  a.q_box = most_toks * G * 128;
  a.q_box_own = own_toks * G * 128;
  a.thin = !int8 || ctas == 2 ? 0 : most_toks * G <= 32 ? 1 : most_toks * G <= 64 ? 2 : 0;
  a.q_sub = ctas == 2 ? kRows * 128 : (a.q_box + 1023) / 1024 * 1024;
  const Shared sh = shared_layout(d, ctas, int8, a.q_sub);
  a.q_bytes = sh.q_bytes;
  a.stages = sh.stages;
  a.staging = sh.staging;

  Maps<true> maps;
  if (!encode_pools(maps, k_pool, v_pool, int8, Hkv, d, n_pool_rows, ctas, a.rb) ||
      !encode_query(&maps.q, q, q_stride, n_tok, Hq, G, d, most_toks) ||
      !encode_query(&maps.q_own, q, q_stride, n_tok, Hq, G, d, own_toks))
    return SKV_ECUDA;
  cudaStream_t st = as_stream(stream);
  if (d == 128)
    return ctas == 2 ? launch_kind<128, 2>(a, maps, int8, sh.total, sms, st)
                     : launch_kind<128, 1>(a, maps, int8, sh.total, sms, st);
  return ctas == 2 ? launch_kind<256, 2>(a, maps, int8, sh.total, sms, st)
                   : launch_kind<256, 1>(a, maps, int8, sh.total, sms, st);
}
