// paged.cu -- attention of new tokens over a paged cache: the merge of cut
// requests and the C entry points; the attention kernel is in paged.cuh.
#include "paged.cuh"

namespace skv {
namespace {

// Joins the pieces of split items in piece order.  With few rows a block takes
// a row, its warps every eighth piece; with many a warp takes a row.  It is
// launched while the attention still writes what it reads, so none of that is
// declared read-only or unaliased: such loads could be moved ahead of the wait.
template <int D>
__global__ void __launch_bounds__(256) merge_kernel(const int* head, const int4* item, const float2* ml, const float* o,
                                                    int listable, int part_rows, int G, int Hq, uint16_t* out) {
  constexpr int E = D / 32;  // columns per lane: float4 f at 4 (lane + 32 f)
  constexpr int Q = kMaxPieces / 32;
  __shared__ __align__(16) float red[8][D];
  __shared__ float weight[8][kMaxPieces];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  // It lets nothing start early in its turn: kernels that read before they wait
  // count on everything but the kernel just before them being complete.
  grid_dependency_wait();  // launched early: the partials are complete from here on
  // Single CTAs list a split item at the CTA where it begins, so the list has
  // gaps: every warp closes it up for itself, in order, as masks of the used
  // entries (its loads go out with the head's).
  uint32_t used[Q];
  int pieces[Q];
#pragma unroll
  for (int i = 0; i < Q; i++) pieces[i] = lane + 32 * i < listable ? item[2 * (lane + 32 * i) + 1].x : 0;
  const int4 hd = *reinterpret_cast<const int4*>(head);
  const int listed = hd.x, rows = hd.y;
  const bool gaps = hd.z != 0;
  int n_items = gaps ? 0 : listed;
#pragma unroll
  for (int i = 0; i < Q; i++) {
    used[i] = __ballot_sync(0xffffffffu, lane + 32 * i < listed && pieces[i] > 0);
    n_items += gaps ? __popc(used[i]) : 0;
  }
  const int tasks = n_items * rows;
  // A block per row while there is one for each: four requests of 131072 tokens
  // (64 rows) 190 us, a warp per row 193.5; eight of 8 drafts (1024 rows) 115.5
  // against 109, two of 100 tokens 194.5 against 178.5.
  const bool wide = tasks <= static_cast<int>(gridDim.x);
  const int step = wide ? gridDim.x : gridDim.x * 8, first = wide ? blockIdx.x : blockIdx.x * 8 + warp;
  const int s0 = wide ? warp : 0, ds = wide ? 8 : 1;
#pragma unroll 1
  for (int w = first; w < tasks; w += step) {
    const int at = w / rows, row = w - at * rows;
    int it = at;
    if (gaps) {
      int left = at;
      uint32_t mask = 0;
#pragma unroll
      for (int i = 0; i < Q; i++) {
        const int n = __popc(used[i]);
        if (left >= 0 && left < n) {
          mask = used[i];
          it = 32 * i;
          const bool is = (mask >> lane & 1u) && __popc(mask & ((1u << lane) - 1u)) == left;
          it += __ffs(__ballot_sync(0xffffffffu, is)) - 1;
        }
        left -= n;
      }
    }
    const int4 x = item[2 * it], y = item[2 * it + 1];
    const int n = y.x;
    if (row >= x.y) continue;  // the same for the whole block where it takes a row
    auto slot_row = [&](int s) { return static_cast<int64_t>(s == 0 ? x.w : y.y + (s - 1) * y.z) * part_rows + row; };
    float2 v[Q];
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < Q; i++) {
      v[i] = make_float2(-INFINITY, 0.f);
      if (lane + 32 * i < n) v[i] = ml[slot_row(lane + 32 * i)];
      m = fmaxf(m, v[i].x);
    }
#pragma unroll
    for (int i = 16; i; i >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, i));
    // A piece without a visible key takes no part, and its O may be unwritten:
    // marked with a weight of -1.  One whose weight vanishes beside another's
    // does take part: what is not finite in it reaches the output.
    float den = 0.f;
    __syncwarp();
#pragma unroll
    for (int i = 0; i < Q; i++) {
      const bool none = v[i].x == -INFINITY && v[i].y == 0.f;
      const float f = none ? 0.f : exp2f(v[i].x - m);
      den += none ? 0.f : f * v[i].y;
      weight[warp][lane + 32 * i] = none ? -1.f : f;
    }
    __syncwarp();
#pragma unroll
    for (int i = 16; i; i >>= 1) den += __shfl_xor_sync(0xffffffffu, den, i);
    float acc[E];
#pragma unroll
    for (int e = 0; e < E; e++) acc[e] = 0.f;
#pragma unroll 8
    for (int s = s0; s < n; s += ds) {
      const float f = weight[warp][s];
      if (f < 0.f) continue;
      const float* src = o + slot_row(s) * D + 4 * lane;
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
    uint16_t* dst = out + (static_cast<int64_t>(x.x + row / G) * Hq + x.z * G + row % G) * D;
    if (wide) {
#pragma unroll
      for (int e = 0; e < E; e += 4)
        *reinterpret_cast<float4*>(&red[warp][4 * lane + 32 * e]) = make_float4(acc[e], acc[e + 1], acc[e + 2], acc[e + 3]);
      __syncthreads();
      if (threadIdx.x < D / 2) {
        float2 sum = make_float2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < 8; i++) {
          const float2 z = *reinterpret_cast<const float2*>(&red[i][2 * threadIdx.x]);
          sum.x += z.x;
          sum.y += z.y;
        }
        *reinterpret_cast<uint32_t*>(dst + 2 * threadIdx.x) = pack_bf16(sum.x * inv, sum.y * inv);
      }
      __syncthreads();
    } else {
#pragma unroll
      for (int e = 0; e < E; e += 4)
        *reinterpret_cast<uint2*>(dst + 4 * lane + 32 * e) =
            make_uint2(pack_bf16(acc[e] * inv, acc[e + 1] * inv), pack_bf16(acc[e + 2] * inv, acc[e + 3] * inv));
    }
  }
}

struct Layout {  // workspace
  int max_split, part_rows;
  size_t item, ml, o, total;
};

Layout layout(int n_tok, int G, int d, int ctas, int sms) {
  Layout w;
  if (sms > kMaxPieces) sms = kMaxPieces;
  w.max_split = ctas == 1 ? 2 * sms : kSplitPerPair * (sms / 2);
  w.part_rows = tile_rows(n_tok, G, ctas);
  w.item = 256;
  w.ml = w.item + static_cast<size_t>(w.max_split) * 2 * sizeof(int4);
  w.o = w.ml + ((static_cast<size_t>(w.max_split) * w.part_rows * sizeof(float2) + 255) & ~static_cast<size_t>(255));
  w.total = w.o + static_cast<size_t>(w.max_split) * w.part_rows * d * sizeof(float);
  return w;
}

template <int D, int CTAS, bool INT8>
int launch(const PagedArgs& a, const Maps<false>& maps, int smem, int sms, cudaStream_t st) {
  static std::atomic<int> configured[kMaxDevices];
  auto kernel = paged_kernel<D, CTAS, INT8, false>;
  if (smem_limit_once(configured, kernel, kMaxSmem) != SKV_OK) return SKV_ECUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((sms < kMaxPieces ? sms : kMaxPieces) / CTAS * CTAS, 1, 1);  // an item has a piece per CTA at most
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
  // Four blocks per SM: 64 ragged int8 requests 127.2 us with two, 122.4 with
  // four, 124.0 with six; 256 tokens at 262144 keys 587, 576, 576.
  cfg.gridDim = dim3(4 * sms, 1, 1);
  cfg.blockDim = dim3(256, 1, 1);
  cfg.dynamicSmemBytes = 0;
  cfg.numAttrs = 1;
  const int listable = a.max_split < kMaxPieces ? a.max_split : kMaxPieces;
  const int* head = a.ws_head;
  const int4* item = a.ws_item;
  const float2* ml = a.ws_ml;
  const float* o = a.ws_o;
  if (cudaLaunchKernelEx(&cfg, merge_kernel<D>, head, item, ml, o, listable, a.part_rows, a.G, a.Hkv * a.G, a.out) !=
      cudaSuccess) {
    cudaGetLastError();
    return SKV_ECUDA;
  }
  return SKV_OK;
}

template <int D, int CTAS>
int launch_kind(const PagedArgs& a, const Maps<false>& maps, bool int8, int smem, int sms, cudaStream_t st) {
  return int8 ? launch<D, CTAS, true>(a, maps, smem, sms, st) : launch<D, CTAS, false>(a, maps, smem, sms, st);
}

// CTA pairs where requests have more rows than a single CTA's query tile, which
// would read the cache twice.  Eight requests of 30000 tokens, rows 128 / 192
// each, single against pairs: bf16 of 256 dims 127 / 185 us against 126 / 119,
// int8 136 / 205 against 165 / 157; of 128 dims 90 / 112 against 106 / 96, int8
// 100 / 134 against 134 / 123.  The rule goes by the batch's mean, the lengths
// being on the device, so a mixed batch runs as one kind: 63 single tokens at
// 5000 keys and a chunk of 900 at 20000 (16 / 2 heads of 256) take 337 us as one
// bf16 call and 328 as two, 502 and 374 for int8 rows.
int ctas_for(int B, int n_tok, int G, bool single) {
  return !single && static_cast<int64_t>(n_tok) * G > static_cast<int64_t>(B) * kRows ? 2 : 1;
}

}  // namespace
}  // namespace skv

using namespace skv;

SKV_EXPORT size_t skv_paged_attend_workspace_size(int B, int n_tok, int Hq, int Hkv, int d) {
  if (B < 1 || n_tok < 1 || Hkv < 1 || Hq < 1 || Hq % Hkv || Hq / Hkv > 128 || (d != 128 && d != 256)) return 0;
  const int sms = sm_count() > 0 ? sm_count() : 152;
  const int G = Hq / Hkv;
  // Enough for every call of up to n_tok tokens: by the number of requests one
  // runs as pairs or not, but never with so few rows (ctas_for).
  const size_t one = layout(n_tok, G, d, 1, sms).total;
  if (static_cast<int64_t>(n_tok) * G <= kRows) return one;
  const size_t two = layout(n_tok, G, d, 2, sms).total;
  return one > two ? one : two;
}

SKV_EXPORT int skv_paged_attend(int kv_kind, int B, int n_tok, int Hq, int Hkv, int d, const uint16_t* q,
                                int64_t q_stride, const void* k_pool, const void* v_pool, const uint16_t* k_scale,
                                const uint16_t* v_scale, int64_t n_pool_rows, int page, const int32_t* block_table,
                                int64_t n_pages, const int32_t* q_start, const int32_t* lengths, int S, int W,
                                float softmax_scale, uint16_t* out, void* workspace, size_t workspace_bytes,
                                int32_t* dev_status, void* stream) {
  if (kv_kind != SKV_KV_BF16 && kv_kind != SKV_KV_INT8) return SKV_EINVAL;
  if (B < 0 || B > 4096 || n_tok < 0 || Hkv < 1 || Hq < 1 || Hq % Hkv || S < 0 || W < 0 || n_pages < 0)
    return SKV_EINVAL;
  if ((d != 128 && d != 256) || Hq / Hkv > 128 || page < 8 || page % 8) return SKV_EUNSUPPORTED;
  if (B == 0 || n_tok == 0) return SKV_OK;
  if (!q || !k_pool || !v_pool || !block_table || !lengths || !out || n_pages < 1 || n_pool_rows < page)
    return SKV_EINVAL;
  const bool int8 = kv_kind == SKV_KV_INT8;
  if (int8 && (!k_scale || !v_scale)) return SKV_EINVAL;
  if (!q_start && n_tok != B) return SKV_EINVAL;
  if (!aligned16(q) || !aligned16(k_pool) || !aligned16(v_pool) || !aligned16(out) || q_stride % 8 ||
      q_stride < static_cast<int64_t>(Hq) * d)
    return SKV_EINVAL;
  if (!(softmax_scale > 0.f) || softmax_scale > 2.0e38f) return SKV_EINVAL;  // in log2 units it is finite, too
  // 32-bit positions, tile coordinates and work-list counts
  if (n_pages > INT32_MAX / page || n_pages * page > INT32_MAX - 1024 || static_cast<int64_t>(n_tok) * Hq > INT32_MAX ||
      n_pool_rows > (static_cast<int64_t>(1) << 33))
    return SKV_EINVAL;
  if (W >= n_pages * page) W = 0;  // no window: a position does not reach it
  if (W > 1 << 30) return SKV_EINVAL;
  const int G = Hq / Hkv;
  const int ctas = ctas_for(B, n_tok, G, !q_start);
  const int tpt = ctas * (kRows / G);  // tokens per query tile
  const int64_t key_tiles = n_pages * page / keys_per_tile(d, ctas) + 1 + kItem;
  if (key_tiles > INT32_MAX / ((static_cast<int64_t>(B) + n_tok / tpt) * Hkv)) return SKV_EINVAL;
  if (!workspace || !aligned16(workspace) ||
      workspace_bytes < skv_paged_attend_workspace_size(B, n_tok, Hq, Hkv, d))
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
  a.S = S;
  a.W = W;
  a.scale_log2 = softmax_scale * kLog2e;
  a.out = out;
  a.status = dev_status;
  const Layout w = layout(n_tok, G, d, ctas, sms);
  unsigned char* ws = static_cast<unsigned char*>(workspace);
  a.part_rows = w.part_rows;
  a.max_split = w.max_split;
  a.part_cost = part_cost(w.part_rows, d, ctas);
  a.ws_head = reinterpret_cast<int*>(ws);
  a.ws_item = reinterpret_cast<int4*>(ws + w.item);
  a.ws_ml = reinterpret_cast<float2*>(ws + w.ml);
  a.ws_o = reinterpret_cast<float*>(ws + w.o);

  // The query rows that can hold a token (the products read 128 rows of each
  // column block; what they read past these is never used).
  const int q_toks = !q_start ? 1 : n_tok < a.tpc ? n_tok : a.tpc;  // per CTA
  a.q_box = q_toks * G * 128;
  a.thin = int8 && ctas == 1 && q_toks * G <= 32;
  a.q_sub = ctas == 2 ? kRows * 128 : (a.q_box + 1023) / 1024 * 1024;
  const Shared sh = shared_layout(d, ctas, int8, a.q_sub);
  a.q_bytes = sh.q_bytes;
  a.stages = sh.stages;
  a.staging = sh.staging;
  const int smem = sh.total;

  Maps<false> maps;
  if (!encode_pools(maps, k_pool, v_pool, int8, Hkv, d, n_pool_rows, ctas, a.rb) ||
      !encode_query(&maps.q, q, q_stride, n_tok, Hq, G, d, q_toks))
    return SKV_ECUDA;
  cudaStream_t st = as_stream(stream);
  int e;
  if (d == 128)
    e = ctas == 2 ? launch_kind<128, 2>(a, maps, int8, smem, sms, st)
                  : launch_kind<128, 1>(a, maps, int8, smem, sms, st);
  else
    e = ctas == 2 ? launch_kind<256, 2>(a, maps, int8, smem, sms, st)
                  : launch_kind<256, 1>(a, maps, int8, smem, sms, st);
  return e;
}
