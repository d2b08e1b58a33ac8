// paged.cu -- attention of new tokens over a paged cache: a chunk of a
// prompt, a few drafted tokens or one token per request, causal, optionally
// through a sliding window with the first tokens kept visible.
//
// Token i of request b (n_b new tokens, T = lengths[b] in the cache, these
// included) stands at p = T - n_b + i and sees the keys t <= p that lie in the
// window (W == 0, or t > p - W) or among the first S:
//   out = sum_t softmax_t(scale q.k_t) v_t over the visible t; none: 0.
#include "common.cuh"

namespace skv {
namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;

struct PagedArgs {
  int B, n_tok, Hq, Hkv;
  const uint16_t* q;
  int64_t q_stride;
  const void *k_pool, *v_pool;
  const __half *k_scale, *v_scale;
  int64_t n_blocks;
  int page;
  const int32_t* block_table;
  int64_t n_pages;
  const int32_t *q_start, *lengths;
  int S, W;
  float scale_log2;
  uint16_t* out;
  int32_t* status;
};

// One CTA per (token, query head): warp w takes keys w, w + 4, ...; each lane
// holds D / 32 dims.  Online softmax per warp, the warps joined at the end.
template <int D, bool INT8>
__global__ void __launch_bounds__(kThreads) paged_kernel(const PagedArgs a) {
  constexpr int E = D / 32;
  __shared__ float so[kWarps][D], sm_m[kWarps], sm_l[kWarps];
  const int tok = blockIdx.x, g = blockIdx.y, h = g / (a.Hq / a.Hkv);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // Every row of work here is a dot product per key on the plain cores: right
  // for every case, bound by their instruction rate.
  int b = tok, start = tok, end = tok + 1;
  if (a.q_start) {
    if (tok == 0 && g == 0)
      for (int r = threadIdx.x; r < a.B; r += kThreads)
        if (a.q_start[r] < 0 || a.q_start[r + 1] < a.q_start[r] || a.q_start[r + 1] > a.n_tok)
          set_status(a.status, SKV_DEV_RANGE);
    int lo = 0, hi = a.B;  // last b with q_start[b] <= tok
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (a.q_start[mid] <= tok) lo = mid; else hi = mid;
    }
    b = lo;
    start = a.q_start[b];
    end = a.q_start[b + 1];
    if (tok < start || tok >= end) return;  // behind the last sequence: left as it was
  }
  const int T = a.lengths[b];
  const int p = T - (end - start) + (tok - start);
  float q[E], o[E], m = -INFINITY, l = 0.f;
  for (int e = 0; e < E; e++) {
    q[e] = bf16_bits_to_f32(a.q[tok * a.q_stride + static_cast<int64_t>(g) * D + E * lane + e]) * a.scale_log2;
    o[e] = 0.f;
  }
  const int w0 = a.W ? max(0, p - a.W + 1) : 0;
  for (int t = warp; t <= p; t += kWarps) {
    if (t >= a.S && t < w0) continue;
    const int64_t pg = t / a.page;
    const int64_t blk = pg < a.n_pages ? a.block_table[b * a.n_pages + pg] : -1;
    if (blk < 0 || blk >= a.n_blocks) {
      if (lane == 0) set_status(a.status, SKV_DEV_RANGE);
      continue;
    }
    const int64_t vec = (blk * a.page + t % a.page) * a.Hkv + h;
    float s = 0.f, v[E];
    for (int e = 0; e < E; e++) {
      const int64_t at = vec * D + E * lane + e;
      if (INT8) {
        s += q[e] * static_cast<const int8_t*>(a.k_pool)[at];
        v[e] = static_cast<const int8_t*>(a.v_pool)[at] * __half2float(a.v_scale[vec]);
      } else {
        s += q[e] * bf16_bits_to_f32(static_cast<const uint16_t*>(a.k_pool)[at]);
        v[e] = bf16_bits_to_f32(static_cast<const uint16_t*>(a.v_pool)[at]);
      }
    }
    for (int x = 16; x; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
    if (INT8) s *= __half2float(a.k_scale[vec]);
    const float mn = fmaxf(m, s);
    const float c = m == -INFINITY ? 0.f : exp2f(m - mn), w = exp2f(s - (mn == -INFINITY ? 0.f : mn));
    m = mn;
    l = l * c + w;
    for (int e = 0; e < E; e++) o[e] = o[e] * c + w * v[e];
  }
  for (int e = 0; e < E; e++) so[warp][E * lane + e] = o[e];
  if (lane == 0) {
    sm_m[warp] = m;
    sm_l[warp] = l;
  }
  __syncthreads();
  float M = -INFINITY, L = 0.f;
  for (int w = 0; w < kWarps; w++) M = fmaxf(M, sm_m[w]);
  for (int x = threadIdx.x; x < D; x += kThreads) {
    float acc = 0.f;
    L = 0.f;
    for (int w = 0; w < kWarps; w++) {
      const float f = sm_m[w] == -INFINITY ? 0.f : exp2f(sm_m[w] - M);
      L += f * sm_l[w];
      acc += f * so[w][x];
    }
    const __nv_bfloat16 r = __float2bfloat16_rn(L == 0.f ? 0.f : acc / L);
    a.out[(static_cast<int64_t>(tok) * a.Hq + g) * D + x] = *reinterpret_cast<const uint16_t*>(&r);
  }
}

}  // namespace
}  // namespace skv

using namespace skv;

SKV_EXPORT size_t skv_paged_attend_workspace_size(int B, int n_tok, int Hq, int Hkv, int d) {
  if (B < 1 || n_tok < 1 || Hkv < 1 || Hq < 1 || Hq % Hkv || Hq / Hkv > 128 || (d != 128 && d != 256)) return 0;
  return 16;
}

SKV_EXPORT int skv_paged_attend(int kv_kind, int B, int n_tok, int Hq, int Hkv, int d, const uint16_t* q,
                                int64_t q_stride, const void* k_pool, const void* v_pool, const uint16_t* k_scale,
                                const uint16_t* v_scale, int64_t n_pool_rows, int page, const int32_t* block_table,
                                int64_t n_pages, const int32_t* q_start, const int32_t* lengths, int S, int W,
                                float softmax_scale, uint16_t* out, void* workspace, size_t workspace_bytes,
                                int32_t* dev_status, void* stream) {
  if (kv_kind != SKV_KV_BF16 && kv_kind != SKV_KV_INT8) return SKV_EINVAL;
  if (B < 0 || B > 4096 || n_tok < 0 || Hkv < 1 || Hq < 1 || Hq % Hkv || S < 0 || W < 0 || n_pages < 0) return SKV_EINVAL;
  if ((d != 128 && d != 256) || Hq / Hkv > 128 || page < 8 || page % 8) return SKV_EUNSUPPORTED;
  if (B == 0 || n_tok == 0) return SKV_OK;
  if (!q || !k_pool || !v_pool || !block_table || !lengths || !out || n_pages < 1 || n_pool_rows < page)
    return SKV_EINVAL;
  if (kv_kind == SKV_KV_INT8 && (!k_scale || !v_scale)) return SKV_EINVAL;
  if (!q_start && n_tok != B) return SKV_EINVAL;
  if (!aligned16(q) || !aligned16(k_pool) || !aligned16(v_pool) || !aligned16(out) || q_stride % 8 ||
      q_stride < static_cast<int64_t>(Hq) * d)
    return SKV_EINVAL;
  if (!workspace || !aligned16(workspace) ||
      workspace_bytes < skv_paged_attend_workspace_size(B, n_tok, Hq, Hkv, d))
    return SKV_ENOMEM;
  PagedArgs a{B, n_tok, Hq, Hkv, q, q_stride, k_pool, v_pool, reinterpret_cast<const __half*>(k_scale),
              reinterpret_cast<const __half*>(v_scale), n_pool_rows / page, page, block_table, n_pages, q_start,
              lengths, S, W, softmax_scale * kLog2e, out, dev_status};
  const dim3 grid(n_tok, Hq);
  cudaStream_t st = as_stream(stream);
  if (d == 128 && kv_kind == SKV_KV_BF16)
    paged_kernel<128, false><<<grid, kThreads, 0, st>>>(a);
  else if (d == 128)
    paged_kernel<128, true><<<grid, kThreads, 0, st>>>(a);
  else if (kv_kind == SKV_KV_BF16)
    paged_kernel<256, false><<<grid, kThreads, 0, st>>>(a);
  else
    paged_kernel<256, true><<<grid, kThreads, 0, st>>>(a);
  return launch_status();
}
