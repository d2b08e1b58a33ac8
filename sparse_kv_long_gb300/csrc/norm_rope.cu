// norm_rope.cu -- the step between a layer's projections and its attention:
// queries and keys normed per head and rotated by position, keys and values
// appended to the (paged) cache, in one pass over the projections.
//
// Per head x of d values at position p:
//   y = x * rsqrt(mean(x^2) + eps) * w                           (fp32)
//   z = y, except in dims [0, rot): the pair (a, b) of frequency f becomes
//       (a cos t - b sin t, b cos t + a sin t),  t = p * inv_freq[f]
//   q_out = bf16(z); a key is bf16(z), then the cache's row encoding.
//
// The angle.  A position of a million at frequency 1 needs t mod 2 pi to 1e-7
// of a turn: 45 bits.  inv_freq / 2 pi (fp64, once per thread) is kept as a
// 64-bit fixed-point fraction of a turn; p times it modulo 2^64 is the angle
// modulo one turn, exactly as unsigned integers wrap, and its top 32 bits go
// to sincospif.  Error: 2^-26 of a turn from the fp32 argument, plus
// |p| * inv_freq / 2 pi * 2^-53 turns from the fp64 quotient.
//
// Bound: memory.  Every value is read once and written once, 16 bytes per
// lane; d / 8 lanes share a head, so a head's sum is a shuffle reduction and
// no value passes through shared memory.  A warp takes a token's heads one
// after the other and computes the token's sines once; with few tokens a
// token's heads are spread over several warps instead (launch rule below).
#include "common.cuh"

namespace skv {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kBatch = 4;  // heads per lane group whose loads are in flight together

struct NormArgs {
  int64_t n_tok;
  int Hq, Hkv, rot;
  int slots;        // heads handled per token: those of q, then of k, then of v that are given
  int slots_q, slots_k;
  int chunk, chunks;  // heads per work item, work items per token
  const uint16_t *q, *k, *v;
  int64_t q_stride, k_stride, v_stride;
  const float *q_weight, *k_weight;
  float eps;
  const int32_t* positions;
  const float* inv_freq;
  uint16_t* q_out;
  const int64_t* out_rows;
  int64_t n_pool_rows;
  void *k_pool, *v_pool;
  __half *k_scale, *v_scale;
  int32_t* status;
};

__device__ __forceinline__ void unpack8(const uint4& r, float (&x)[8]) {
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int e = 0; e < 4; e++) {
    x[2 * e] = __uint_as_float(w[e] << 16);
    x[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
  }
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// One lane's 8 values of an int8 row: scale = fp16(max|x| / 127) over the
// head's lanes, codes = rint(x / scale), as skv_quantize_int8_rows.
template <int LPH>
__device__ __forceinline__ void store_int8(const uint4& bits, int8_t* codes, __half* scale, bool write, bool first) {
  float x[8];
  unpack8(bits, x);
  float m = 0.f;
#pragma unroll
  for (int e = 0; e < 8; e++) m = fmaxf(m, fabsf(x[e]));
#pragma unroll
  for (int o = LPH / 2; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  const __half sh = __float2half_rn(__fdiv_rn(m, 127.f));
  const float s = __half2float(sh);
  uint32_t w[2] = {0u, 0u};
  if (s != 0.f) {
#pragma unroll
    for (int e = 0; e < 8; e++)
      w[e >> 2] |= static_cast<uint32_t>(rint_clamp(__fdiv_rn(x[e], s), -127, 127) & 255) << (8 * (e & 3));
  }
  if (write) {
    *reinterpret_cast<uint2*>(codes) = make_uint2(w[0], w[1]);
    if (first) *scale = sh;
  }
}

template <int D, bool INTER, bool INT8>
__global__ void __launch_bounds__(kThreads) norm_rope_kernel(const NormArgs a) {
  constexpr int LPH = D / 8;    // lanes per head
  constexpr int HPW = 32 / LPH;  // heads a warp takes at once
  constexpr int NF = INTER ? 4 : 8;  // frequencies per lane
  __shared__ __align__(16) float sw[2][D];
  for (int x = threadIdx.x; x < D; x += kThreads) {
    sw[0][x] = a.q_weight ? a.q_weight[x] : 1.f;
    sw[1][x] = a.k_weight ? a.k_weight[x] : 1.f;
  }
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int sub = lane % LPH, grp = lane / LPH;
  const int x0 = 8 * sub;  // this lane's dims x0 .. x0 + 7 of its head
  const bool rotated = x0 < a.rot;
  const int half = a.rot / 2;
  const bool low = x0 < half;  // half-split pairs: this lane holds the first member
  const int partner = INTER ? lane : (rotated ? (low ? lane + half / 8 : lane - half / 8) : lane);
  const int px0 = INTER || !rotated ? x0 : (low ? x0 + half : x0 - half);
  uint64_t turn[NF];  // inv_freq / 2 pi as a 64-bit fraction of a turn
#pragma unroll
  for (int e = 0; e < NF; e++) {
    turn[e] = 0;
    if (rotated) {
      const int f = INTER ? x0 / 2 + e : (low ? x0 : x0 - half) + e;
      const double t = static_cast<double>(a.inv_freq[f]) * 0.15915494309189535;  // 1 / (2 pi)
      const double frac = t - floor(t);
      turn[e] = static_cast<uint64_t>(frac * 18446744073709551616.0);  // 2^64; frac < 1
    }
  }
  __syncthreads();

  const int64_t items = a.n_tok * a.chunks;
  const int64_t step = static_cast<int64_t>(gridDim.x) * kWarps;
  for (int64_t item = static_cast<int64_t>(blockIdx.x) * kWarps + warp; item < items; item += step) {
    const int64_t tok = item / a.chunks;
    const int s0 = static_cast<int>(item - tok * a.chunks) * a.chunk;
    const int s1 = min(a.slots, s0 + a.chunk);
    const int64_t pos = a.positions[tok];
    int64_t row = tok;
    if (a.out_rows) row = a.out_rows[tok];
    const bool bad = row >= a.n_pool_rows;
    if (bad && s1 > a.slots_q && lane == 0) set_status(a.status, SKV_DEV_RANGE);
    const bool keep = row >= 0 && !bad;
    float co[NF], si[NF];
    bool have_angles = false;

    for (int sb = s0; sb < s1; sb += HPW * kBatch) {
      uint4 raw[kBatch];
      // every load of the batch first
#pragma unroll
      for (int u = 0; u < kBatch; u++) {
        const int s = sb + u * HPW + grp;
        raw[u] = make_uint4(0u, 0u, 0u, 0u);
        if (s < s1) {
          const uint16_t* src;
          if (s < a.slots_q)
            src = a.q + tok * a.q_stride + static_cast<int64_t>(s) * D;
          else if (s < a.slots_q + a.slots_k)
            src = a.k + tok * a.k_stride + static_cast<int64_t>(s - a.slots_q) * D;
          else
            src = a.v + tok * a.v_stride + static_cast<int64_t>(s - a.slots_q - a.slots_k) * D;
          raw[u] = ld_stream16(src + x0);
        }
      }
      if (!have_angles) {  // the sines overlap the first batch's loads
        have_angles = true;
#pragma unroll
        for (int e = 0; e < NF; e++) {
          const uint64_t t = static_cast<uint64_t>(pos) * turn[e];
          const float h = static_cast<float>(static_cast<int32_t>(t >> 32)) * 4.656612873077393e-10f;  // 2^-31
          sincospif(h, &si[e], &co[e]);
        }
      }
#pragma unroll
      for (int u = 0; u < kBatch; u++) {
        const int s = sb + u * HPW + grp;
        if (sb + u * HPW >= s1) break;  // uniform in the warp
        const bool live = s < s1;
        const bool is_q = s < a.slots_q, is_v = s >= a.slots_q + a.slots_k;
        const int h = is_q ? s : (is_v ? s - a.slots_q - a.slots_k : s - a.slots_q);
        uint4 z = raw[u];
        // A warp of one head (D = 256) skips this for a value; where heads
        // share a warp all lanes take part in the shuffles.
        if (HPW > 1 || !is_v) {
          float x[8];
          unpack8(raw[u], x);
          float ss = 0.f;
#pragma unroll
          for (int e = 0; e < 8; e++) ss = fmaf(x[e], x[e], ss);
#pragma unroll
          for (int o = LPH / 2; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
          const bool normed = is_q ? a.q_weight != nullptr : a.k_weight != nullptr;
          const float inv = normed ? rsqrtf(ss * (1.f / D) + a.eps) : 1.f;
          const float* w = sw[is_q ? 0 : 1];
          float wv[8];
          *reinterpret_cast<float4*>(wv) = *reinterpret_cast<const float4*>(w + x0);
          *reinterpret_cast<float4*>(wv + 4) = *reinterpret_cast<const float4*>(w + x0 + 4);
          float y[8];
#pragma unroll
          for (int e = 0; e < 8; e++) y[e] = x[e] * inv * wv[e];
          float r[8];
          if (INTER) {
#pragma unroll
            for (int e = 0; e < 4; e++) {
              r[2 * e] = y[2 * e] * co[e % NF] - y[2 * e + 1] * si[e % NF];
              r[2 * e + 1] = y[2 * e + 1] * co[e % NF] + y[2 * e] * si[e % NF];
            }
          } else {
            uint4 other;  // the pairs' other members, as they were loaded
            other.x = __shfl_sync(0xffffffffu, raw[u].x, partner);
            other.y = __shfl_sync(0xffffffffu, raw[u].y, partner);
            other.z = __shfl_sync(0xffffffffu, raw[u].z, partner);
            other.w = __shfl_sync(0xffffffffu, raw[u].w, partner);
            float xo[8], wo[8];
            unpack8(other, xo);
            *reinterpret_cast<float4*>(wo) = *reinterpret_cast<const float4*>(w + px0);
            *reinterpret_cast<float4*>(wo + 4) = *reinterpret_cast<const float4*>(w + px0 + 4);
#pragma unroll
            for (int e = 0; e < 8; e++) {
              const float yo = xo[e] * inv * wo[e];
              const float sn = low ? -si[e % NF] : si[e % NF];
              r[e] = y[e] * co[e % NF] + yo * sn;
            }
          }
          if (!is_v)
            z = rotated ? make_uint4(pack_bf16(r[0], r[1]), pack_bf16(r[2], r[3]), pack_bf16(r[4], r[5]),
                                     pack_bf16(r[6], r[7]))
                        : make_uint4(pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3]), pack_bf16(y[4], y[5]),
                                     pack_bf16(y[6], y[7]));
        }
        if (live && is_q)
          *reinterpret_cast<uint4*>(a.q_out + (tok * a.Hq + h) * D + x0) = z;
        const bool write = live && !is_q && keep;
        const int64_t vec = row * a.Hkv + h;
        if (INT8) {
          if (HPW > 1 || !is_q)
            store_int8<LPH>(z, static_cast<int8_t*>(is_v ? a.v_pool : a.k_pool) + vec * D + x0,
                            (is_v ? a.v_scale : a.k_scale) + vec, write, sub == 0);
        } else if (write) {
          *reinterpret_cast<uint4*>(static_cast<uint16_t*>(is_v ? a.v_pool : a.k_pool) + vec * D + x0) = z;
        }
      }
    }
  }
}

template <int D>
void launch(const NormArgs& a, bool inter, bool int8, int grid, cudaStream_t st) {
  if (inter && int8)
    norm_rope_kernel<D, true, true><<<grid, kThreads, 0, st>>>(a);
  else if (inter)
    norm_rope_kernel<D, true, false><<<grid, kThreads, 0, st>>>(a);
  else if (int8)
    norm_rope_kernel<D, false, true><<<grid, kThreads, 0, st>>>(a);
  else
    norm_rope_kernel<D, false, false><<<grid, kThreads, 0, st>>>(a);
}

}  // namespace
}  // namespace skv

using namespace skv;

SKV_EXPORT int skv_norm_rope_append(int64_t n_tok, int Hq, int Hkv, int d, int rot, int interleaved,
                                    const uint16_t* q, int64_t q_stride, const uint16_t* k, int64_t k_stride,
                                    const uint16_t* v, int64_t v_stride, const float* q_weight,
                                    const float* k_weight, float eps, const int32_t* positions,
                                    const float* inv_freq, uint16_t* q_out, int kv_kind, const int64_t* out_rows,
                                    int64_t n_pool_rows, void* k_pool, void* v_pool, uint16_t* k_scale,
                                    uint16_t* v_scale, int32_t* dev_status, void* stream) {
  if (n_tok < 0 || Hq < 0 || Hkv < 0 || Hq > 4096 || Hkv > 4096 || n_pool_rows < 0) return SKV_EINVAL;
  if (d != 64 && d != 128 && d != 256) return SKV_EUNSUPPORTED;
  if (rot < 0 || rot > d || rot % 16 || (interleaved != 0 && interleaved != 1)) return SKV_EINVAL;
  if (kv_kind != SKV_KV_BF16 && kv_kind != SKV_KV_INT8) return SKV_EINVAL;
  if (!(eps >= 0.f)) return SKV_EINVAL;
  if (n_tok == 0) return SKV_OK;
  if (!q && !k && !v) return SKV_EINVAL;
  if ((rot > 0 && (q || k) && !inv_freq) || !positions) return SKV_EINVAL;
  const bool int8 = kv_kind == SKV_KV_INT8;
  if (q && (Hq < 1 || !q_out || !aligned16(q) || !aligned16(q_out) || q_stride % 8 ||
            q_stride < static_cast<int64_t>(Hq) * d))
    return SKV_EINVAL;
  if (k && (Hkv < 1 || !k_pool || !aligned16(k) || !aligned16(k_pool) || k_stride % 8 ||
            k_stride < static_cast<int64_t>(Hkv) * d || (int8 && !k_scale)))
    return SKV_EINVAL;
  if (v && (Hkv < 1 || !v_pool || !aligned16(v) || !aligned16(v_pool) || v_stride % 8 ||
            v_stride < static_cast<int64_t>(Hkv) * d || (int8 && !v_scale)))
    return SKV_EINVAL;
  if (!out_rows && (k || v) && n_pool_rows < n_tok) return SKV_EINVAL;
  const int sms = sm_count();
  if (sms <= 0) return SKV_ECUDA;
  NormArgs a{};
  a.n_tok = n_tok;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.rot = rot;
  a.slots_q = q ? Hq : 0;
  a.slots_k = k ? Hkv : 0;
  a.slots = a.slots_q + a.slots_k + (v ? Hkv : 0);
  a.q = q;
  a.k = k;
  a.v = v;
  a.q_stride = q_stride;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.q_weight = q_weight;
  a.k_weight = k_weight;
  a.eps = eps;
  a.positions = positions;
  a.inv_freq = inv_freq;
  a.q_out = q_out;
  a.out_rows = out_rows;
  a.n_pool_rows = n_pool_rows;
  a.k_pool = k_pool;
  a.v_pool = v_pool;
  a.k_scale = reinterpret_cast<__half*>(k_scale);
  a.v_scale = reinterpret_cast<__half*>(v_scale);
  a.status = dev_status;
  // Work items: enough of them for every resident warp, so a token's heads
  // are split over up to slots / HPW warps when there are few tokens.
  const int hpw = 32 / (d / 8);
  const int64_t warps = static_cast<int64_t>(sms) * 4 * kWarps;
  const int steps = (a.slots + hpw - 1) / hpw;
  int64_t chunks = (warps + n_tok - 1) / n_tok;
  if (chunks > steps) chunks = steps;
  const int per = static_cast<int>((steps + chunks - 1) / chunks);
  a.chunk = per * hpw;
  a.chunks = (steps + per - 1) / per;
  const int64_t want = (n_tok * a.chunks + kWarps - 1) / kWarps;
  const int grid = static_cast<int>(want < 4L * sms ? want : 4L * sms);
  cudaStream_t st = as_stream(stream);
  if (d == 64)
    launch<64>(a, interleaved, int8, grid, st);
  else if (d == 128)
    launch<128>(a, interleaved, int8, grid, st);
  else
    launch<256>(a, interleaved, int8, grid, st);
  return launch_status();
}
