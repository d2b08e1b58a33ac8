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
// of a turn: 45 bits.  inv_freq / 2 pi is kept as a 64-bit fixed-point
// fraction of a turn, made with integers (the fp32 mantissa times 2^66 / 2 pi,
// shifted; this GPU's fp64 rate would cost more than the whole pass).  p times
// it modulo 2^64 is the angle modulo one turn, exactly as unsigned integers
// wrap; its top 31 bits past the sign go to sincospif as far as fp32 holds
// them, and the rest turns the result: |p| 2^-64 of a turn from the fraction.
//
// Weights and rotation are folded: with wc = w cos and ws = -+ w' sin (w' the
// partner's weight) a value is inv (x wc + x' ws), x' the partner's input.
//
// A lane holds both members of its pairs: four dims x of a head and their
// partners x + rot/2 (eight consecutive dims where pairs are neighbours or
// nothing is rotated), so the rotation needs no exchange and the products run
// two to an instruction (f32x2).
//
// Bound: memory, then instruction issue (about 60 per head and warp): every
// value is read once and written once; d / 8 lanes share a head, so a head's
// sum is a shuffle reduction and no value passes through shared memory.  A
// warp takes a token's heads one after the other, a few in flight, and
// computes the token's sines once; with few tokens a token's heads are spread
// over several warps instead (launch rule below).  Measured (copy rate 6.79
// TB/s): 2048 tokens of 16 + 2 + 2 heads, 256 dims, 9.9 us (4.2 TB/s); 5237 of
// 32 + 8 + 8, 128 dims, pairs neighbours, 22.0 us (5.8 TB/s); 32768 of 24 + 4 + 4
// int8, 256 dims, 205 us (4.9 TB/s, 59 % of the issue slots); 8 tokens 3.6 us.
#include "common.cuh"

namespace skv {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
// 64 registers a thread.  32768 int8 tokens of 256 dims / 5237 bf16 tokens of
// 128 took 219 / 23.0 us with three CTAs, 208 / 22.0 with four, 284 / 26.2
// (spills) with five.
constexpr int kCtasPerSm = 4;
// Heads per lane group whose loads are in flight together.  The same two: two
// heads 205 / 25.1 us, four 208 / 22.0, six 225 / 23.7; 2048 bf16 tokens of 256
// dims: two 9.9, four 10.4.
template <int D>
constexpr int kBatch = D == 256 ? 2 : 4;

struct NormArgs {
  int64_t n_tok;
  int Hq, Hkv, rot;
  int steps_q, steps_k, steps_v;  // warp steps (32 lanes: 256 / d heads) per token; 0: part left out
  int chunk, chunks;              // steps per work item, work items per token
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

__device__ __forceinline__ F2 unpack2(uint32_t w) {
  return f2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}

__device__ __forceinline__ uint32_t pack2(F2 a) {
  const float2 x = f2_out(a);
  const __nv_bfloat162 h = __floats2bfloat162_rn(x.x, x.y);
  return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ uint2 ld_stream8(const void* p) {
  uint2 v;
  asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
  return v;
}

// A lane's eight values of a head: words 0, 1 at dims xa .., words 2, 3 at dims xb ..
struct Vals {
  uint32_t w[4];
};

// 1 / (2 pi) in units of 2^-66.
constexpr uint64_t kInvTwoPi = 0xA2F9836E4E44152Aull;

// f / 2 pi modulo one turn, in units of 2^-64 turns (f finite).
__device__ __forceinline__ uint64_t turn_of(float f) {
  const uint32_t u = __float_as_uint(f);
  const int e = max(1, static_cast<int>((u >> 23) & 255u));
  const uint64_t m = (u & 0x7fffffu) | (((u >> 23) & 255u) ? 0x800000u : 0u);  // f = m 2^(e - 150)
  const uint64_t lo = m * kInvTwoPi, hi = __umul64hi(m, kInvTwoPi);
  const int s = 152 - e;  // m kInvTwoPi 2^(e - 150 - 66 + 64)
  uint64_t t;
  if (s <= 0)
    t = s > -64 ? lo << -s : 0;
  else if (s < 64)
    t = (lo >> s) | (hi << (64 - s));
  else
    t = s < 128 ? hi >> (s - 64) : 0;
  return u >> 31 ? 0 - t : t;
}

// A lane's part of an int8 row: scale = fp16(max|x| / 127) over the head's
// lanes, codes = rint(x / scale), as skv_quantize_int8_rows.  The quotients
// come from a reciprocal (off by at most 127 * 3 * 2^-24 < 3e-5) unless one
// lies that near a half-integer, about one head in 40; then from the
// correctly rounded division.
template <int LPH>
__device__ __forceinline__ void store_int8(const Vals& z, int8_t* row, int xa, int xb, __half* scale, bool write,
                                           bool first) {
  float x[8];
  float m = 0.f;
#pragma unroll
  for (int e = 0; e < 4; e++) {
    x[2 * e] = __uint_as_float(z.w[e] << 16);
    x[2 * e + 1] = __uint_as_float(z.w[e] & 0xffff0000u);
    m = fmaxf(m, fmaxf(fabsf(x[2 * e]), fabsf(x[2 * e + 1])));
  }
#pragma unroll
  for (int o = LPH / 2; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  const __half sh = __float2half_rn(__fdiv_rn(m, 127.f));
  const float s = __half2float(sh);
  uint32_t w[2] = {0u, 0u};
  if (s != 0.f && s < 3.0e38f) {  // a zero or infinite scale: zero codes
    const float inv = __frcp_rn(s);
    float y[8];
    bool near = false;
#pragma unroll
    for (int e = 0; e < 8; e++) {
      y[e] = x[e] * inv;
      near |= !(fabsf(y[e] - rintf(y[e])) < 0.49995f);  // also where x is not finite
    }
    if (near) {
#pragma unroll
      for (int e = 0; e < 8; e++) y[e] = __fdiv_rn(x[e], s);
    }
#pragma unroll
    for (int e = 0; e < 8; e++) w[e >> 2] |= static_cast<uint32_t>(rint_clamp(y[e], -127, 127) & 255) << (8 * (e & 3));
  }
  if (write) {
    *reinterpret_cast<uint32_t*>(row + xa) = w[0];
    *reinterpret_cast<uint32_t*>(row + xb) = w[1];
    if (first) *scale = sh;
  }
}

enum { kQ = 0, kK = 1, kV = 2 };

// Steps [lo, hi) of one token's heads of one kind.
template <int D, bool INTER, bool INT8, int KIND>
__device__ __forceinline__ void run_heads(const NormArgs& a, int64_t tok, int64_t row, bool keep, int lo, int hi,
                                          int lane, bool rotated, int xa, int xb, const F2 (&wc)[4], const F2 (&ws)[4]) {
  constexpr int LPH = D / 8, HPW = 32 / LPH;
  const int grp = lane / LPH;
  const int H = KIND == kQ ? a.Hq : a.Hkv;
  const uint16_t* src = KIND == kQ ? a.q + tok * a.q_stride
                                   : KIND == kK ? a.k + tok * a.k_stride : a.v + tok * a.v_stride;
  const bool normed = KIND == kQ ? a.q_weight != nullptr : a.k_weight != nullptr;
  for (int s0 = lo; s0 < hi; s0 += kBatch<D>) {
    Vals raw[kBatch<D>];
#pragma unroll
    for (int u = 0; u < kBatch<D>; u++) {  // every load of the batch first
      const int h = (s0 + u) * HPW + grp;
      raw[u] = Vals{{0u, 0u, 0u, 0u}};
      if (s0 + u < hi && (HPW == 1 || h < H)) {
        const uint2 x = ld_stream8(src + h * D + xa), y = ld_stream8(src + h * D + xb);
        raw[u] = Vals{{x.x, x.y, y.x, y.y}};
      }
    }
#pragma unroll
    for (int u = 0; u < kBatch<D>; u++) {
      if (s0 + u >= hi) break;
      const int h = (s0 + u) * HPW + grp;
      const bool live = HPW == 1 || h < H;
      Vals z = raw[u];
      if (KIND != kV) {
        F2 x[4];
#pragma unroll
        for (int e = 0; e < 4; e++) x[e] = unpack2(raw[u].w[e]);
        float inv = 1.f;
        if (normed) {
          F2 q2 = f2_mul(x[0], x[0]);
#pragma unroll
          for (int e = 1; e < 4; e++) q2 = f2_fma(x[e], x[e], q2);
          const float2 q = f2_out(q2);
          float ss = q.x + q.y;
#pragma unroll
          for (int o = LPH / 2; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
          inv = rsqrtf(fmaf(ss, 1.f / D, a.eps));
        }
        const F2 inv2 = f2(inv, inv);
#pragma unroll
        for (int e = 0; e < 4; e++) {
          F2 o;  // the partners: the other half's, or the pair swapped
          if (INTER) {
            const float2 y = f2_out(x[e]);
            o = f2(y.y, y.x);
          } else {
            o = x[e ^ 2];
          }
          F2 r = f2_mul(x[e], wc[e]);
          if (rotated) r = f2_fma(o, ws[e], r);  // else an infinite neighbour would make 0 * inf
          z.w[e] = pack2(f2_mul(r, inv2));
        }
      }
      if (KIND == kQ) {
        if (live) {
          uint16_t* dst = a.q_out + (tok * a.Hq + h) * D;
          *reinterpret_cast<uint2*>(dst + xa) = make_uint2(z.w[0], z.w[1]);
          *reinterpret_cast<uint2*>(dst + xb) = make_uint2(z.w[2], z.w[3]);
        }
      } else {
        void* pool = KIND == kK ? a.k_pool : a.v_pool;
        const int64_t vec = row * a.Hkv + h;
        if (INT8) {
          store_int8<LPH>(z, static_cast<int8_t*>(pool) + vec * D, xa, xb, (KIND == kK ? a.k_scale : a.v_scale) + vec,
                          live && keep, lane % LPH == 0);
        } else if (live && keep) {
          uint16_t* dst = static_cast<uint16_t*>(pool) + vec * D;
          *reinterpret_cast<uint2*>(dst + xa) = make_uint2(z.w[0], z.w[1]);
          *reinterpret_cast<uint2*>(dst + xb) = make_uint2(z.w[2], z.w[3]);
        }
      }
    }
  }
}

template <int D, bool INTER, bool INT8>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) norm_rope_kernel(const NormArgs a) {
  constexpr int LPH = D / 8;  // lanes per head
  __shared__ __align__(16) float sw[2][D];
  __shared__ uint64_t turn[D / 2];
  __shared__ __align__(16) float2 cs[kWarps][D / 2];  // each warp's token: (cos, sin) by frequency
  for (int x = threadIdx.x; x < D; x += kThreads) {
    sw[0][x] = a.q_weight ? a.q_weight[x] : 1.f;
    sw[1][x] = a.k_weight ? a.k_weight[x] : 1.f;
    if (x < a.rot / 2) turn[x] = turn_of(a.inv_freq[x]);
  }
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int sub = lane % LPH;
  const int half = a.rot / 2;
  const bool rotated = sub < a.rot / 8;
  // this lane's dims xa .. xa + 3 and xb .. xb + 3, and the frequency of dim xa
  const int xa = !INTER && rotated ? 4 * sub : 8 * sub, xb = !INTER && rotated ? xa + half : xa + 4;
  __syncthreads();

  const int64_t items = a.n_tok * a.chunks;
  const int64_t step = static_cast<int64_t>(gridDim.x) * kWarps;
  const int off_k = a.steps_q, off_v = off_k + a.steps_k, end = off_v + a.steps_v;
  for (int64_t item = static_cast<int64_t>(blockIdx.x) * kWarps + warp; item < items; item += step) {
    const int64_t tok = a.chunks == 1 ? item : item / a.chunks;
    const int p0 = static_cast<int>(item - tok * a.chunks) * a.chunk, p1 = min(end, p0 + a.chunk);
    int64_t row = tok;
    if (a.out_rows) row = a.out_rows[tok];
    const int32_t pos = a.positions[tok];
    const bool bad = row >= a.n_pool_rows;
    if (bad && p1 > off_k && lane == 0) set_status(a.status, SKV_DEV_RANGE);
    const bool keep = row >= 0 && !bad;
    if (p0 < off_v) {
      __syncwarp();  // the previous token's values have been read
      for (int f = lane; f < half; f += 32) {
        const uint64_t t = turn[f];
        const uint32_t lo = static_cast<uint32_t>(t), hi = static_cast<uint32_t>(t >> 32);
        // top half of the low 64 bits of pos * t (pos sign-extended)
        uint32_t top = static_cast<uint32_t>(pos) * hi + __umulhi(static_cast<uint32_t>(pos), lo);
        if (pos < 0) top -= lo;
        // half turns: 31 bits, of which a float holds 24; the rest turns the result by a small angle
        // (without it one more rounding to bf16 in 50000 falls to the other side)
        const int32_t ht = static_cast<int32_t>(top);
        const float x = static_cast<float>(ht);
        const float rest = static_cast<float>(ht - static_cast<int32_t>(x)) * 1.4629180792671596e-9f;  // pi 2^-31
        float sn, cn;
        sincospif(x * 4.656612873077393e-10f, &sn, &cn);  // 2^-31
        cs[warp][f] = make_float2(fmaf(-sn, rest, cn), fmaf(cn, rest, sn));
      }
      __syncwarp();
    }
    F2 wc[4], ws[4];
    auto fold = [&](const float* w) {
#pragma unroll
      for (int e = 0; e < 4; e++) {
        const int x = (e < 2 ? xa : xb) + 2 * (e & 1);         // dims x, x + 1
        const int f = INTER ? x / 2 : xa + 2 * (e & 1);        // frequency of dim x (and, interleaved, of x + 1)
        float2 c0 = make_float2(1.f, 0.f), c1 = c0;
        if (rotated) {
          c0 = cs[warp][f];
          c1 = INTER ? c0 : cs[warp][f + 1];
        }
        wc[e] = f2(w[x] * c0.x, w[x + 1] * c1.x);
        if (INTER) {
          ws[e] = f2(-w[x + 1] * c0.y, w[x] * c0.y);
        } else {
          const int y = (e < 2 ? xb : xa) + 2 * (e & 1);       // the partners' dims
          ws[e] = e < 2 ? f2(-w[y] * c0.y, -w[y + 1] * c1.y) : f2(w[y] * c0.y, w[y + 1] * c1.y);
        }
      }
    };
    if (p0 < off_k) {
      fold(sw[0]);
      run_heads<D, INTER, INT8, kQ>(a, tok, row, keep, p0, min(p1, off_k), lane, rotated, xa, xb, wc, ws);
    }
    if (p0 < off_v && p1 > off_k) {
      fold(sw[1]);
      run_heads<D, INTER, INT8, kK>(a, tok, row, keep, max(p0, off_k) - off_k, min(p1, off_v) - off_k, lane, rotated, xa,
                                    xb, wc, ws);
    }
    if (p1 > off_v)
      run_heads<D, INTER, INT8, kV>(a, tok, row, keep, max(p0, off_v) - off_v, p1 - off_v, lane, rotated, xa, xb, wc, ws);
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
  a.rot = q || k ? rot : 0;  // values are not rotated: inv_freq may be NULL, and is not read
  const int hpw = 256 / d;
  a.steps_q = q ? (Hq + hpw - 1) / hpw : 0;
  a.steps_k = k ? (Hkv + hpw - 1) / hpw : 0;
  a.steps_v = v ? (Hkv + hpw - 1) / hpw : 0;
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
  // Work items: a token's heads in `chunks` parts, so that the rounds of the
  // resident warps times the steps of a part (each part paying about three
  // steps for its position and sines) come out lowest.
  const int64_t warps = static_cast<int64_t>(sms) * kCtasPerSm * kWarps;
  const int steps = a.steps_q + a.steps_k + a.steps_v;
  int64_t best = INT64_MAX;
  for (int c = 1; c <= steps; c++) {
    const int per = (steps + c - 1) / c, parts = (steps + per - 1) / per;
    const int64_t cost = (n_tok * parts + warps - 1) / warps * (per + 3);
    if (cost < best) {
      best = cost;
      a.chunk = per;
      a.chunks = parts;
    }
    if (n_tok >= 16 * warps) break;  // whole tokens
  }
  const int64_t want = (n_tok * a.chunks + kWarps - 1) / kWarps;
  const int64_t cap = static_cast<int64_t>(sms) * kCtasPerSm;
  const int grid = static_cast<int>(want < cap ? want : cap);
  cudaStream_t st = as_stream(stream);
  if (d == 64)
    launch<64>(a, interleaved, int8, grid, st);
  else if (d == 128)
    launch<128>(a, interleaved, int8, grid, st);
  else
    launch<256>(a, interleaved, int8, grid, st);
  return launch_status();
}
