// move_rows.cu -- cached rows from one place, position and encoding to another:
// parts of a prefix that were cached elsewhere, a tier's rows brought back, cold
// rows made smaller.
//
// Per listed token, K and V of every KV head:
//   x = the values that the source row stands for (exact in fp32: a code of up
//       to 8 bits times an fp16 scale)
//   keys that are turned: the pair (a, b) of frequency f becomes
//       (a cos t - b sin t, b cos t + a sin t),
//       t = new_position new_inv_freq[f] - old_position old_inv_freq[f]
//   destination row = x in its encoding, from the fp32 values.
// Without a turn and with the same encoding on both sides the bytes are copied.
//
// The angle is the difference of two 64-bit fixed-point fractions of a turn, as
// in norm_rope.cu: unsigned integers wrap, so neither position's size costs any
// of it.
//
// A lane holds eight values of a head as two runs of four: where halves are
// rotated against each other four dims x and their partners x + rot/2, so that a
// turn needs no exchange; elsewhere eight dims in a row.  d / 8 lanes share a
// head and a warp takes 256 values at a time.
#include "rope.cuh"

namespace skv {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kCtasPerSm = 4;
constexpr int kBatch = 4;  // heads per lane group whose loads are in flight together

struct RowSet {
  const unsigned char *k, *v;  // (written through on the destination's side)
  const __half *k_scale, *v_scale;
  int64_t n_rows, token_pitch, head_pitch;  // pitches in bytes
};

struct MoveArgs {
  int64_t n;
  int Hkv, rot;
  int turn;                  // keys are turned
  int steps_k, steps_v;      // warp steps (256 / d heads) per token; 0: part left out
  int chunk, chunks;         // steps per work item, work items per token
  RowSet src, dst;
  const int64_t *src_rows, *dst_rows;
  const int32_t *old_pos, *new_pos;
  const float *old_freq, *new_freq;
  int32_t* status;
};

enum Mode { kCopy, kConvert, kTurn };

// A lane's eight values as they lie in a row: bf16 words 0, 1 at dims xa .. and
// 2, 3 at dims xb ..; int8 words 0 and 2; int4 the low halves of words 0 and 2.
struct Raw {
  uint32_t w[4];
  uint16_t s[2];  // scales of the two runs
};

template <int KIND, bool RUN>  // RUN: xb == xa + 4
__device__ __forceinline__ Raw load(const unsigned char* vec, const __half* scale, int xa, int xb, int D) {
  Raw r{};
  if (KIND == SKV_KV_BF16) {
    if (RUN) {
      const uint4 x = ld_stream16(vec + 2 * xa);
      r.w[0] = x.x, r.w[1] = x.y, r.w[2] = x.z, r.w[3] = x.w;
    } else {
      const uint2 x = ld_stream8(vec + 2 * xa), y = ld_stream8(vec + 2 * xb);
      r.w[0] = x.x, r.w[1] = x.y, r.w[2] = y.x, r.w[3] = y.y;
    }
  } else if (KIND == SKV_KV_INT8) {
    if (RUN) {
      const uint2 x = ld_stream8(vec + xa);
      r.w[0] = x.x, r.w[2] = x.y;
    } else {
      r.w[0] = *reinterpret_cast<const uint32_t*>(vec + xa);
      r.w[2] = *reinterpret_cast<const uint32_t*>(vec + xb);
    }
    r.s[0] = r.s[1] = *reinterpret_cast<const uint16_t*>(scale);
  } else {
    if (RUN) {
      const uint32_t x = *reinterpret_cast<const uint32_t*>(vec + xa / 2);
      r.w[0] = x & 0xffffu, r.w[2] = x >> 16;
    } else {
      r.w[0] = *reinterpret_cast<const uint16_t*>(vec + xa / 2);
      r.w[2] = *reinterpret_cast<const uint16_t*>(vec + xb / 2);
    }
    r.s[0] = *reinterpret_cast<const uint16_t*>(vec + D / 2 + (xa >> 6) * 2);
    r.s[1] = RUN ? r.s[0] : *reinterpret_cast<const uint16_t*>(vec + D / 2 + (xb >> 6) * 2);
  }
  return r;
}

template <int KIND>
__device__ __forceinline__ void decode(const Raw& r, float (&x)[8]) {
  if (KIND == SKV_KV_BF16) {
#pragma unroll
    for (int e = 0; e < 4; e++) {
      x[2 * e] = __uint_as_float(r.w[e] << 16);
      x[2 * e + 1] = __uint_as_float(r.w[e] & 0xffff0000u);
    }
  } else {
#pragma unroll
    for (int run = 0; run < 2; run++) {
      float s = __half2float(__ushort_as_half(r.s[run]));
      if (!(fabsf(s) <= 65504.f)) s = 0.f;  // the encodings give such a row zero codes
      const int w = static_cast<int>(r.w[2 * run]);
#pragma unroll
      for (int e = 0; e < 4; e++) {
        const int c = KIND == SKV_KV_INT8 ? (w << (24 - 8 * e)) >> 24 : (w << (28 - 4 * e)) >> 28;
        x[4 * run + e] = static_cast<float>(c) * s;
      }
    }
  }
}

// rint(x / s) of four values, clamped.  The quotients come from a reciprocal
// (off by at most 127 * 3 * 2^-24 < 3e-5) unless one lies that near a
// half-integer; then from the correctly rounded division.
__device__ __forceinline__ void codes_of(const float* x, float s, int lo, int hi, int (&c)[4]) {
  const float inv = __frcp_rn(s);
  float y[4];
  bool near = false;
#pragma unroll
  for (int e = 0; e < 4; e++) {
    y[e] = x[e] * inv;
    near |= !(fabsf(y[e] - rintf(y[e])) < 0.49995f);  // also where x is not finite
  }
  if (near) {
#pragma unroll
    for (int e = 0; e < 4; e++) y[e] = __fdiv_rn(x[e], s);
  }
#pragma unroll
  for (int e = 0; e < 4; e++) c[e] = rint_clamp(y[e], lo, hi);
}

// A zero or infinite scale gives zero codes.
__device__ __forceinline__ bool usable(float s) { return s != 0.f && s < 3.0e38f; }

__device__ __forceinline__ float max4(const float* x) {  // of the absolute values; a NaN takes no part
  return fmaxf(fmaxf(fmaxf(0.f, fabsf(x[0])), fabsf(x[1])), fmaxf(fabsf(x[2]), fabsf(x[3])));
}

// Every lane of the warp takes part; `write`: this lane's head is written.
template <int KIND, bool RUN, int LPH>
__device__ __forceinline__ void encode(const float (&x)[8], unsigned char* vec, __half* scale, int xa, int xb, bool write) {
  constexpr int D = 8 * LPH;
  if (KIND == SKV_KV_BF16) {
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; e++) w[e] = pack2(f2(x[2 * e], x[2 * e + 1]));
    if (!write) return;
    if (RUN) {
      *reinterpret_cast<uint4*>(vec + 2 * xa) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
      *reinterpret_cast<uint2*>(vec + 2 * xa) = make_uint2(w[0], w[1]);
      *reinterpret_cast<uint2*>(vec + 2 * xb) = make_uint2(w[2], w[3]);
    }
  } else if (KIND == SKV_KV_INT8) {
    float m = fmaxf(max4(x), max4(x + 4));
#pragma unroll
    for (int o = LPH / 2; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    const __half sh = __float2half_rn(__fdiv_rn(m, 127.f));
    const float s = __half2float(sh);
    uint32_t w[2] = {0u, 0u};
    if (usable(s)) {
#pragma unroll
      for (int run = 0; run < 2; run++) {
        int c[4];
        codes_of(x + 4 * run, s, -127, 127, c);
#pragma unroll
        for (int e = 0; e < 4; e++) w[run] |= static_cast<uint32_t>(c[e] & 255) << (8 * e);
      }
    }
    if (!write) return;
    if (RUN) {
      *reinterpret_cast<uint2*>(vec + xa) = make_uint2(w[0], w[1]);
    } else {
      *reinterpret_cast<uint32_t*>(vec + xa) = w[0];
      *reinterpret_cast<uint32_t*>(vec + xb) = w[1];
    }
    if (xa == 0) *scale = sh;
  } else {
    static_assert(KIND != SKV_KV_INT4 || LPH == 32, "a warp per vector");
    const float ma = max4(x), mb = max4(x + 4);
    const int ga = xa >> 6, gb = xb >> 6;
    float m[2] = {0.f, 0.f};
#pragma unroll
    for (int g = 0; g < D / 64; g++) {  // as bits: neither NaN nor negative
      const float mine = fmaxf(ga == g ? ma : 0.f, gb == g ? mb : 0.f);
      const float all = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(mine)));
      if (ga == g) m[0] = all;
      if (gb == g) m[1] = all;
    }
    uint32_t w[2] = {0u, 0u};
    uint16_t sb[2];
#pragma unroll
    for (int run = 0; run < 2; run++) {
      const __half sh = __float2half_rn(__fdiv_rn(m[run], 7.f));
      const float s = __half2float(sh);
      sb[run] = __half_as_ushort(sh);
      if (usable(s)) {
        int c[4];
        codes_of(x + 4 * run, s, -8, 7, c);
#pragma unroll
        for (int e = 0; e < 4; e++) w[run] |= static_cast<uint32_t>(c[e] & 15) << (4 * e);
      }
    }
    if (!write) return;
    if (RUN) {
      *reinterpret_cast<uint32_t*>(vec + xa / 2) = w[0] | w[1] << 16;
    } else {
      *reinterpret_cast<uint16_t*>(vec + xa / 2) = static_cast<uint16_t>(w[0]);
      *reinterpret_cast<uint16_t*>(vec + xb / 2) = static_cast<uint16_t>(w[1]);
    }
    if ((xa & 63) == 0) *reinterpret_cast<uint16_t*>(vec + D / 2 + 2 * ga) = sb[0];
    if ((xb & 63) == 0) *reinterpret_cast<uint16_t*>(vec + D / 2 + 2 * gb) = sb[1];
  }
}

// The bytes as they are (RUN).
template <int KIND, int LPH>
__device__ __forceinline__ void store(const Raw& r, unsigned char* vec, __half* scale, int xa) {
  if (KIND == SKV_KV_BF16) {
    *reinterpret_cast<uint4*>(vec + 2 * xa) = make_uint4(r.w[0], r.w[1], r.w[2], r.w[3]);
  } else if (KIND == SKV_KV_INT8) {
    *reinterpret_cast<uint2*>(vec + xa) = make_uint2(r.w[0], r.w[2]);
    if (xa == 0) *reinterpret_cast<uint16_t*>(scale) = r.s[0];
  } else {
    *reinterpret_cast<uint32_t*>(vec + xa / 2) = r.w[0] | r.w[2] << 16;
    if ((xa & 63) == 0) *reinterpret_cast<uint16_t*>(vec + 4 * LPH + (xa >> 6) * 2) = r.s[0];
  }
}

// Steps [lo, hi) of one token's K or V.
template <int LPH, int SRC, int DST, bool INTER, Mode MODE>
__device__ __forceinline__ void run_heads(const MoveArgs& a, bool values, int64_t from, int64_t to, int lo, int hi,
                                          int lane, const float2* cs) {
  constexpr int D = 8 * LPH, HPW = 32 / LPH;
  constexpr bool RUN = MODE != kTurn || INTER;
  const int sub = lane % LPH, grp = lane / LPH, half = a.rot / 2;
  const bool rotated = MODE == kTurn && sub < a.rot / 8;
  const int xa = !RUN && rotated ? 4 * sub : 8 * sub, xb = !RUN && rotated ? xa + half : xa + 4;
  F2 co[4], si[4];
  if (MODE == kTurn) {
#pragma unroll
    for (int e = 0; e < 4; e++) {  // of values 2 e, 2 e + 1
      float2 c0 = make_float2(1.f, 0.f), c1 = c0;
      if (rotated) {
        c0 = cs[INTER ? xa / 2 + e : xa + 2 * (e & 1)];
        c1 = INTER ? c0 : cs[xa + 2 * (e & 1) + 1];
      }
      co[e] = f2(c0.x, c1.x);
      si[e] = INTER ? f2(-c0.y, c0.y) : e < 2 ? f2(-c0.y, -c1.y) : f2(c0.y, c1.y);
    }
  }
  const unsigned char* src = (values ? a.src.v : a.src.k) + from * a.src.token_pitch;
  unsigned char* dst = const_cast<unsigned char*>(values ? a.dst.v : a.dst.k) + to * a.dst.token_pitch;
  const __half* sscale = SRC == SKV_KV_INT8 ? (values ? a.src.v_scale : a.src.k_scale) + from * a.Hkv : nullptr;
  __half* dscale = DST == SKV_KV_INT8 ? const_cast<__half*>(values ? a.dst.v_scale : a.dst.k_scale) + to * a.Hkv : nullptr;
  for (int s0 = lo; s0 < hi; s0 += kBatch) {
    Raw raw[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; u++) {  // every load of the batch first
      const int h = (s0 + u) * HPW + grp;
      raw[u] = Raw{};
      if (s0 + u < hi && (HPW == 1 || h < a.Hkv)) raw[u] = load<SRC, RUN>(src + h * a.src.head_pitch, sscale + h, xa, xb, D);
    }
#pragma unroll
    for (int u = 0; u < kBatch; u++) {
      if (s0 + u >= hi) break;
      const int h = (s0 + u) * HPW + grp;
      const bool live = HPW == 1 || h < a.Hkv;
      unsigned char* vec = dst + h * a.dst.head_pitch;
      if constexpr (MODE == kCopy) {
        if (live) store<SRC, LPH>(raw[u], vec, dscale + h, xa);
      } else {
        float x[8];
        decode<SRC>(raw[u], x);
        if constexpr (MODE == kTurn) {
          if (rotated) {  // elsewhere an infinite neighbour would make 0 * inf
            F2 y[4];
#pragma unroll
            for (int e = 0; e < 4; e++) {
              const F2 own = f2(x[2 * e], x[2 * e + 1]);
              const F2 other = INTER ? f2(x[2 * e + 1], x[2 * e]) : f2(x[2 * (e ^ 2)], x[2 * (e ^ 2) + 1]);
              y[e] = f2_fma(other, si[e], f2_mul(own, co[e]));
            }
#pragma unroll
            for (int e = 0; e < 4; e++) {
              const float2 z = f2_out(y[e]);
              x[2 * e] = z.x;
              x[2 * e + 1] = z.y;
            }
          }
        }
        encode<DST, RUN, LPH>(x, vec, dscale + h, xa, xb, live);
      }
    }
  }
}

template <int D, int SRC, int DST, bool INTER>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) move_kernel(const MoveArgs a) {
  constexpr int LPH = D / 8;
  __shared__ uint64_t turns[2][D / 2];
  __shared__ __align__(16) float2 cs[kWarps][D / 2];  // each warp's token: (cos, sin) by frequency
  const int half = a.rot / 2;
  if (a.turn) {
    for (int f = threadIdx.x; f < half; f += kThreads) {
      turns[0][f] = a.old_pos ? turn_of(a.old_freq[f]) : 0;
      turns[1][f] = a.new_pos ? turn_of(a.new_freq[f]) : 0;
    }
  }
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  __syncthreads();
  const int64_t items = a.n * a.chunks;
  const int64_t step = static_cast<int64_t>(gridDim.x) * kWarps;
  const int end = a.steps_k + a.steps_v;
  for (int64_t item = static_cast<int64_t>(blockIdx.x) * kWarps + warp; item < items; item += step) {
    const int64_t tok = a.chunks == 1 ? item : item / a.chunks;
    const int p0 = static_cast<int>(item - tok * a.chunks) * a.chunk, p1 = min(end, p0 + a.chunk);
    const int64_t from = a.src_rows ? a.src_rows[tok] : tok, to = a.dst_rows ? a.dst_rows[tok] : tok;
    if (from < 0 || to < 0) continue;  // padding
    if (from >= a.src.n_rows || to >= a.dst.n_rows) {
      if (lane == 0) set_status(a.status, SKV_DEV_RANGE);
      continue;
    }
    if (p0 < a.steps_k) {
      if (a.turn) {
        const uint64_t old_pos = a.old_pos ? static_cast<int64_t>(a.old_pos[tok]) : 0;
        const uint64_t new_pos = a.new_pos ? static_cast<int64_t>(a.new_pos[tok]) : 0;
        __syncwarp();  // the previous token's values have been read
        for (int f = lane; f < half; f += 32)
          cs[warp][f] = cos_sin(static_cast<uint32_t>((new_pos * turns[1][f] - old_pos * turns[0][f]) >> 32));
        __syncwarp();
        run_heads<LPH, SRC, DST, INTER, kTurn>(a, false, from, to, p0, min(p1, a.steps_k), lane, cs[warp]);
      } else {
        run_heads<LPH, SRC, DST, INTER, SRC == DST ? kCopy : kConvert>(a, false, from, to, p0, min(p1, a.steps_k), lane,
                                                                       nullptr);
      }
    }
    if (p1 > a.steps_k)
      run_heads<LPH, SRC, DST, INTER, SRC == DST ? kCopy : kConvert>(a, true, from, to, max(p0, a.steps_k) - a.steps_k,
                                                                     p1 - a.steps_k, lane, nullptr);
  }
}

template <int D, int SRC, int DST>
void launch(const MoveArgs& a, bool inter, int grid, cudaStream_t st) {
  if (inter)
    move_kernel<D, SRC, DST, true><<<grid, kThreads, 0, st>>>(a);
  else
    move_kernel<D, SRC, DST, false><<<grid, kThreads, 0, st>>>(a);
}

template <int D>
void launch_kinds(const MoveArgs& a, int src, int dst, bool inter, int grid, cudaStream_t st) {
  constexpr int B = SKV_KV_BF16, I8 = SKV_KV_INT8, I4 = SKV_KV_INT4;
  if constexpr (D == 256) {
    if (src == I4) {
      if (dst == B) return launch<D, I4, B>(a, inter, grid, st);
      if (dst == I8) return launch<D, I4, I8>(a, inter, grid, st);
      return launch<D, I4, I4>(a, inter, grid, st);
    }
    if (dst == I4) return src == B ? launch<D, B, I4>(a, inter, grid, st) : launch<D, I8, I4>(a, inter, grid, st);
  }
  if (src == B) return dst == B ? launch<D, B, B>(a, inter, grid, st) : launch<D, B, I8>(a, inter, grid, st);
  return dst == B ? launch<D, I8, B>(a, inter, grid, st) : launch<D, I8, I8>(a, inter, grid, st);
}

// Checks one side and fills its addresses and pitches.
int side(const skv_row_set* s, int64_t n, int Hkv, int d, const int64_t* rows, RowSet* out) {
  if (s->n_rows < 0 || (!rows && s->n_rows < n)) return SKV_EINVAL;
  out->k = static_cast<const unsigned char*>(s->k);
  out->v = static_cast<const unsigned char*>(s->v);
  out->k_scale = reinterpret_cast<const __half*>(s->k_scale);
  out->v_scale = reinterpret_cast<const __half*>(s->v_scale);
  out->n_rows = s->n_rows;
  if (s->kind == SKV_KV_INT4) {
    out->token_pitch = s->token_pitch;
    out->head_pitch = s->head_pitch;
    if (s->head_pitch < d / 2 + d / 32 || s->token_pitch < Hkv * s->head_pitch) return SKV_EINVAL;
    if ((reinterpret_cast<uintptr_t>(s->k) | reinterpret_cast<uintptr_t>(s->v) | s->token_pitch | s->head_pitch) & 3)
      return SKV_EINVAL;
    return SKV_OK;
  }
  out->head_pitch = d * (s->kind == SKV_KV_INT8 ? 1 : 2);
  out->token_pitch = Hkv * out->head_pitch;
  if (!aligned16(s->k) || !aligned16(s->v)) return SKV_EINVAL;
  if (s->kind == SKV_KV_INT8 && ((s->k && !s->k_scale) || (s->v && !s->v_scale))) return SKV_EINVAL;
  return SKV_OK;
}

}  // namespace
}  // namespace skv

using namespace skv;

SKV_EXPORT int skv_move_rows(int64_t n, int Hkv, int d, const skv_row_set* src, const int64_t* src_rows,
                             const skv_row_set* dst, const int64_t* dst_rows, int rot, int interleaved,
                             const int32_t* old_positions, const float* old_inv_freq, const int32_t* new_positions,
                             const float* new_inv_freq, int32_t* dev_status, void* stream) {
  if (n < 0 || Hkv < 1 || Hkv > 4096 || !src || !dst) return SKV_EINVAL;
  for (const skv_row_set* s : {src, dst})
    if (s->kind != SKV_KV_BF16 && s->kind != SKV_KV_INT8 && s->kind != SKV_KV_INT4) return SKV_EINVAL;
  if (d != 256 && ((d != 64 && d != 128) || src->kind == SKV_KV_INT4 || dst->kind == SKV_KV_INT4)) return SKV_EUNSUPPORTED;
  if (rot < 0 || rot > d || rot % 16 || (interleaved != 0 && interleaved != 1)) return SKV_EINVAL;
  if (n == 0) return SKV_OK;
  if (!src->k != !dst->k || !src->v != !dst->v || (!src->k && !src->v)) return SKV_EINVAL;
  const bool turn = src->k && rot > 0 && (old_positions || new_positions);
  if (turn && ((old_positions && !old_inv_freq) || (new_positions && !new_inv_freq))) return SKV_EINVAL;
  MoveArgs a{};
  int e = side(src, n, Hkv, d, src_rows, &a.src);
  if (e == SKV_OK) e = side(dst, n, Hkv, d, dst_rows, &a.dst);
  if (e != SKV_OK) return e;
  const int sms = sm_count();
  if (sms <= 0) return SKV_ECUDA;
  a.n = n;
  a.Hkv = Hkv;
  a.rot = rot;
  a.turn = turn;
  const int hpw = 256 / d;
  a.steps_k = src->k ? (Hkv + hpw - 1) / hpw : 0;
  a.steps_v = src->v ? (Hkv + hpw - 1) / hpw : 0;
  a.src_rows = src_rows;
  a.dst_rows = dst_rows;
  a.old_pos = old_positions;
  a.new_pos = new_positions;
  a.old_freq = old_inv_freq;
  a.new_freq = new_inv_freq;
  a.status = dev_status;
  // Work items: a token's heads in `chunks` parts, so that the rounds of the
  // resident warps times the steps of a part (each paying about three steps for
  // its rows and sines) come out lowest.
  const int64_t warps = static_cast<int64_t>(sms) * kCtasPerSm * kWarps;
  const int steps = a.steps_k + a.steps_v;
  int64_t best = INT64_MAX;
  for (int c = 1; c <= steps; c++) {
    const int per = (steps + c - 1) / c, parts = (steps + per - 1) / per;
    const int64_t cost = (n * parts + warps - 1) / warps * (per + 3);
    if (cost < best) {
      best = cost;
      a.chunk = per;
      a.chunks = parts;
    }
    if (n >= 16 * warps) break;  // whole tokens
  }
  const int64_t want = (n * a.chunks + kWarps - 1) / kWarps;
  const int64_t cap = static_cast<int64_t>(sms) * kCtasPerSm;
  const int grid = static_cast<int>(want < cap ? want : cap);
  cudaStream_t st = as_stream(stream);
  if (d == 64)
    launch_kinds<64>(a, src->kind, dst->kind, interleaved, grid, st);
  else if (d == 128)
    launch_kinds<128>(a, src->kind, dst->kind, interleaved, grid, st);
  else
    launch_kinds<256>(a, src->kind, dst->kind, interleaved, grid, st);
  return launch_status();
}
