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
//
// Bound: memory where nothing is encoded, instruction issue where rows become int8
// or int4 (a head's largest value, its scale, the codes): 57 to 65 % of the issue
// slots, the rest steps that wait for one another.  Measured (copy rate 6.79 TB/s;
// K and V of 4 heads of 256, 32768 rows): bf16 44.6 us (6.0 TB/s), int8 copied 23.5
// (5.8), with keys turned 41.2 (3.3), bf16 to int8 37.3 (5.4), turned 45.4 (4.5), int4
// to int8 40.7 (2.6), turned 51.9 (2.0), int4 to bf16 33.4 (5.1), turned 40.9 (4.2), bf16
// to int4 48.4 (3.5), turned 67.6 (2.5); 64 rows 3.3 us.
#include "rope.cuh"

namespace skv {
namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kLoad = 4;  // heads per lane group whose loads are in flight together
// Of them decoded and encoded together, and resident CTAs (64 or 72 registers a
// thread).  Four heads share the work on their scales; rows of 64 dims, eight of
// them, would wait for one another.  65536 int4 rows to int8 / 32768 int8 rows
// turned / 32768 of 64 dims / 32768 int8 rows to bf16, turned: two heads and eight
// CTAs 108.2 / 40.9 / 31.0 / 39.6 us, four and seven 103.1 / 41.5 / 35.9 / 41.4, two
// and six 114.6 / 45.2 / 31.0 / 45.3, one and ten 118.3 / 44.9 / 33.2 / 40.6.
template <int D, int DST>
constexpr int kBatch = DST != SKV_KV_BF16 && D > 64 ? 4 : 2;
constexpr int ctas_per_sm(int d, int dst) { return dst != SKV_KV_BF16 && d > 64 ? 7 : 8; }

struct RowSet {
  const unsigned char *k, *v;  // (written through on the destination's side)
  const __half *k_scale, *v_scale;
  int64_t n_rows, token_pitch, head_pitch;  // pitches in bytes
};

struct MoveArgs {
  int64_t n;
  int Hkv, rot;
  int turn;                  // keys are turned
  int steps;                 // warp steps (256 / d heads) of a token's K or V
  int chunk;                 // steps per work item
  int chunks_k, chunks_v;    // work items per token; 0: part left out
  RowSet src, dst;
  const int64_t *src_rows, *dst_rows;
  const int32_t *old_pos, *new_pos;
  const float *old_freq, *new_freq;
  int32_t* status;
};

enum Mode { kCopy, kConvert, kTurn };

// A lane's eight values as they lie in a row: bf16 words 0, 1 at dims xa .. and
// 2, 3 at dims xb ..; int8 words 0 and 2; int4 (RUN) word 0, else the low halves of
// words 0 and 2.
struct Raw {
  uint32_t w[4];
  uint16_t s[2];  // scales of the two runs
};

// A cache may be its own destination, so rows are read as memory that the kernel
// writes, not by the read-only path (32768 int8 rows turned 41.3 us either way,
// 5237 bf16 rows 5.5; without the hint, rows copied 27.4 against 23.4).
__device__ __forceinline__ uint4 ld_row16(const unsigned char* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p)
               : "memory");
  return v;
}
__device__ __forceinline__ uint2 ld_row8(const unsigned char* p) {
  uint2 v;
  asm volatile("ld.global.L1::no_allocate.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p) : "memory");
  return v;
}

template <int KIND, bool RUN>  // RUN: xb == xa + 4
__device__ __forceinline__ Raw load(const unsigned char* vec, const __half* scale, int xa, int xb, int D) {
  Raw r{};
  if (KIND == SKV_KV_BF16) {
    if (RUN) {
      const uint4 x = ld_row16(vec + 2 * xa);
      r.w[0] = x.x, r.w[1] = x.y, r.w[2] = x.z, r.w[3] = x.w;
    } else {
      const uint2 x = ld_row8(vec + 2 * xa), y = ld_row8(vec + 2 * xb);
      r.w[0] = x.x, r.w[1] = x.y, r.w[2] = y.x, r.w[3] = y.y;
    }
  } else if (KIND == SKV_KV_INT8) {
    if (RUN) {
      const uint2 x = ld_row8(vec + xa);
      r.w[0] = x.x, r.w[2] = x.y;
    } else {
      r.w[0] = *reinterpret_cast<const uint32_t*>(vec + xa);
      r.w[2] = *reinterpret_cast<const uint32_t*>(vec + xb);
    }
    r.s[0] = r.s[1] = *reinterpret_cast<const uint16_t*>(scale);
  } else {
    if (RUN) {
      r.w[0] = *reinterpret_cast<const uint32_t*>(vec + xa / 2);
    } else {
      r.w[0] = *reinterpret_cast<const uint16_t*>(vec + xa / 2);
      r.w[2] = *reinterpret_cast<const uint16_t*>(vec + xb / 2);
    }
    r.s[0] = *reinterpret_cast<const uint16_t*>(vec + D / 2 + (xa >> 6) * 2);
    r.s[1] = RUN ? r.s[0] : *reinterpret_cast<const uint16_t*>(vec + D / 2 + (xb >> 6) * 2);
  }
  return r;
}

// The eight values, exact: run a in x[0], x[1], run b in x[2], x[3].  A code
// becomes a float as the low bits of 2^23: conversions run at an eighth of the
// rate of the rest.
template <int KIND, bool RUN>
__device__ __forceinline__ void decode(const Raw& r, F2 (&x)[4]) {
  if (KIND == SKV_KV_BF16) {
#pragma unroll
    for (int e = 0; e < 4; e++) x[e] = unpack2(r.w[e]);
  } else {
    const float zero = KIND == SKV_KV_INT8 ? -8388736.f : -8388616.f;  // 2^23 and the codes' offset
    float s[2], f[8];
#pragma unroll
    for (int run = 0; run < 2; run++) {
      s[run] = run && RUN ? s[0] : __half2float(__ushort_as_half(r.s[run]));
      if (!(fabsf(s[run]) <= 65504.f)) s[run] = 0.f;  // the encodings give such a row zero codes
      if (KIND == SKV_KV_INT8) {
        const uint32_t w = r.w[2 * run] ^ 0x80808080u;
#pragma unroll
        for (int e = 0; e < 4; e++) f[4 * run + e] = __uint_as_float(prmt(w, 0x4b000000u, 0x7650u + e));
      } else {
        const uint32_t w = (RUN ? r.w[0] : r.w[2 * run]) ^ 0x88888888u;
        const uint32_t even = w & 0x0f0f0f0fu, odd = (w >> 4) & 0x0f0f0f0fu;
#pragma unroll
        for (int e = 0; e < 4; e++)
          f[4 * run + e] = __uint_as_float(prmt(e & 1 ? odd : even, 0x4b000000u, 0x7650u + e / 2 + (RUN ? 2 * run : 0)));
      }
    }
#pragma unroll
    for (int e = 0; e < 4; e++)
      x[e] = f2_mul(f2_add(f2(f[2 * e], f[2 * e + 1]), f2(zero, zero)), f2(s[e / 2], s[e / 2]));
  }
}

// The largest absolute value of N pairs; a NaN takes no part.
template <int N>
__device__ __forceinline__ float amax(const F2* x) {
  float m = 0.f;
#pragma unroll
  for (int e = 0; e < N; e++) {
    const float2 v = f2_out(x[e]);
    m = fmaxf(fmaxf(m, fabsf(v.x)), fabsf(v.y));
  }
  return m;
}

// The largest of each LANES lanes (not negative, no NaN).
template <int LANES>
__device__ __forceinline__ float lanes_max(float m) {
  if (LANES == 32) return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(m)));
#pragma unroll
  for (int o = LANES / 2; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  return m;
}

// This lane's scale's largest value: lane `sub` of LANES holds the one of step sub.
template <int LANES, int N>
__device__ __forceinline__ float scale_max(const F2 (&v)[N][4], int sub) {
  float mine = 0.f;
#pragma unroll
  for (int u = 0; u < N; u++) {
    const float m = lanes_max<LANES>(amax<4>(v[u]));
    if (sub == u) mine = m;
  }
  return mine;
}

// fp16(m / TOP), the quotient rounded to fp32 and then to fp16: q0 = m c with c =
// 1 / TOP rounded, and q0 + (m - TOP q0) c, which rounds as the quotient does
// (Markstein's correction; tested for every mantissa of m).  A quotient too small
// for that is zero in fp16, and an infinite m is replaced by the largest number,
// whose quotient is beyond fp16, too.
template <int TOP>
__device__ __forceinline__ __half scale_of(float m) {
  constexpr float c = 1.f / TOP;
  m = fminf(m, 3.402823466e38f);
  const float q0 = m * c;
  return __float2half_rn(fmaf(fmaf(-q0, static_cast<float>(TOP), m), c, q0));
}

// A zero or infinite scale gives zero codes.
__device__ __forceinline__ bool usable(float s) { return s != 0.f && s < 3.0e38f; }

__device__ __forceinline__ float max_nan(float a, float b, float c) {  // NaN if one is
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// The codes rint(x / s) of a run's four values, clamped, as bytes.  x is multiplied
// with the reciprocal and rounded to r by adding 2^23 + 2^22; the remainder x - r s
// is exact (r s has 19 bits) and below s / 2 wherever r is the nearest integer.
// `off` is the largest remainder, NaN where there is none.  (The values of bf16,
// int8 and int4 rows are too coarse for the quotient's own rounding to meet a
// half-integer that it is not, so this is the rounded quotient's code, too.)
struct Codes {
  F2 r[2], e[2];
};
__device__ __forceinline__ float try_codes(const F2* x, float s, float inv, Codes& c) {
  const F2 up = f2(12582912.f, 12582912.f), down = f2(-12582912.f, -12582912.f), i2 = f2(inv, inv), ms = f2(-s, -s);
#pragma unroll
  for (int p = 0; p < 2; p++) {
    c.r[p] = f2_fma(x[p], i2, up);
    c.e[p] = f2_fma(f2_add(c.r[p], down), ms, x[p]);
  }
  const float2 e0 = f2_out(c.e[0]), e1 = f2_out(c.e[1]);
  return max_nan(max_nan(0.f, fabsf(e0.x), fabsf(e0.y)), fabsf(e1.x), fabsf(e1.y));
}
__device__ __forceinline__ uint32_t bytes_of(const Codes& c) {
  const float2 a = f2_out(c.r[0]), b = f2_out(c.r[1]);
  return prmt(prmt(__float_as_uint(a.x), __float_as_uint(a.y), 0x0040u),
              prmt(__float_as_uint(b.x), __float_as_uint(b.y), 0x0040u), 0x5410u);
}
// Where a remainder is s / 2 (ties go to the even code) or more, a value is no
// number, or the scale is so small that fp16 holds it too coarsely for the largest
// code to stay in range by itself.
template <int TOP>
__device__ __forceinline__ uint32_t other_codes(const Codes& c, const F2* x, float s) {
  constexpr int lo = TOP == 7 ? -8 : -TOP;
  uint32_t w = 0;
#pragma unroll
  for (int i = 0; i < 4; i++) {
    const float2 rr = f2_out(c.r[i / 2]), ee = f2_out(c.e[i / 2]), xx = f2_out(x[i / 2]);
    const float r = i & 1 ? rr.y : rr.x, e = i & 1 ? ee.y : ee.x, v = i & 1 ? xx.y : xx.x;
    int q = static_cast<int>(__float_as_uint(r)) - 0x4b400000;
    if (fabsf(e) > 0.5f * s || (fabsf(e) == 0.5f * s && (q & 1))) q += e > 0.f ? 1 : -1;
    q = v != v ? lo : min(max(q, lo), TOP);
    if (usable(s)) w |= static_cast<uint32_t>(q & 255) << (8 * i);
  }
  return w;
}

// The codes of a step's two runs, of scales that lanes la and lb hold.
template <int TOP, bool ONE>  // one scale for both
__device__ __forceinline__ void codes_of(const F2 (&v)[4], float s_own, float i_own, int la, int lb, uint32_t (&w)[2]) {
  constexpr uint32_t full = 0xffffffffu;
  const float sa = __shfl_sync(full, s_own, la), ia = __shfl_sync(full, i_own, la);
  const float sb = ONE ? sa : __shfl_sync(full, s_own, lb), ib = ONE ? ia : __shfl_sync(full, i_own, lb);
  Codes a, b;
  const float oa = try_codes(&v[0], sa, ia, a), ob = try_codes(&v[2], sb, ib, b);
  w[0] = bytes_of(a);
  w[1] = bytes_of(b);
  const float ha = sa < 6.103515625e-5f ? -1.f : 0.5f * sa, hb = ONE ? ha : sb < 6.103515625e-5f ? -1.f : 0.5f * sb;
  if (!(oa < ha) || !(ob < hb)) {
    w[0] = other_codes<TOP>(a, &v[0], sa);
    w[1] = other_codes<TOP>(b, &v[2], sb);
  }
}

__device__ __forceinline__ float reciprocal(float s) {  // to 2^-23
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(s));
  return r;
}

// Encodes the heads of a batch, v[u] of step s0 + u; every lane of the warp takes
// part.  One lane per scale makes it and its reciprocal for all.
template <int KIND, bool RUN, int LPH, int N>
__device__ __forceinline__ void encode(const F2 (&v)[N][4], unsigned char* dst, int64_t pitch, __half* scale, int h0,
                                       int H, int steps, int lane, int xa, int xb) {
  constexpr int D = 8 * LPH, HPW = 32 / LPH;
  const int sub = lane % LPH;
  if (KIND == SKV_KV_BF16) {
#pragma unroll
    for (int u = 0; u < N; u++) {
      const int h = h0 + u * HPW;
      if (u >= steps || h >= H) break;
      unsigned char* vec = dst + u * HPW * pitch;
      uint32_t w[4];
#pragma unroll
      for (int e = 0; e < 4; e++) w[e] = pack2(v[u][e]);
      if (RUN) {
        *reinterpret_cast<uint4*>(vec + 2 * xa) = make_uint4(w[0], w[1], w[2], w[3]);
      } else {
        *reinterpret_cast<uint2*>(vec + 2 * xa) = make_uint2(w[0], w[1]);
        *reinterpret_cast<uint2*>(vec + 2 * xb) = make_uint2(w[2], w[3]);
      }
    }
  } else if (KIND == SKV_KV_INT8) {
    const float mine = scale_max<LPH, N>(v, sub);
    const __half sh = scale_of<127>(mine);
    const float s_own = __half2float(sh), i_own = reciprocal(s_own);
    if (sub < steps && h0 + sub * HPW < H) scale[h0 + sub * HPW] = sh;
#pragma unroll
    for (int u = 0; u < N; u++) {
      if (u >= steps) break;
      const int from = lane - sub + u, h = h0 + u * HPW;
      uint32_t w[2];
      codes_of<127, true>(v[u], s_own, i_own, from, from, w);
      unsigned char* vec = dst + u * HPW * pitch;
      if (HPW > 1 && h >= H) continue;
      if (RUN) {
        *reinterpret_cast<uint2*>(vec + xa) = make_uint2(w[0], w[1]);
      } else {
        *reinterpret_cast<uint32_t*>(vec + xa) = w[0];
        *reinterpret_cast<uint32_t*>(vec + xb) = w[1];
      }
    }
  } else {
    static_assert(KIND != SKV_KV_INT4 || LPH == 32, "a warp per vector");
    // Lane 8 g + u: the scale of group g of step u.
    const int ga = xa >> 6, gb = xb >> 6;
    float mine = 0.f;
    if constexpr (RUN) {
      mine = scale_max<8, N>(v, lane & 7);
    } else {
#pragma unroll
      for (int u = 0; u < N; u++) {
        const float ma = amax<2>(&v[u][0]), mb = amax<2>(&v[u][2]);
#pragma unroll
        for (int g = 0; g < D / 64; g++) {
          const float all = lanes_max<32>(fmaxf(ga == g ? ma : 0.f, gb == g ? mb : 0.f));
          if (lane == 8 * g + u) mine = all;
        }
      }
    }
    const __half sh = scale_of<7>(mine);
    const float s_own = __half2float(sh), i_own = reciprocal(s_own);
    if ((lane & 7) < steps)
      *reinterpret_cast<uint16_t*>(dst + (lane & 7) * pitch + D / 2 + 2 * (lane >> 3)) = __half_as_ushort(sh);
#pragma unroll
    for (int u = 0; u < N; u++) {
      if (u >= steps) break;
      uint32_t w[2];
      codes_of<7, RUN>(v[u], s_own, i_own, 8 * ga + u, 8 * gb + u, w);
      w[0] &= 0x0f0f0f0fu;
      w[1] &= 0x0f0f0f0fu;
      w[0] |= w[0] >> 4;  // bytes 0 and 2 hold two codes each
      w[1] |= w[1] >> 4;
      unsigned char* vec = dst + u * pitch;
      if (RUN) {
        *reinterpret_cast<uint32_t*>(vec + xa / 2) = prmt(w[0], w[1], 0x6420u);
      } else {
        *reinterpret_cast<uint16_t*>(vec + xa / 2) = static_cast<uint16_t>(prmt(w[0], 0u, 0x0020u));
        *reinterpret_cast<uint16_t*>(vec + xb / 2) = static_cast<uint16_t>(prmt(w[1], 0u, 0x0020u));
      }
    }
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
    *reinterpret_cast<uint32_t*>(vec + xa / 2) = r.w[0];
    if ((xa & 63) == 0) *reinterpret_cast<uint16_t*>(vec + 4 * LPH + (xa >> 6) * 2) = r.s[0];
  }
}

// Steps [lo, hi) of one token's K or V.
template <int LPH, int SRC, int DST, bool INTER, Mode MODE>
__device__ __forceinline__ void run_heads(const MoveArgs& a, bool values, int64_t from, int64_t to, int lo, int hi,
                                          int lane, const float2* cs) {
  constexpr int D = 8 * LPH, HPW = 32 / LPH, N = kBatch<D, DST>;
  constexpr bool RUN = MODE != kTurn || INTER;
  const int sub = lane % LPH, grp = lane / LPH, half = a.rot / 2;
  const bool rotated = MODE == kTurn && sub < a.rot / 8;
  const int xa = !RUN && rotated ? 4 * sub : 8 * sub, xb = !RUN && rotated ? xa + half : xa + 4;
  const unsigned char* src = (values ? a.src.v : a.src.k) + from * a.src.token_pitch;
  unsigned char* dst = const_cast<unsigned char*>(values ? a.dst.v : a.dst.k) + to * a.dst.token_pitch;
  const __half* sscale = SRC == SKV_KV_INT8 ? (values ? a.src.v_scale : a.src.k_scale) + from * a.Hkv : nullptr;
  __half* dscale = DST == SKV_KV_INT8 ? const_cast<__half*>(values ? a.dst.v_scale : a.dst.k_scale) + to * a.Hkv : nullptr;
  // from head to head: known but for int4 rows
  const int64_t src_pitch = SRC == SKV_KV_BF16 ? 2 * D : SRC == SKV_KV_INT8 ? D : a.src.head_pitch;
  const int64_t dst_pitch = DST == SKV_KV_BF16 ? 2 * D : DST == SKV_KV_INT8 ? D : a.dst.head_pitch;
  for (int s0 = lo; s0 < hi; s0 += kLoad) {
    Raw raw[kLoad];
    const int h0 = s0 * HPW + grp;
    const unsigned char* src0 = src + h0 * src_pitch;
    unsigned char* dst0 = dst + h0 * dst_pitch;
    if (s0 + kLoad <= hi && (HPW == 1 || (s0 + kLoad) * HPW <= a.Hkv)) {  // every load first
#pragma unroll
      for (int u = 0; u < kLoad; u++) raw[u] = load<SRC, RUN>(src0 + u * HPW * src_pitch, sscale + h0 + u * HPW, xa, xb, D);
    } else {
#pragma unroll
      for (int u = 0; u < kLoad; u++) {
        const int h = h0 + u * HPW;
        raw[u] = Raw{};
        if (s0 + u < hi && h < a.Hkv) raw[u] = load<SRC, RUN>(src0 + u * HPW * src_pitch, sscale + h, xa, xb, D);
      }
    }
    if constexpr (MODE == kCopy) {
#pragma unroll
      for (int u = 0; u < kLoad; u++) {
        const int h = h0 + u * HPW;
        if (s0 + u < hi && (HPW == 1 || h < a.Hkv)) store<SRC, LPH>(raw[u], dst0 + u * HPW * dst_pitch, dscale + h, xa);
      }
    } else {
#pragma unroll
      for (int first = 0; first < kLoad; first += N) {
        if (s0 + first >= hi) break;
        F2 v[N][4];
#pragma unroll
        for (int u = 0; u < N; u++) decode<SRC, RUN>(raw[first + u], v[u]);
        if constexpr (MODE == kTurn) {
          if (rotated) {  // elsewhere an infinite neighbour would make 0 * inf
#pragma unroll
            for (int e = 0; e < (INTER ? 4 : 2); e++) {
              // of values 2 e, 2 e + 1 (and, halves, of their partners)
              const float2 c0 = cs[INTER ? xa / 2 + e : xa + 2 * e], c1 = INTER ? c0 : cs[xa + 2 * e + 1];
              const F2 co = f2(c0.x, c1.x), si = INTER ? f2(-c0.y, c0.y) : f2(c0.y, c1.y), ni = f2(-c0.y, -c1.y);
#pragma unroll
              for (int u = 0; u < N; u++) {
                const F2 p = v[u][e];
                if (INTER) {
                  const float2 x = f2_out(p);
                  v[u][e] = f2_fma(f2(x.y, x.x), si, f2_mul(p, co));
                } else {
                  const F2 q = v[u][e ^ 2];
                  v[u][e] = f2_fma(q, ni, f2_mul(p, co));
                  v[u][e ^ 2] = f2_fma(p, si, f2_mul(q, co));
                }
              }
            }
          }
        }
        encode<DST, RUN, LPH>(v, dst0 + first * HPW * dst_pitch, dst_pitch, dscale, h0 + first * HPW, a.Hkv,
                              min(N, hi - s0 - first), lane, xa, xb);
      }
    }
  }
}

template <int D, int SRC, int DST, bool INTER>
__global__ void __launch_bounds__(kThreads, ctas_per_sm(D, DST)) move_kernel(const MoveArgs a) {
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
  // First every token's keys, then every token's values, so that each warp gets
  // as much of the one as of the other.
  const uint32_t keys = static_cast<uint32_t>(a.n) * a.chunks_k, items = keys + static_cast<uint32_t>(a.n) * a.chunks_v;
  for (uint32_t item = blockIdx.x * kWarps + warp; item < items; item += gridDim.x * kWarps) {
    const bool values = item >= keys;
    const uint32_t i = values ? item - keys : item, chunks = values ? a.chunks_v : a.chunks_k;
    const uint32_t tok = chunks == 1 ? i : i / chunks;
    const int lo = static_cast<int>(i - tok * chunks) * a.chunk, hi = min(a.steps, lo + a.chunk);
    const int64_t from = a.src_rows ? a.src_rows[tok] : tok, to = a.dst_rows ? a.dst_rows[tok] : tok;
    if (from < 0 || to < 0) continue;  // padding
    if (from >= a.src.n_rows || to >= a.dst.n_rows) {
      if (lane == 0) set_status(a.status, SKV_DEV_RANGE);
      continue;
    }
    if (!values && a.turn) {
      const uint64_t old_pos = a.old_pos ? static_cast<int64_t>(a.old_pos[tok]) : 0;
      const uint64_t new_pos = a.new_pos ? static_cast<int64_t>(a.new_pos[tok]) : 0;
      __syncwarp();  // the previous token's values have been read
      for (int f = lane; f < half; f += 32)
        cs[warp][f] = cos_sin(static_cast<uint32_t>((new_pos * turns[1][f] - old_pos * turns[0][f]) >> 32));
      __syncwarp();
      run_heads<LPH, SRC, DST, INTER, kTurn>(a, false, from, to, lo, hi, lane, cs[warp]);
    } else {
      run_heads<LPH, SRC, DST, INTER, SRC == DST ? kCopy : kConvert>(a, values, from, to, lo, hi, lane, nullptr);
    }
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
    if (s->head_pitch < d / 2 + d / 32 || s->head_pitch > INT64_MAX / Hkv || s->token_pitch < Hkv * s->head_pitch)
      return SKV_EINVAL;
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
  if (n < 0 || n > 1 << 29 || Hkv < 1 || Hkv > 4096 || !src || !dst) return SKV_EINVAL;  // 32-bit work items
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
  const int hpw = 256 / d, parts = (src->k ? 1 : 0) + (src->v ? 1 : 0);
  a.steps = (Hkv + hpw - 1) / hpw;
  a.src_rows = src_rows;
  a.dst_rows = dst_rows;
  a.old_pos = old_positions;
  a.new_pos = new_positions;
  a.old_freq = old_inv_freq;
  a.new_freq = new_inv_freq;
  a.status = dev_status;
  // Work items: a token's K or V heads in pieces, so that the rounds of the
  // resident warps times the steps of a piece (each paying about three steps for
  // its rows and sines) come out lowest.
  const int per_sm = ctas_per_sm(d, dst->kind);
  const int64_t warps = static_cast<int64_t>(sms) * per_sm * kWarps;
  int64_t best = INT64_MAX;
  int chunks = 1;
  for (int c = 1; c <= a.steps; c++) {
    const int per = (a.steps + c - 1) / c, pieces = (a.steps + per - 1) / per;
    const int64_t cost = (n * parts * pieces + warps - 1) / warps * (per + 3);
    if (cost < best) {
      best = cost;
      a.chunk = per;
      chunks = pieces;
    }
    if (n * parts >= 16 * warps) break;  // whole tokens
  }
  a.chunks_k = src->k ? chunks : 0;
  a.chunks_v = src->v ? chunks : 0;
  const int64_t want = (n * parts * chunks + kWarps - 1) / kWarps;
  const int64_t cap = static_cast<int64_t>(sms) * per_sm;
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
