// rope.cuh -- angles of rotated positions, and pairs of bf16 values.
#pragma once

#include "common.cuh"

namespace skv {
namespace {

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

// (cos, sin) of an angle in turns, as the top 32 bits of its 64-bit fraction.
// Half turns: 31 bits, of which a float holds 24; the rest turns the result by a
// small angle (without it one more rounding to bf16 in 50000 falls to the other
// side).
__device__ __forceinline__ float2 cos_sin(uint32_t top) {
  const int32_t ht = static_cast<int32_t>(top);
  const float x = static_cast<float>(ht);
  const float rest = static_cast<float>(ht - static_cast<int32_t>(x)) * 1.4629180792671596e-9f;  // pi 2^-31
  float sn, cn;
  sincospif(x * 4.656612873077393e-10f, &sn, &cn);  // 2^-31
  return make_float2(fmaf(-sn, rest, cn), fmaf(cn, rest, sn));
}

}  // namespace
}  // namespace skv
