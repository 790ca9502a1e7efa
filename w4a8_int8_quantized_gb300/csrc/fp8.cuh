// The library's 8-bit float rows: e4m3 codes with one power-of-two scale (an
// e8m0 byte: 2^(byte - 127)) for every 128 consecutive elements of a row, the
// last group of a row possibly shorter.
//
// The scale of a group is the smallest 2^e with max|x| / 2^e <= 448 (the
// largest e4m3 value), 1 for a group of zeros, and at least 2^-126, so that
// 2^-e is a normal fp32 number too.  x / 2^e is then exact in fp32 (but for
// results below 2^-126), and the only rounding is the one to e4m3 (to nearest,
// ties to even): half a step, 2^-4 relative, or 2^-10 of the scale below 2^-6
// of it.  A power of two costs a float format nothing but up to one of the 17
// binades it spans, and the tensor core takes it as an operand, so that no sum
// is rescaled in a pass of its own.
#pragma once

#include <cuda_fp16.h>
#include <stdint.h>

namespace w8a8 {

constexpr int kFp8Group = 128;

// e8m0 byte of a group whose largest magnitude is a: a = 1.m 2^E against
// 448 = 1.75 2^8.
__device__ __forceinline__ uint32_t fp8_scale_byte(float a) {
  const uint32_t b = __float_as_uint(a);
  const int e = static_cast<int>(b >> 23) - 8 + ((b & 0x7fffffu) > 0x600000u ? 1 : 0);
  return a == 0.f ? 127u : static_cast<uint32_t>(e < 1 ? 1 : e);
}

// 1 / 2^(byte - 127), for bytes 1 .. 253
__device__ __forceinline__ float fp8_scale_inverse(uint32_t byte) {
  return __uint_as_float((254u - byte) << 23);
}

// Four e4m3 codes (element 0 in the low byte)
__device__ __forceinline__ uint32_t fp8_pack4(float a, float b, float c, float d) {
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
  return static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
}

// act(g) u, with act(g) = g / (1 + exp(-t)): t = g is SiLU; t = 2 sqrt(2 / pi)
// (g + 0.044715 g^3) is GELU in its tanh form, since (1 + tanh z) / 2 = 1 / (1 +
// exp(-2 z)).  exp and the reciprocal are the approximate ones (a few 2^-22
// relative for |t| below 16, and where |t| is larger the exponential hardly
// counts or the value is below 1e-6 of g): far inside one rounding to fp16 or
// e4m3, which follows.  From exp(-t) = 2^126 on (t below -87) the reciprocal, and
// with it the value, is 0.  Measured: with expf and a rounded division 2049 x 14336
// x 4096 to codes has the same errors against 64 bits (1.7e-5 of the codes beside a
// border, 3.06e-4 on the whole; they are the tensor core's sums) and takes 193 us
// instead of 159.
template <bool GELU>
__device__ __forceinline__ float gated(float g, float u) {
  const float t = GELU ? 1.5957691216057308f * fmaf(0.044715f * g * g, g, g) : g;
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + __expf(-t)));
  return g * r * u;
}

// The same for N pairs; which function is decided once.
template <int N>
__device__ __forceinline__ void gate_all(bool gelu, const float (&g)[N], const float (&u)[N], float (&h)[N]) {
  if (gelu) {
#pragma unroll
    for (int e = 0; e < N; ++e) h[e] = gated<true>(g[e], u[e]);
  } else {
#pragma unroll
    for (int e = 0; e < N; ++e) h[e] = gated<false>(g[e], u[e]);
  }
}

}  // namespace w8a8
