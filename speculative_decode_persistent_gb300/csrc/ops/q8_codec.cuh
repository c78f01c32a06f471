// The q8 block codec of the KV pool: 32 codes and one binary16 scale, in single
// precision only and exactly as defined in 64 bits.
#pragma once

#include <cuda_fp16.h>

#include <cstdint>

#include "sm103.cuh"

namespace mk {
namespace ops {

// binary16 nearest to amax / 127 (ties to even): a candidate at most one step
// off, then the exact comparison of amax with 127 x the midpoints to its
// neighbours (at most 19 significant bits, so exact).
static __device__ __noinline__ float q8_scale_near(float amax, float hf) {
  const unsigned u = __half_as_ushort(__float2half_rn(hf));
  unsigned r = u;
  auto value = [](unsigned b) {  // binary16's infinity as the value it would have one step up
    return b < 0x7c00u ? __half2float(__ushort_as_half(static_cast<unsigned short>(b))) : 65536.0f;
  };
  if (u < 0x7c00u) {
    const float pm = 127.0f * (0.5f * (value(u) + value(u + 1)));
    if (amax > pm || (amax == pm && (u & 1u))) r = u + 1;
  }
  if (u > 0) {
    const float pm = 127.0f * (0.5f * (value(u - 1) + value(u)));
    if (amax < pm || (amax == pm && (u & 1u))) r = u - 1;
  }
  return __half2float(__ushort_as_half(static_cast<unsigned short>(r)));
}
// The same as a float. With 2^e <= hf < 2^(e+1) (or binary16's least normal
// exponent) the midpoints lie 2^(e-11) away, or half that below a power of
// two; the remainder amax - 127 hf is exact. What is not clearly inside goes
// through the comparison above.
__device__ __forceinline__ float q8_scale(float amax) {
  const float hf = __half2float(__float2half_rn(amax * (1.0f / 127.0f)));
  const uint32_t bits = __float_as_uint(hf);
  const float step = fmaxf(__uint_as_float(bits & 0x7f800000u), 6.103515625e-05f) * (127.0f / 2048.0f);
  const float r = fmaf(-127.0f, hf, amax);
  return fabsf(r) < step && (r >= 0.f || (bits & 0x7fffffu)) ? hf : q8_scale_near(amax, hf);
}

// round-half-even of x / d clamped to [-127, 127], exactly: the rounded
// single-precision quotient is at most one step off, and the exact remainder
// x - q d (q d has at most 19 significant bits) says in which direction.
static __device__ __noinline__ int q8_code(float x, float d) {
  if (d == 0.f) return 0;
  float q = rintf(x / d);
  const float r = fmaf(-q, d, x), h = 0.5f * d;
  const bool odd = (static_cast<int>(q) & 1) != 0;
  if (r > h || (r == h && odd)) q += 1.f;
  else if (r < -h || (r == -h && odd)) q -= 1.f;
  return static_cast<int>(fminf(fmaxf(q, -127.f), 127.f));
}

// N codes (a multiple of four) of values of one block, packed four to a word.
// x inv + 1.5 x 2^23 rounds to the nearest integer and leaves it in the low
// bits; it is right unless the remainder reaches half a step. Such values,
// NaN, and blocks whose scale is 0, not finite or so small that its own
// rounding takes codes past 127 go through q8_code.
template <int N>
__device__ __forceinline__ void q8_codes(const float* x, float d, float amax, uint32_t* words) {
  constexpr float kMagic = 12582912.0f;
  float inv;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(d));
  const float below = __uint_as_float(__float_as_uint(0.5f * d) - 1u);
  bool sure = amax <= 127.25f * d && d > 0.f && d < 65520.f;
  uint32_t t[N];
  const uint64_t inv2 = pack2(inv, inv), d2 = pack2(d, d), magic2 = pack2(kMagic, kMagic), one2 = pack2(-1.f, -1.f);
#pragma unroll
  for (int i = 0; i < N; i += 2) {
    const uint64_t x2 = pack2(x[i], x[i + 1]), y2 = fma2(x2, inv2, magic2);
    const uint64_t r2 = fma2(fma2(y2, one2, magic2), d2, x2);  // x - q d
    float y0, y1, r0, r1;
    unpack2(y2, y0, y1);
    unpack2(r2, r0, r1);
    t[i] = __float_as_uint(y0);
    t[i + 1] = __float_as_uint(y1);
    sure = sure && fabsf(r0) <= below && fabsf(r1) <= below;  // false for NaN
  }
  if (!sure) {
#pragma unroll  // (indexed by a loop the values would live in local memory)
    for (int i = 0; i < N; ++i) t[i] = static_cast<uint32_t>(q8_code(x[i], d));
  }
#pragma unroll
  for (int i = 0; i < N; i += 4)
    words[i / 4] = __byte_perm(__byte_perm(t[i], t[i + 1], 0x0040), __byte_perm(t[i + 2], t[i + 3], 0x0040), 0x5410);
}

}  // namespace ops
}  // namespace mk
