// Symmetric integer codes of a row of values (a token's activations, one head
// of a token's key or value), shared by the token and cache quantizers.
//
//   amax = max |x|, scale = amax / top (fp32, correctly rounded), top = 2^(b-1) - 1
//   code = the integer nearest to top x / amax, ties to the even one
// The code is that of the exact quotient: it is first taken from an fp32
// product, whose error is under 2^-16 of a step (two roundings of 2^-24 on at
// most 127), and where that lies within 2^-15 of a rounding border the two sides
// 2 top |x| and (2 k + 1) amax are compared in fp64, which holds both exactly.
// A row of zeros has scale 0 and codes 0; a row with a NaN or an infinity has
// scale NaN and codes 0.
// The kernels that use it would be bound by these instructions before HBM:
// adding 3 2^22 rounds to the nearest even integer and leaves it in the low
// byte, and eight values share one test for the border.
#pragma once

#include "gptq_common.h"

namespace gptq {

// max of |x| is kept on the bit patterns: ordered like the magnitudes, and
// NaN and infinity stay visible (>= 0x7F800000)
GPTQ_DEV uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7FFFFFFFu; }

struct RowScale {
  float amax;   // exact, times 2^100 for rows below 2^-60 (the same ratio, and no fp32 overflow of 1 / amax)
  float mul;    // 1 or 2^100: what x is multiplied by
  float inv;    // top / amax in fp32; 0 for a row of zeros or one that is not finite
  float scale;  // what is stored
};

GPTQ_DEV RowScale row_scale(uint32_t amax_bits, float top) {
  RowScale r;
  const float a = __uint_as_float(amax_bits);
  const bool finite = amax_bits < 0x7F800000u;
  r.mul = (a < 0x1p-60f) ? 0x1p100f : 1.0f;
  r.amax = a * r.mul;
  r.inv = (finite && amax_bits != 0u) ? top / r.amax : 0.0f;
  r.scale = finite ? __fdiv_rn(a, top) : __uint_as_float(0x7FC00000u);
  return r;
}

// the code of xs (times r.mul already) next to the border: t is the product that lies there
template <int TOP>
GPTQ_DEV int border_code(float xs, float t, const RowScale& r) {
  const float lo = floorf(fabsf(t));
  const double a = static_cast<double>(fabsf(xs)) * (2 * TOP);
  const double b = static_cast<double>(r.amax) * static_cast<double>(2.0f * lo + 1.0f);
  const bool odd = (static_cast<int>(lo) & 1) != 0;
  const float m = (a > b || (a == b && odd)) ? lo + 1.0f : lo;
  return static_cast<int>(copysignf(m, t));
}

// the codes of eight values, plus BIAS, as bytes of two words
template <int TOP, int BIAS>
GPTQ_DEV void row_codes(const float (&x)[8], const RowScale& r, uint32_t (&w)[2]) {
  constexpr float kMagic = 12582912.f + BIAS;  // 3 2^22
  float v[8], t[8], most = 0.f;
  uint32_t f[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = x[i];
  if (r.mul != 1.0f) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] *= r.mul;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    t[i] = v[i] * r.inv;
    const float s = t[i] + kMagic;
    f[i] = __float_as_uint(s);
    most = fmaxf(most, fabsf(t[i] - (s - kMagic)));
  }
  constexpr float kNear = 0.5f - 0x1p-15f;
  if (most > kNear) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (fabsf(t[i] - (__uint_as_float(f[i]) - kMagic)) > kNear)
        f[i] = static_cast<uint32_t>(border_code<TOP>(v[i], t[i], r) + BIAS);
  }
#pragma unroll
  for (int i = 0; i < 2; ++i)
    w[i] = __builtin_amdgcn_perm(f[4 * i + 1], f[4 * i], 0x0C0C0400u) |
           __builtin_amdgcn_perm(f[4 * i + 3], f[4 * i + 2], 0x04000C0Cu);
  if (r.inv == 0.0f) w[0] = w[1] = static_cast<uint32_t>(BIAS) * 0x01010101u;  // zeros, or not finite
}

// max over the lanes l ^ 1, ... of a group of N lanes (N a power of two up to 64)
template <int N>
GPTQ_DEV uint32_t group_max(uint32_t v) {
#pragma unroll
  for (int s = 1; s < N; s <<= 1) v = max(v, static_cast<uint32_t>(__shfl_xor(static_cast<int>(v), s)));
  return v;
}
template <int N>
GPTQ_DEV int group_sum(int v) {
#pragma unroll
  for (int s = 1; s < N; s <<= 1) v += __shfl_xor(v, s);
  return v;
}

// eight consecutive values: 16 bytes of bf16 or 32 of fp32
template <bool BF16>
GPTQ_DEV void load8(const void* base, int64_t elem, float (&x)[8]) {
  if (BF16) {
    const u32x4_t v = *reinterpret_cast<const u32x4_t*>(static_cast<const uint16_t*>(base) + elem);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(v[i] << 16);
      x[2 * i + 1] = __uint_as_float(v[i] & 0xFFFF0000u);
    }
  } else {
    const f32x4_t* p = reinterpret_cast<const f32x4_t*>(static_cast<const float*>(base) + elem);
    const f32x4_t a = p[0], b = p[1];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[i] = a[i];
      x[4 + i] = b[i];
    }
  }
}

template <bool BF16>
GPTQ_DEV float load1(const void* base, int64_t elem) {
  return BF16 ? bf16_to_f32(static_cast<const uint16_t*>(base)[elem]) : static_cast<const float*>(base)[elem];
}

// fp32 -> bf16, NaN kept (f32_to_bf16_rn is for finite values)
GPTQ_DEV uint16_t f32_to_bf16(float x) {
  const uint16_t r = f32_to_bf16_rn(x);
  return (x != x) ? static_cast<uint16_t>(0x7FC0u) : r;
}

}  // namespace gptq
