// FP8 with a scale for each block of 128: the element encoder and the launch interface of the
// FP8 kernels.
//
//   value = e4m3(code) * fp32 scale;  scale = rn(amax / 448) of its group;  code = e4m3(x / scale)
//
// Groups are 1 x 128 (activations: one row, 128 consecutive elements along K) or 128 x 128
// (weights).  The code is the E4M3 value nearest to the real quotient x / scale (ties to even),
// so it does not depend on how a kernel divides.
#pragma once

#include "common.cuh"

namespace nvfp4moe {

constexpr int FP8_BLOCK = 128;
constexpr float FP8_MAX = 448.0f;

inline int64_t fp8_blocks(int64_t n) { return (n + FP8_BLOCK - 1) / FP8_BLOCK; }

// |x| as an integer: ordered like the magnitudes, infinity above every finite value and NaN above
// infinity, so a maximum of these keeps a NaN.
__device__ __forceinline__ uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7FFFFFFFu; }

// How a group divides by its scale.  mul scales the element before the division (a power of two, so
// that residuals of very small groups stay normal numbers), s and inv are the scale times mul and
// its reciprocal; plain: divide with the IEEE operation (zero, infinite or NaN scales).
struct Fp8Scale {
  float scale, s, inv, mul;
  bool plain;
};

__device__ __forceinline__ Fp8Scale fp8_scale(uint32_t amax_bits) {
  Fp8Scale f;
  f.scale = __fdiv_rn(__uint_as_float(amax_bits), FP8_MAX);
  f.mul = f.scale < 0x1p-60f ? 0x1p96f : 1.0f;
  f.s = f.scale * f.mul;
  f.inv = __frcp_rn(f.s);
  f.plain = !(f.scale > 0.0f && f.scale < __uint_as_float(0x7F800000u));
  return f;
}

// A value on the same side of every E4M3 border as the real quotient x / scale.  q, one Newton
// step from x * inv, is one of the two fp32 values next to the quotient; where it is not exact
// (the residual r is not zero) the result is the neighbour towards zero with its last bit set.
// Borders have four or five significant bits, so the result is never a border unless the quotient is.
__device__ __forceinline__ float fp8_quotient(float x, const Fp8Scale& f) {
  const float xm = x * f.mul;
  const float q0 = xm * f.inv;
  const float q = __fmaf_rn(__fmaf_rn(-q0, f.s, xm), f.inv, q0);
  const float r = __fmaf_rn(-q, f.s, xm);
  uint32_t b = __float_as_uint(q);
  if (r != 0.0f) {
    // the quotient is nearer to zero than q when r's sign differs from q's; q = +-0 stays
    if (int32_t(__float_as_uint(r) ^ b) < 0 && (b & 0x7FFFFFFFu) != 0u) b -= 1u;
    b |= 1u;
  }
  return __uint_as_float(b);
}

// Zero scale: every code 0.  Infinite scale: 0 for finite x, NaN for an infinite one.  NaN: NaN.
__device__ __forceinline__ float fp8_quotient_plain(float x, const Fp8Scale& f) {
  return f.scale == 0.0f ? 0.0f : __fdiv_rn(x, f.scale);
}

// Four codes, v[0] in the low byte.
__device__ __forceinline__ uint32_t fp8_encode4(const float* v, const Fp8Scale& f) {
  if (f.plain)
    return e4m3x2_from_f32(fp8_quotient_plain(v[0], f), fp8_quotient_plain(v[1], f)) |
           (e4m3x2_from_f32(fp8_quotient_plain(v[2], f), fp8_quotient_plain(v[3], f)) << 16);
  return e4m3x2_from_f32(fp8_quotient(v[0], f), fp8_quotient(v[1], f)) |
         (e4m3x2_from_f32(fp8_quotient(v[2], f), fp8_quotient(v[3], f)) << 16);
}

}  // namespace nvfp4moe
