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

// A block's sum v takes two scales, a and b.  Their fp32 product serves as one factor where it is an ordinary
// number (or either is zero).  Elsewhere it would lose bits that v * a * b need not lose, or overflow, and
// (v * first) * second is formed: of two large scales the smaller first, of two small ones the larger, so
// that the first product is an ordinary number wherever the result is (an infinite scale first: its sign and
// NaN stand).
__device__ __forceinline__ bool fp8_needs_both(float a, float b) {
  const uint32_t p = __float_as_uint(a * b) & 0x7FFFFFFFu;
  return p - 0x00800000u >= 0x7F000000u && a != 0.0f && b != 0.0f;
}
__device__ __forceinline__ void fp8_factors(float a, float b, float& first, float& second) {
  first = 1.0f, second = a * b;
  if (!fp8_needs_both(a, b)) return;
  const float large = fabsf(a) >= fabsf(b) ? a : b, small = fabsf(a) >= fabsf(b) ? b : a;
  const bool large_first = fabsf(second) < 1.0f || isinf(large);
  first = large_first ? large : small;
  second = large_first ? small : large;
}

// silu(g) u by e^-|g|, which is at most 1: 1 + e^-g leaves fp32's range (or the fast division's, 2^126) where
// the result need not.  The fast exponential is off by 2 + 1.2 |g| of 2^-23 (2^-19 at |g| = 12, 2^-17 at 88), before
// codes whose step is 2^-4 and more: expf took 138.0 us where this takes 134.0 (512 tokens, 512 experts 2048 x 512).
__device__ __forceinline__ float silu_times(float g, float u) {
  const float e = __expf(-fabsf(g));
  return __fdividef(g < 0.0f ? g * e : g, 1.0f + e) * u;
}

// How a group divides by its scale.  fast: the scale is an ordinary number; inv approximates its
// reciprocal to an ulp, and lo and hi are the reciprocal less and plus 2^-21 of it.  Otherwise (zero,
// tiny, infinite or NaN maxima) elements take the slow form.
struct Fp8Scale {
  float scale, inv, lo, hi;
  bool fast;
};

__device__ __forceinline__ Fp8Scale fp8_scale(uint32_t amax_bits) {
  Fp8Scale f;
  const float amax = __uint_as_float(amax_bits);
  f.fast = amax_bits >= 0x26800000u && amax_bits < 0x7F800000u;  // [2^-50, infinity)
  if (f.fast) {
    // rn(amax / 448): one residual step on amax * rn(1 / 448)
    constexpr float c = 1.0f / FP8_MAX;
    const float q = amax * c;
    f.scale = __fmaf_rn(__fmaf_rn(-FP8_MAX, q, amax), c, q);
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(f.inv) : "f"(f.scale));
  } else {
    f.scale = __fdiv_rn(amax, FP8_MAX);
    f.inv = 0.0f;
  }
  f.lo = f.inv * (1.0f - 0x1p-21f);
  f.hi = f.inv * (1.0f + 0x1p-21f);
  return f;
}

// A value on the same side of every E4M3 border as the real quotient x / s.  q, one Newton step from
// x * inv, is one of the two fp32 values next to the quotient; where it is not exact (the residual r
// is not zero) the result is the neighbour towards zero with its last bit set.  Borders have four or
// five significant bits, so the result is on one only if the quotient is.  (A quotient that
// underflows keeps the sign of x and stays below the smallest border.)
__device__ __forceinline__ float fp8_quotient(float x, float s, float inv) {
  const float q0 = x * inv;
  const float q = __fmaf_rn(__fmaf_rn(-q0, s, x), inv, q0);
  const float r = __fmaf_rn(-q, s, x);
  const int32_t b = __float_as_int(q);
  const int32_t odd = (b + ((__float_as_int(r) ^ b) >> 31)) | 1;  // towards zero when r's sign is not q's
  return r != 0.0f ? __int_as_float(odd) : q;
}

// Zero scale: 0.  Infinite: 0 for a finite x, NaN for an infinite one.  NaN: NaN.  Tiny: as above
// with both sides scaled up by 2^96, so that the residuals are ordinary numbers.
__device__ __forceinline__ float fp8_quotient_slow(float x, float scale) {
  if (scale == 0.0f) return 0.0f;
  if (!(scale < 1.0f)) return __fdiv_rn(x, scale);
  const float s = scale * 0x1p96f;
  return fp8_quotient(x * 0x1p96f, s, __frcp_rn(s));
}

static __device__ __noinline__ uint32_t fp8_encode4_exact(float v0, float v1, float v2, float v3, float scale, float inv,
                                                         bool fast) {
  const float v[4] = {v0, v1, v2, v3};
  float q[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) q[i] = fast ? fp8_quotient(v[i], scale, inv) : fp8_quotient_slow(v[i], scale);
  return e4m3x2_from_f32(q[0], q[1]) | (e4m3x2_from_f32(q[2], q[3]) << 16);
}

// Four codes, v[0] in the low byte.  The real quotients lie between v * lo and v * hi; where both
// round to the same codes those are the answer (four instructions an element), and where a border
// lies between (one element in 2^16, and ties) the exact form decides.
__device__ __forceinline__ uint32_t fp8_encode4(const float* v, const Fp8Scale& f) {
  const uint32_t lo = e4m3x2_from_f32(v[0] * f.lo, v[1] * f.lo) | (e4m3x2_from_f32(v[2] * f.lo, v[3] * f.lo) << 16);
  const uint32_t hi = e4m3x2_from_f32(v[0] * f.hi, v[1] * f.hi) | (e4m3x2_from_f32(v[2] * f.hi, v[3] * f.hi) << 16);
  if (lo == hi && f.fast) return lo;
  return fp8_encode4_exact(v[0], v[1], v[2], v[3], f.scale, f.inv, f.fast);
}

// The same codes for bf16 elements, without a branch.  With x = mx 2^i, amax = ma 2^j (integers below
// 256), 448 x / amax differs from a border t 2^k (t odd, below 32) by nothing or by more than 2^-13 of
// it: |7 mx 2^h - ma t| is 0 or at least 1.  Where it differs, any multiplier within 2^-20 of 1 / scale
// rounds to the right code.  Where it does not, x / scale lies on the side of the border that the
// scale's own rounding left it on, the same for the whole group: m is the reciprocal less 2^-21 of
// it if the scale was rounded up, plus 2^-21 if down; and if the scale is exact, so is the quotient,
// and a Newton step (n = the reciprocal, else 0) finds it.
struct Fp8ScaleBf16 {
  float scale, m, n;
  bool fast;
};

__device__ __forceinline__ Fp8ScaleBf16 fp8_scale_bf16(uint32_t amax_bits) {
  const Fp8Scale f = fp8_scale(amax_bits);
  const float r = __fmaf_rn(-FP8_MAX, f.scale, __uint_as_float(amax_bits));
  return Fp8ScaleBf16{f.scale, r > 0.0f ? f.hi : (r < 0.0f ? f.lo : f.inv), r == 0.0f ? f.inv : 0.0f, f.fast};
}

__device__ __forceinline__ uint32_t fp8_encode4(const float* v, const Fp8ScaleBf16& f) {
  if (!f.fast) return fp8_encode4_exact(v[0], v[1], v[2], v[3], f.scale, 0.0f, false);
  float q[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float q0 = v[i] * f.m;
    q[i] = __fmaf_rn(__fmaf_rn(-q0, f.scale, v[i]), f.n, q0);
  }
  return e4m3x2_from_f32(q[0], q[1]) | (e4m3x2_from_f32(q[2], q[3]) << 16);
}

// The list of row groups that the expert products run over, by one CTA of THREADS threads: {expert, first row,
// rows, -} for every `group` rows of every expert from groups[1] on, groups[0].x their number, and a zeroed
// counter for each where there are counters.  first(e), rows(e) of an expert; s_sum: a word a warp.
template <int THREADS, typename First, typename Rows>
__device__ __forceinline__ void fp8_list_groups(int E, int group, First first, Rows rows, int* s_sum, int4* groups,
                                                int* counters) {
  constexpr int PER = 1024 / THREADS;  // at most 1024 experts
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, e0 = int(threadIdx.x) * PER;
  int from[PER], n[PER], mine = 0;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    from[i] = e0 + i < E ? first(e0 + i) : 0;
    n[i] = e0 + i < E ? rows(e0 + i) : 0;
    mine += (n[i] + group - 1) / group;
  }
  int incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  __syncthreads();  // the scratch was read before
  if (lane == 31) s_sum[warp] = incl;
  __syncthreads();
  int at = incl - mine, total = 0;
  for (int w = 0; w < THREADS / 32; ++w) {
    if (w < warp) at += s_sum[w];
    total += s_sum[w];
  }
#pragma unroll
  for (int i = 0; i < PER; ++i)
    for (int r = 0; r < n[i]; r += group) groups[1 + at++] = make_int4(e0 + i, from[i] + r, min(group, n[i] - r), 0);
  if (threadIdx.x == 0) groups[0] = make_int4(total, 0, 0, 0);
  if (counters)
    for (int i = threadIdx.x; i < total; i += THREADS) counters[i] = 0;
}

// Eight bf16 elements as they are in memory: the largest magnitudes of them and of m, as pairs of bf16 bits
// (fp8_amax_bits: the larger of a pair as fp32 bits), and their codes.
__device__ __forceinline__ uint32_t bf16x8_max(uint32_t m, const uint4& q) {
  m = __vmaxu2(m, __vmaxu2(q.x & 0x7FFF7FFFu, q.y & 0x7FFF7FFFu));
  return __vmaxu2(m, __vmaxu2(q.z & 0x7FFF7FFFu, q.w & 0x7FFF7FFFu));
}
__device__ __forceinline__ uint32_t fp8_amax_bits(uint32_t pair) { return max(pair << 16, pair & 0xFFFF0000u); }
__device__ __forceinline__ uint2 fp8_encode8(const uint4& q, const Fp8ScaleBf16& f) {
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
  float v[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
  return make_uint2(fp8_encode4(v, f), fp8_encode4(v + 4, f));
}

}  // namespace nvfp4moe
