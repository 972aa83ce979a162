// The score rule's arithmetic, shared by the dense attention kernels.
#pragma once
#include "dense.h"
#include "ptx.cuh"

namespace spd {

// tanh(z) = z T(z^2).  T as polynomials fitted for least relative error:
// |z| <= 0.6, 5 terms (9.1e-8; 4.3 x 2^-24 with fp32 arithmetic), and |z| <= 1, 7
// terms (6.9e-8; 4.3 x 2^-24).  Beyond 1, 1 - 2 / (1 + e^2z) has no cancellation
// left (2 / (1 + e^2) = 0.24).
__device__ __forceinline__ float2 f2_dup(float x) { return make_float2(x, x); }

// cap tanh(s / cap) in base-2 units, for |s / cap| <= 0.6: two scores at once.
__device__ __forceinline__ float2 cap_small(const ScoreRule &r, float2 s) {
  const float2 z = f2_mul(s, f2_dup(r.z_in)), u = f2_mul(z, z);
  float2 p = f2_dup(r.poly[4]);
#pragma unroll
  for (int i = 3; i >= 0; --i) p = f2_fma(p, u, f2_dup(r.poly[i]));
  return f2_mul(z, p);
}

// The same for any score, by 2^x and a reciprocal: off by about 2^-22 of the cap
// near 0, which 16-bit weights (2^-9 and 2^-12 of each) do not show.
// cap tanh(s / cap) = cap - 2 cap / (1 + e^(2 s / cap)).  (8,192 capped tokens with a
// prefix of 30%: 804 us with this alone, 614 with cap_quick where it holds.)
__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float2 cap_16bit(const ScoreRule &r, float2 s) {
  const float2 x = f2_mul(s, f2_dup(r.e_in));
  const float2 e = f2_add(make_float2(ex2_approx(x.x), ex2_approx(x.y)), f2_dup(1.f));
  return f2_fma(make_float2(rcp_approx(e.x), rcp_approx(e.y)), f2_dup(-2.f * r.cap_out),
                f2_dup(r.cap_out));
}

// cap tanh(s / cap) + add in base-2 units by a polynomial of five terms in s^2 that
// is 6.1e-7 of the score off for |s / cap| <= 0.75, for the scores of a row whose
// largest lies in [-0.25, 0.75] cap, cap >= 30.  What lies below -0.75 cap has a
// weight under e^(-0.39 cap) of the largest; there the polynomial stays monotonic
// and on the lower side (8e-4 of the score at -cap, then falling away to 0 weight),
// an error of at most 5e-9 of the largest weight.
__device__ __forceinline__ float2 cap_quick(const ScoreRule &r, float2 s, float2 add) {
  const float2 u = f2_mul(s, s);
  float2 p = f2_dup(r.quick_poly[4]);
#pragma unroll
  for (int i = 3; i >= 0; --i) p = f2_fma(p, u, f2_dup(r.quick_poly[i]));
  return f2_fma(s, p, add);
}

// The same for any score, precise.
__device__ __forceinline__ float cap_any(const ScoreRule &r, float s) {
  constexpr float c[7] = {0.9999999403953552f,  -0.33332839608192444f, 0.13325203955173492f,
                          -0.05345702916383743f, 0.020289979875087738f, -0.006203378085047007f,
                          0.001041022245772183f};
  const float z = s * r.z_in, u = z * z;
  float p = c[6];
#pragma unroll
  for (int i = 5; i >= 0; --i) p = fmaf(p, u, c[i]);
  const float e = ex2_approx(fabsf(z) * 2.8853900817779268f);  // e^(2 |z|)
  const float far = copysignf(r.cap_out - __fdividef(2.f * r.cap_out, 1.f + e), s);
  // (a NaN score fails the comparison's negation and stays NaN through p)
  return fabsf(z) > 1.f ? far : s * r.scale_log2 * p;
}

}  // namespace spd
