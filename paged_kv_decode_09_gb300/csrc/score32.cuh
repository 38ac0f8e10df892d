// score32.cuh — capped scores, 32 at a time.
#pragma once

#include <cmath>

#include "tcgen05.cuh"

namespace pkv {

// Scores are small next to their cap, so cap2 tanh(k v) = v q(v^2) with a
// polynomial, fitted by least squares of the relative error at Chebyshev nodes.
// The arithmetic decides: an fp32 operation takes a scheduler one cycle for an
// element of a warp's row, where the exponential that follows takes four.

// |k v| <= 0.35: q of degree 3 (off by 4.3e-8 of the value, less than the fp32
// arithmetic), with k and cap2 in its coefficients.  A k that would take those
// out of the normal range has no near values.
struct NearCap {
  float q[4], most;
  __device__ __forceinline__ NearCap(float k, float cap2) {
    constexpr float kQ[4] = {1.0f, -0.333326429f, 0.132993743f, -0.0491235033f};
    float f = k * cap2;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      q[e] = kQ[e] * f;
      f *= k * k;
    }
    most = fabsf(k) > 1e-4f && fabsf(k) < 1e4f && fabsf(cap2) < 1e9f ? 0.35f / fabsf(k) : -1.0f;
  }
  // The largest magnitude that lets a lane take the near form, or the other
  // always.  The two differ in their last bits, so what does not count towards a
  // result must not choose between them: a lane of no row takes no part.
  __device__ __forceinline__ float limit(bool live, bool near = true) const {
    return !live ? INFINITY : near ? most : -1.0f;
  }
  // a value of the warp is beyond its lane's limit
  static __device__ __forceinline__ bool beyond(const float (&v)[32], float limit) {
    float m0 = 0.0f, m1 = 0.0f;
#pragma unroll
    for (int e = 0; e < 32; e += 4) {
      m0 = tc::max3(m0, fabsf(v[e]), fabsf(v[e + 1]));
      m1 = tc::max3(m1, fabsf(v[e + 2]), fabsf(v[e + 3]));
    }
    return __any_sync(kFull, fmaxf(m0, m1) > limit);
  }
};

constexpr float kTanhNear = 0.7f;

// v = cap2 * tanh(k v) for any v, for the warp's 32 lanes: |k v| <= 0.7 by a
// polynomial of degree 5 (off by 2.8e-8 of the value).  A group with a value beyond takes
// 1 - 2 / (1 + e^2z) for such values, which loses the low bits of small ones, in
// a loop over 16 columns of tensor memory (tS: the columns that v was loaded
// from, free to be written): few instructions, seldom run.  A near value gets
// the same bits there, whatever the others are.  Not finite stays not finite,
// or +-cap2.
__device__ __forceinline__ void cap32(float (&v)[32], uint32_t tS, float k, float cap2) {
  constexpr float kQ[6] = {1.0f, -0.333331257f, 0.133283168f, -0.0535204448f, 0.0200115982f, -0.00507791527f};
  float m0 = 0.0f, m1 = 0.0f;
#pragma unroll
  for (int e = 0; e < 32; e += 4) {
    m0 = tc::max3(m0, fabsf(v[e]), fabsf(v[e + 1]));
    m1 = tc::max3(m1, fabsf(v[e + 2]), fabsf(v[e + 3]));
  }
  const float kc = k * cap2;
  if (__builtin_expect(__any_sync(kFull, fmaxf(m0, m1) * fabsf(k) > kTanhNear), 0)) {
    tc::st32(tS, v);
    tc::wait_st();
#pragma unroll 1
    for (int c = 0; c < 32; c += 16) {
      uint32_t w[16];
      tc::ld16w(tS + c, w);
      tc::wait_ld();
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const float x = __uint_as_float(w[e]), z = x * k, z2 = z * z;
        float q = kc * kQ[5];
#pragma unroll
        for (int i = 4; i >= 0; --i) q = fmaf(q, z2, kc * kQ[i]);
        const float t = 1.0f - __fdividef(2.0f, 1.0f + tc::ex2(z * 2.8853900817779268f));
        w[e] = __float_as_uint(fabsf(z) <= kTanhNear ? x * q : t * cap2);
      }
      tc::st16(tS + c, w);
    }
    tc::wait_st();
    tc::ld32(tS, v);
    tc::wait_ld();
    return;
  }
  const float2 zero = make_float2(0.0f, 0.0f), kk = make_float2(k, k);
#pragma unroll
  for (int e = 0; e < 32; e += 2) {
    const float2 x = make_float2(v[e], v[e + 1]);
    const float2 z = tc::fma2(x, kk, zero), w = tc::fma2(z, z, zero);
    float2 q = make_float2(kc * kQ[5], kc * kQ[5]);
#pragma unroll
    for (int i = 4; i >= 0; --i) q = tc::fma2(q, w, make_float2(kc * kQ[i], kc * kQ[i]));
    const float2 y = tc::fma2(x, q, zero);
    v[e] = y.x;
    v[e + 1] = y.y;
  }
}

}  // namespace pkv
