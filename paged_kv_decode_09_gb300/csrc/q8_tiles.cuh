// q8_tiles.cuh — q8_0 tokens as two f16 operands of a tensor core product.
//
// A q8_0 value is scale * code, an f16 times an integer of 8 bits: up to 19
// significant bits, which one f16 (11 bits) would round.  It is split into hi =
// f16(scale * code) and lo = f16(scale * code - hi), exact but for lo's own
// rounding (2^-22 of the value; values near f16's smallest keep its absolute
// spacing), and a product takes both parts into the same accumulators.
//
// A scale below 512 keeps every value (128 codes of 511.75 are 65504) in f16's
// range.  Beyond, hi is infinite and lo its opposite, and products that meet
// them are NaN: the caller looks for such scales.
#pragma once

#include <cstdint>

#include "pkv_device.cuh"

namespace pkv {

// Magnitudes of a scale's 16 bits: 512, and the smallest that is not finite.
constexpr unsigned kLargeScale = 0x6000u;
constexpr unsigned kNotFinite = 0x7C00u;

// 8 codes (offset-binary bytes) times their block's scale (both halves of s):
// the hi and lo parts of 8 dims.
__device__ __forceinline__ void q8_split8(uint2 codes, __half2 s, uint4& hi, uint4& lo) {
  uint32_t h[4], l[4];
  const __half2 bias = __floats2half2_rn(1152.0f, 1152.0f);
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    // bytes 2e and 2e + 1 as the low mantissa bits of 1024 (0x6400): 1024 + code + 128
    const uint32_t w = e < 2 ? codes.x : codes.y;
    const uint32_t u = __byte_perm(w, 0x64646464u, (e & 1) ? 0x4342u : 0x4140u);
    const __half2 c = __hsub2(*reinterpret_cast<const __half2*>(&u), bias);
    const __half2 a = __hmul2(c, s);
    const __half2 b = __hfma2(c, s, __hneg2(a));
    h[e] = *reinterpret_cast<const uint32_t*>(&a);
    l[e] = *reinterpret_cast<const uint32_t*>(&b);
  }
  hi = make_uint4(h[0], h[1], h[2], h[3]);
  lo = make_uint4(l[0], l[1], l[2], l[3]);
}

// Byte offset of 16-byte vector c (dims 8c ..) of token row t in a block laid
// out as [token groups of 8][2 halves of 64 dims][8 tokens][128 bytes] under
// the 128-byte swizzle, as the 16-bit page copies land.
__device__ __forceinline__ uint32_t tile_vec(int t, int c) {
  return static_cast<uint32_t>((t >> 3) * 2048 + (c >> 3) * 1024 + (t & 7) * 128 + (((c & 7) ^ (t & 7)) << 4));
}

}  // namespace pkv
