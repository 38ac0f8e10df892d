// chunk_device.cuh — device helpers shared by the long-prompt kernels: rows of
// a ragged chunk, the tokens a query attends to, and vectors of 8 elements.
#pragma once

#include <cstdint>

#include "chunk_internal.h"
#include "pkv_device.cuh"

namespace pkv {

// A row of a chunk call: its tokens start .. start + n - 1 in the token arrays,
// the last n of its L cached tokens.
struct RowInfo {
  int start;  // cu_seqlens[i]
  int n;      // new tokens; 0 where cu_seqlens is not valid for the row
  int L;      // cached tokens, or -1 where the row is to be skipped
};

__device__ __forceinline__ RowInfo row_info(const ChunkRows& r, int i, int32_t* status) {
  RowInfo x;
  x.start = __ldg(r.cu + i);
  const int end = __ldg(r.cu + i + 1);
  x.L = __ldg(r.seq_lens + i);
  const bool valid = x.start >= 0 && end >= x.start && end <= r.total_tokens;
  x.n = valid ? end - x.start : 0;
  if (!valid || x.L < x.n || static_cast<long long>(x.L) > static_cast<long long>(r.bt_stride) * kPage) {
    record_status(status, PKV_DEV_BAD_LENGTH);
    x.L = -1;
  }
  return x;
}

// Records the rows that row_info rejects (the threads of one CTA share them).
__device__ __forceinline__ void report_rows(const ChunkRows& r, int32_t* status) {
  if (status)
    for (int i = threadIdx.x; i < r.num_rows; i += blockDim.x) row_info(r, i, status);
}

// The row holding token tok of the token arrays: the last row i with cu[i] <=
// tok, found by the warp (32 probes a round); -1 where that row does not hold
// it.  Every lane of the warp must call it with the same tok.
__device__ __forceinline__ int row_of_token(const ChunkRows& r, int tok) {
  const int lane = threadIdx.x & 31;
  int lo = 0, n = r.num_rows;  // the row lies in [lo, lo + n)
  while (n > 1) {
    const int step = (n + 31) / 32;
    const int at = lane * step;
    const bool le = at < n && __ldg(r.cu + lo + at) <= tok;
    const unsigned m = __ballot_sync(kFull, le);
    const int hit = m ? 31 - __clz(m) : 0;
    lo += hit * step;
    n = min(step, n - hit * step);
  }
  const bool in = tok >= __ldg(r.cu + lo) && tok < __ldg(r.cu + lo + 1);
  return in ? lo : -1;
}

// First token a query at position P attends to under window W (0: none), and
// the end of its range in a row of L tokens with a prefix of F.
__device__ __forceinline__ int seen_from(int P, int W) { return W > 0 && P + 1 > W ? P + 1 - W : 0; }
__device__ __forceinline__ int seen_to(int P, int L, int F) { return min(L, max(P + 1, F)); }

// log2(e) and its inverse: scores are kept in base 2.
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// 8 consecutive elements of a token array as fp32 (16-byte aligned).
__device__ __forceinline__ void load8(const uint8_t* base, long long elem, int dtype, float (&x)[8]) {
  if (dtype == PKV_KV_F32) {
    const float4* p = reinterpret_cast<const float4*>(base + elem * 4);
    const float4 a = p[0], b = p[1];
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
    return;
  }
  const uint4 w = *reinterpret_cast<const uint4*>(base + elem * 2);
  const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if (dtype == PKV_KV_BF16) {
      x[2 * e] = __uint_as_float(v[e] << 16);
      x[2 * e + 1] = __uint_as_float(v[e] & 0xFFFF0000u);
    } else {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&v[e]));
      x[2 * e] = f.x;
      x[2 * e + 1] = f.y;
    }
  }
}

// 8 fp32 values rounded (to nearest even) and stored as f16, bf16 or f32.
__device__ __forceinline__ void store8(uint8_t* base, long long elem, int dtype, const float (&x)[8]) {
  if (dtype == PKV_KV_F32) {
    float4* p = reinterpret_cast<float4*>(base + elem * 4);
    p[0] = make_float4(x[0], x[1], x[2], x[3]);
    p[1] = make_float4(x[4], x[5], x[6], x[7]);
    return;
  }
  uint32_t v[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if (dtype == PKV_KV_BF16) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * e], x[2 * e + 1]);
      v[e] = *reinterpret_cast<const uint32_t*>(&h);
    } else {
      const __half2 h = __floats2half2_rn(x[2 * e], x[2 * e + 1]);
      v[e] = *reinterpret_cast<const uint32_t*>(&h);
    }
  }
  *reinterpret_cast<uint4*>(base + elem * 2) = make_uint4(v[0], v[1], v[2], v[3]);
}

}  // namespace pkv
