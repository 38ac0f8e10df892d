// attend_row.cuh — one (query, query head) row of chunk attention by one warp,
// straight from the pages: a token per lane for the scores, four dims per lane
// for the values.  Only tokens the query attends to are read.
#pragma once

#include <cmath>

#include "chunk_device.cuh"

namespace pkv {

// Score of a product <q, K>, in base 2 (see pkv_scores).
__device__ __forceinline__ float score2(float dot, float scale, float softcap, float slope, int dist) {
  float s = dot * scale;
  if (softcap > 0.0f) s = softcap * tanhf(s / softcap);
  return (s - slope * static_cast<float>(dist)) * kLog2e;
}

// 8 dims from 8 * vec of a stored token row (r = (page * n_kv + head) * 16 +
// slot) as fp32.
template <int DT>
__device__ __forceinline__ void load_kv8(const uint8_t* data, const uint8_t* scales, long long r, int vec,
                                         float (&x)[8]) {
  if constexpr (DT == PKV_KV_Q8_0) {
    const uint2 w = *reinterpret_cast<const uint2*>(data + r * kD + 8 * vec);
    const float sc = __half2float(reinterpret_cast<const __half*>(scales)[r * (kD / kQBlock) + vec / 4]);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const uint32_t b = ((e < 4 ? w.x : w.y) >> (8 * (e & 3))) & 255u;
      x[e] = sc * (static_cast<float>(b) - 128.0f);
    }
  } else {
    load8(data, r * kD + 8 * vec, DT, x);
  }
}

// The state of a row over the tokens [t0, t1) of row i (all attended): running
// maximum m and sum l in base 2, and dims 4 lane .. + 3 of the unnormalised
// output.  q points at the row's 128 dims (f16 or bf16).  The whole warp must
// call it.
template <int DT>
__device__ __forceinline__ void attend_row(const PoolView& pool, const ChunkRows& rows, const ScoreArgs& sc, int i,
                                           int h, float slope, int P, const uint8_t* q, int t0, int t1, float& m,
                                           float& l, float (&acc)[4]) {
  constexpr int kIo = DT == PKV_KV_BF16 ? PKV_KV_BF16 : PKV_KV_F16;
  const int lane = threadIdx.x & 31;
  const int32_t* bt = rows.block_table + static_cast<long long>(i) * rows.bt_stride;
  m = -INFINITY;
  l = 0.0f;
  acc[0] = acc[1] = acc[2] = acc[3] = 0.0f;
  for (int base = t0; base < t1; base += 32) {
    const int t = base + lane;
    const bool in = t < t1;
    long long r = 0;
    float s = -INFINITY;
    if (in) {
      int pg = __ldg(bt + t / kPage);
      if (pg < 0 || pg >= pool.num_pages) {
        record_status(pool.status, PKV_DEV_BAD_PAGE);
        pg = 0;
      }
      r = (static_cast<long long>(pg) * pool.n_kv + h) * kPage + t % kPage;
      float dot = 0.0f;
#pragma unroll 8
      for (int vec = 0; vec < kD / 8; ++vec) {
        float x[8], y[8];
        load_kv8<DT>(pool.k_data, pool.k_scales, r, vec, x);
        load8(q, 8 * vec, kIo, y);
#pragma unroll
        for (int e = 0; e < 8; ++e) dot = fmaf(x[e], y[e], dot);
      }
      s = score2(dot, sc.scale, sc.softcap, slope, abs(P - t));
    }
    float mx = s;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, o));
    const float mn = fmaxf(m, mx);
    const float base2 = mn == -INFINITY ? 0.0f : mn;  // every score so far -inf: weights 0
    const float al = exp2f(m - base2);
    const float p = in ? exp2f(s - base2) : 0.0f;
    float ps = p;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) ps += __shfl_xor_sync(kFull, ps, o);
    l = l * al + ps;
    m = mn;
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[e] *= al;
    const int n = min(32, t1 - base);
#pragma unroll 8
    for (int u = 0; u < n; ++u) {
      const float pu = __shfl_sync(kFull, p, u);
      const long long ru = __shfl_sync(kFull, r, u);
      float x[8];
      load_kv8<DT>(pool.v_data, pool.v_scales, ru, lane >> 1, x);
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[e] = fmaf(pu, (lane & 1) ? x[4 + e] : x[e], acc[e]);
    }
  }
}

}  // namespace pkv
