// attend_row.cuh — one query of chunk attention for one KV head by one warp,
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

// 8 dims of a stored token: dims 8 vec .. of token row r = (page * n_kv + head) *
// 16 + slot, as loaded and as fp32.
template <int DT>
struct Stored8 {
  uint2 w[DT == PKV_KV_Q8_0 ? 1 : 2];
  __half scale;  // q8_0
  __device__ __forceinline__ void load(const uint8_t* data, const uint8_t* scales, long long r, int vec) {
    if constexpr (DT == PKV_KV_Q8_0) {
      w[0] = *reinterpret_cast<const uint2*>(data + r * kD + 8 * vec);
      scale = reinterpret_cast<const __half*>(scales)[r * (kD / kQBlock) + vec / 4];
    } else {
      const uint4 v = *reinterpret_cast<const uint4*>(data + (r * kD + 8 * vec) * 2);
      w[0] = make_uint2(v.x, v.y);
      w[1] = make_uint2(v.z, v.w);
    }
  }
  // dims 4 half .. of the 8
  __device__ __forceinline__ void values(int half, float (&x)[4]) const {
    if constexpr (DT == PKV_KV_Q8_0) {
      const float sc = __half2float(scale);
      const uint32_t c = half ? w[0].y : w[0].x;
#pragma unroll
      for (int e = 0; e < 4; ++e) x[e] = sc * (static_cast<float>((c >> (8 * e)) & 255u) - 128.0f);
    } else {
      const uint2 v = half ? w[1] : w[0];
      if constexpr (DT == PKV_KV_BF16) {
        x[0] = __uint_as_float(v.x << 16);
        x[1] = __uint_as_float(v.x & 0xFFFF0000u);
        x[2] = __uint_as_float(v.y << 16);
        x[3] = __uint_as_float(v.y & 0xFFFF0000u);
      } else {
        const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&v.x));
        const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&v.y));
        x[0] = a.x; x[1] = a.y; x[2] = b.x; x[3] = b.y;
      }
    }
  }
};

// The tokens that attend_query visits: t stands for token(t), which it reads
// where seen(token).
struct AllSeen {
  static constexpr bool kAll = true;
  __device__ __forceinline__ int token(int t) const { return t; }
  __device__ __forceinline__ bool seen(int) const { return true; }
};

// The states of a query's G rows for KV head h (1, 2 or 4 query heads, which see
// the same tokens) over [t0, t1) of row i, those of them that `see` lets through
// (all, by default): running maximum m and sum l in base 2, and dims 4 lane .. +
// 3 of the unnormalised outputs.  q points at the first row's 128 dims (f16 or
// bf16), the others follow.  The whole warp must call it.
template <int DT, typename See = AllSeen>
__device__ __forceinline__ void attend_query(const PoolView& pool, const ChunkRows& rows, const ScoreArgs& sc, int i,
                                             int h, int G, int P, const uint8_t* q, int t0, int t1, float (&m)[4],
                                             float (&l)[4], float (&acc)[4][4], const See& see = See()) {
  constexpr int kIo = DT == PKV_KV_BF16 ? PKV_KV_BF16 : PKV_KV_F16;
  const int lane = threadIdx.x & 31;
  const int32_t* bt = rows.block_table + static_cast<long long>(i) * rows.bt_stride;
  float slope[4];
#pragma unroll
  for (int g = 0; g < 4; ++g) {
    slope[g] = sc.slopes && g < G ? __ldg(sc.slopes + h * G + g) : 0.0f;
    m[g] = -INFINITY;
    l[g] = 0.0f;
    acc[g][0] = acc[g][1] = acc[g][2] = acc[g][3] = 0.0f;
  }
  for (int base = t0; base < t1; base += 32) {
    const int t = see.token(base + lane);
    const bool in = base + lane < t1 && see.seen(t);
    const unsigned ins = See::kAll ? kFull : __ballot_sync(kFull, in);
    long long r = 0;
    float s[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY}, w[4];
    if (in) {
      int pg = __ldg(bt + t / kPage);
      if (pg < 0 || pg >= pool.num_pages) {
        record_status(pool.status, PKV_DEV_BAD_PAGE);
        pg = 0;
      }
      r = (static_cast<long long>(pg) * pool.n_kv + h) * kPage + t % kPage;
      float dot[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 1
      for (int v0 = 0; v0 < kD / 8; v0 += 8) {  // eight loads in flight
        Stored8<DT> k[8];
#pragma unroll
        for (int v = 0; v < 8; ++v) k[v].load(pool.k_data, pool.k_scales, r, v0 + v);
#pragma unroll
        for (int v = 0; v < 8; ++v) {
          float x[2][4], y[8];
          k[v].values(0, x[0]);
          k[v].values(1, x[1]);
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            if (g >= G) continue;
            load8(q, g * kD + 8 * (v0 + v), kIo, y);
#pragma unroll
            for (int e = 0; e < 8; ++e) dot[g] = fmaf(x[e >> 2][e & 3], y[e], dot[g]);
          }
        }
      }
#pragma unroll
      for (int g = 0; g < 4; ++g)
        if (g < G) s[g] = score2(dot[g], sc.scale, sc.softcap, slope[g], abs(P - t));
    }
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      w[g] = 0.0f;
      if (g >= G) continue;
      float mx = s[g];
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, o));
      const float mn = fmaxf(m[g], mx);
      const float base2 = mn == -INFINITY ? 0.0f : mn;  // every score so far -inf: weights 0
      const float al = exp2f(m[g] - base2);
      w[g] = in ? exp2f(s[g] - base2) : 0.0f;
      float sum = w[g];
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
      l[g] = l[g] * al + sum;
      m[g] = mn;
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[g][e] *= al;
    }
    const int n = min(32, t1 - base);
#pragma unroll 1
    for (int u0 = 0; u0 < n; u0 += 8) {  // eight loads in flight
      Stored8<DT> v[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) {  // behind the last token: the last, not used
        const long long ru = __shfl_sync(kFull, r, min(u0 + u, n - 1));
        v[u].load(pool.v_data, pool.v_scales, ru, lane >> 1);
      }
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        if (u0 + u >= n) break;
        if (!See::kAll && !(ins >> (u0 + u) & 1u)) continue;  // its value may be anything
        float x[4];
        v[u].values(lane & 1, x);
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          if (g >= G) continue;
          const float wu = __shfl_sync(kFull, w[g], u0 + u);
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[g][e] = fmaf(wu, x[e], acc[g][e]);
        }
      }
    }
  }
}

}  // namespace pkv
