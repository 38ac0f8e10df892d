// chunk_attention.cu — paged_chunk_attention: a warp per (token, query head),
// straight from the pages (attend_row).
#include <cstdint>

#include "attend_row.cuh"
#include "chunk_device.cuh"

namespace pkv {
namespace {

constexpr int kRowWarps = 8;

template <int DT>
__global__ void __launch_bounds__(kRowWarps * 32) chunk_rows_kernel(const __grid_constant__ ChunkAttnArgs a) {
  __shared__ float qs[kRowWarps][kD];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (blockIdx.x == 0) report_rows(a.rows, a.pool.status);
  const long long item = static_cast<long long>(blockIdx.x) * kRowWarps + warp;
  const int tok = static_cast<int>(item / a.n_q), g = static_cast<int>(item % a.n_q);
  if (tok >= a.rows.total_tokens) return;
  constexpr int kIo = DT == PKV_KV_BF16 ? PKV_KV_BF16 : PKV_KV_F16;
  const int i = row_of_token(a.rows, tok);
  if (i < 0) return;
  const RowInfo r = row_info(a.rows, i, nullptr);
  if (r.n == 0) return;
  float m = -INFINITY, l = 0.0f, acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  if (r.L >= 0) {
    if (lane < kD / 8) {
      float x[8];
      load8(a.q, tok * a.q_stride + g * kD + 8 * lane, kIo, x);
#pragma unroll
      for (int e = 0; e < 8; ++e) qs[warp][8 * lane + e] = x[e];
    }
    __syncwarp();
    const int P = r.L - r.n + tok - r.start;
    const int F = a.sc.prefix_lens ? __ldg(a.sc.prefix_lens + i) : 0;
    const float slope = a.sc.slopes ? __ldg(a.sc.slopes + g) : 0.0f;
    attend_row<DT>(a.pool, a.rows, a.sc, i, g / (a.n_q / a.pool.n_kv), slope, P, qs[warp],
                   seen_from(P, a.pool.window), seen_to(P, r.L, F), m, l, acc);
  }
  const float inv = l > 0.0f ? 1.0f / l : 0.0f;
  const long long to = (static_cast<long long>(tok) * a.n_q + g) * kD + 4 * lane;
  uint32_t w[2];
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    if constexpr (kIo == PKV_KV_BF16) {
      const __nv_bfloat162 x = __floats2bfloat162_rn(acc[2 * e] * inv, acc[2 * e + 1] * inv);
      w[e] = *reinterpret_cast<const uint32_t*>(&x);
    } else {
      const __half2 x = __floats2half2_rn(acc[2 * e] * inv, acc[2 * e + 1] * inv);
      w[e] = *reinterpret_cast<const uint32_t*>(&x);
    }
  }
  *reinterpret_cast<uint2*>(a.out + to * 2) = make_uint2(w[0], w[1]);
  if (a.lse && lane == 0)
    a.lse[static_cast<long long>(tok) * a.n_q + g] = l > 0.0f ? (m + log2f(l)) * kLn2 : -INFINITY;
}

}  // namespace

size_t chunk_attention_workspace(int n_q, int n_kv, int chunks) { return 256; }

cudaError_t launch_chunk_attention(const ChunkAttnArgs& a, const TileMaps&, cudaStream_t st) {
  const long long items = static_cast<long long>(a.rows.total_tokens) * a.n_q;
  const dim3 grid(static_cast<unsigned>((items + kRowWarps - 1) / kRowWarps));
  if (a.pool.dtype == PKV_KV_F16)
    chunk_rows_kernel<PKV_KV_F16><<<grid, kRowWarps * 32, 0, st>>>(a);
  else if (a.pool.dtype == PKV_KV_BF16)
    chunk_rows_kernel<PKV_KV_BF16><<<grid, kRowWarps * 32, 0, st>>>(a);
  else
    chunk_rows_kernel<PKV_KV_Q8_0><<<grid, kRowWarps * 32, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace pkv
