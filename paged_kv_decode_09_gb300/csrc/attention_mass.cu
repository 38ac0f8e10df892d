// attention_mass.cu — paged_attention_mass: a warp per (cached token, KV head),
// four dims per lane, over the queries that attend to the token.
#include <cstdint>

#include "attend_row.cuh"
#include "chunk_device.cuh"

namespace pkv {
namespace {

constexpr int kMassWarps = 8;

template <int DT>
__global__ void __launch_bounds__(kMassWarps * 32) mass_rows_kernel(const __grid_constant__ MassArgs a) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int i = blockIdx.z, h = blockIdx.y;
  const int t = blockIdx.x * kMassWarps + warp;
  constexpr int kIo = DT == PKV_KV_BF16 ? PKV_KV_BF16 : PKV_KV_F16;
  if (blockIdx.x == 0 && i == 0 && h == 0) report_rows(a.rows, a.pool.status);
  const RowInfo r = row_info(a.rows, i, nullptr);
  if (r.L > a.mass_stride && t == 0 && h == 0 && lane == 0) record_status(a.pool.status, PKV_DEV_BAD_LENGTH);
  if (r.L < 0 || r.L > a.mass_stride || t >= r.L) return;
  const int G = a.n_q / a.pool.n_kv;
  const int F = a.sc.prefix_lens ? __ldg(a.sc.prefix_lens + i) : 0;
  int pg = __ldg(a.rows.block_table + static_cast<long long>(i) * a.rows.bt_stride + t / kPage);
  const int j0 = a.last_queries > 0 ? max(0, r.n - a.last_queries) : 0;
  float sum = 0.0f;
  bool read = false;
  float k[8];
  for (int j = j0; j < r.n; ++j) {
    const int P = r.L - r.n + j;
    if (t < seen_from(P, a.pool.window) || t >= seen_to(P, r.L, F)) continue;
    if (!read) {
      if (pg < 0 || pg >= a.pool.num_pages) {
        if (lane == 0) record_status(a.pool.status, PKV_DEV_BAD_PAGE);
        pg = 0;
      }
      load_kv8<DT>(a.pool.k_data, a.pool.k_scales, (static_cast<long long>(pg) * a.pool.n_kv + h) * kPage + t % kPage,
                   lane >> 1, k);
      read = true;
    }
    for (int g = h * G; g < (h + 1) * G; ++g) {
      float x[8];
      load8(a.q, (r.start + j) * a.q_stride + g * kD + 8 * (lane >> 1), kIo, x);
      float dot = 0.0f;
#pragma unroll
      for (int e = 0; e < 4; ++e) dot = fmaf((lane & 1) ? x[4 + e] : x[e], (lane & 1) ? k[4 + e] : k[e], dot);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(kFull, dot, o);
      const float slope = a.sc.slopes ? __ldg(a.sc.slopes + g) : 0.0f;
      const float lse = __ldg(a.lse + static_cast<long long>(r.start + j) * a.n_q + g);
      if (isfinite(lse)) sum += exp2f(score2(dot, a.sc.scale, a.sc.softcap, slope, abs(P - t)) - lse * kLog2e);
    }
  }
  if (lane == 0) {
    const long long at = (static_cast<long long>(i) * a.pool.n_kv + h) * a.mass_stride + t;
    a.mass_out[at] = (a.mass_in && t < r.L - r.n ? a.mass_in[at] : 0.0f) + sum;
  }
}

}  // namespace

cudaError_t launch_attention_mass(const MassArgs& a, const TileMaps&, cudaStream_t st) {
  const long long cap = static_cast<long long>(a.rows.bt_stride) * kPage;
  const long long most = a.mass_stride < cap ? a.mass_stride : cap;
  const dim3 grid(static_cast<unsigned>((most + kMassWarps - 1) / kMassWarps), a.pool.n_kv, a.rows.num_rows);
  if (a.pool.dtype == PKV_KV_F16)
    mass_rows_kernel<PKV_KV_F16><<<grid, kMassWarps * 32, 0, st>>>(a);
  else if (a.pool.dtype == PKV_KV_BF16)
    mass_rows_kernel<PKV_KV_BF16><<<grid, kMassWarps * 32, 0, st>>>(a);
  else
    mass_rows_kernel<PKV_KV_Q8_0><<<grid, kMassWarps * 32, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace pkv
