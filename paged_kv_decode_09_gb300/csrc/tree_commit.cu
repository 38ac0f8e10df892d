// tree_commit.cu — kv_tree_commit: the accepted path of each row's drafted tree
// moved to the front of the row's drafted slots, in every layer.
//
// With path_0 < path_1 < .. < path_{a-1} the ancestors of the accepted leaf and
// the leaf itself, and C the slots before the drafted ones,
//     slot C + d  <-  slot C + path_d,   d = 0 .. a - 1
// for K, V and their scales.  path_d >= d, and from the first d with path_d > d
// on every token moves.  The moves overlap (a slot is read as one d's source and
// written as another's destination), but always forward: the destinations of d <
// e lie before the sources of d >= e, so a warp takes the tokens of a layer, KV
// head and side in ascending batches, each loaded whole before it is stored.
//
// A CTA takes a row and a share of the layers' (KV head, K or V) pairs: it walks
// the path once, from the parents up to the leaf in shared memory, and looks the
// pages up once.
#include <cstdint>

#include "chunk_device.cuh"

namespace pkv {
namespace {

constexpr int kWarps = 8;
constexpr int kInFlight = 8;  // 16-byte loads a lane

template <int DT>
__global__ void __launch_bounds__(32 * kWarps) tree_commit_kernel(const __grid_constant__ CommitArgs a) {
  constexpr int kRow = DT == PKV_KV_F32 ? 512 : DT == PKV_KV_Q8_0 ? 128 : 256;  // bytes of a token of a head
  constexpr int kLanes = kRow / 16, kTokens = 32 / kLanes;                      // lanes of a token, tokens of a load
  __shared__ int parents[PKV_MAX_TREE_TOKENS];  // later the pages of the path's tokens
  __shared__ int line[PKV_MAX_TREE_TOKENS];     // the path, at the end; later the pages they move to
  __shared__ int path[PKV_MAX_TREE_TOKENS];
  __shared__ int length;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, i = blockIdx.x;
  const bool first = blockIdx.y == 0;  // of the row's CTAs: records and reports
  grid_dependency_wait();
  grid_launch_dependents();
  int leaf = __ldg(a.leaves + i);
  const RowInfo r = row_info(a.rows, i, first && tid == 0 ? a.pool.status : nullptr);
  if (r.L < 0) {
    if (first && tid == 0) a.new_lens[i] = __ldg(a.rows.seq_lens + i);
    return;
  }
  int32_t* status = first ? a.pool.status : nullptr;
  const int C = r.L - r.n;
  if (leaf < -1 || leaf >= r.n) {
    if (tid == 0) record_status(status, PKV_DEV_BAD_TREE);
    leaf = -1;
  }
  for (int j = tid; j <= leaf; j += blockDim.x) parents[j] = __ldg(a.parents + r.start + j);
  __syncthreads();
  if (tid == 0) {
    int n = 0;
    for (int x = leaf; x >= 0; ++n) {
      line[PKV_MAX_TREE_TOKENS - 1 - n] = x;
      const int p = parents[x];
      if (p >= x || p < -1) record_status(status, PKV_DEV_BAD_TREE);
      x = p < x ? p : -1;
    }
    length = n;
  }
  __syncthreads();
  const int n = length;
  const int32_t* bt = a.rows.block_table + static_cast<long long>(i) * a.rows.bt_stride;
  int still = 0;  // tokens that stay where they are
  for (int d0 = 0; d0 < n; d0 += blockDim.x) {
    const int d = d0 + tid;
    int x = -1;
    if (d < n) {
      x = line[PKV_MAX_TREE_TOKENS - n + d];
      path[d] = x;
      if (first && a.path && d < a.path_stride) a.path[static_cast<long long>(i) * a.path_stride + d] = x;
    }
    still += __syncthreads_count(x == d);
  }
  if (first && tid == 0) a.new_lens[i] = C + n;
  for (int d = still + tid; d < n; d += blockDim.x) {  // line and parents are read: the pages of the moves
    const int from = __ldg(bt + (C + path[d]) / kPage), to = __ldg(bt + (C + d) / kPage);
    const bool ok = from >= 0 && from < a.pool.num_pages && to >= 0 && to < a.pool.num_pages;
    if (!ok) record_status(status, PKV_DEV_BAD_PAGE);
    parents[d] = ok ? from : -1;
    line[d] = to;
  }
  __syncthreads();

  const int pairs = 2 * a.pool.n_kv, all = a.layers * pairs;
  for (int u = blockIdx.y * kWarps + warp; u < all; u += gridDim.y * kWarps) {
    const int layer = u / pairs, pair = u - layer * pairs, h = pair >> 1;
    uint8_t* data = ((pair & 1) ? a.pool.v_data : a.pool.k_data) + layer * a.data_bytes;
    auto row_of = [&](int page, int slot) {
      return (static_cast<long long>(page) * a.pool.n_kv + h) * kPage + slot % kPage;
    };
    const int mine = lane / kLanes, vec = lane % kLanes;
    for (int d0 = still; d0 < n; d0 += kTokens * kInFlight) {
      uint4 w[kInFlight];
#pragma unroll
      for (int e = 0; e < kInFlight; ++e) {
        const int d = d0 + e * kTokens + mine;
        if (d < n && parents[d] >= 0)
          w[e] = *reinterpret_cast<const uint4*>(data + row_of(parents[d], C + path[d]) * kRow + 16 * vec);
      }
      __syncwarp();
#pragma unroll
      for (int e = 0; e < kInFlight; ++e) {
        const int d = d0 + e * kTokens + mine;
        if (d < n && parents[d] >= 0)
          *reinterpret_cast<uint4*>(data + row_of(line[d], C + d) * kRow + 16 * vec) = w[e];
      }
      __syncwarp();
    }
    if constexpr (DT == PKV_KV_Q8_0) {  // four f16 scales a token
      uint8_t* scales = ((pair & 1) ? a.pool.v_scales : a.pool.k_scales) + layer * a.scale_bytes;
      for (int d0 = still; d0 < n; d0 += 32) {
        const int d = d0 + lane;
        const bool ok = d < n && parents[d] >= 0;
        uint2 w = make_uint2(0u, 0u);
        if (ok) w = *reinterpret_cast<const uint2*>(scales + row_of(parents[d], C + path[d]) * 8);
        __syncwarp();
        if (ok) *reinterpret_cast<uint2*>(scales + row_of(line[d], C + d) * 8) = w;
        __syncwarp();
      }
    }
  }
}

template <int DT>
cudaError_t launch(const CommitArgs& a, cudaStream_t st) {
  const int groups = (a.layers * 2 * a.pool.n_kv + kWarps - 1) / kWarps;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(a.rows.num_rows, groups < 1 ? 1 : groups < 65535 ? groups : 65535);
  cfg.blockDim = dim3(32 * kWarps);
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, tree_commit_kernel<DT>, a);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

cudaError_t launch_tree_commit(const CommitArgs& a, cudaStream_t st) {
  switch (a.pool.dtype) {
    case PKV_KV_F32: return launch<PKV_KV_F32>(a, st);
    case PKV_KV_Q8_0: return launch<PKV_KV_Q8_0>(a, st);
    default: return launch<PKV_KV_F16>(a, st);  // bf16 values move like f16 ones
  }
}

}  // namespace pkv
