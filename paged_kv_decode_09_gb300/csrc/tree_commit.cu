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
// pages up once, as rows of KV head 0 that every pair adds its own offset to.
//
// What bounds it: up to some MB the chain before the first move (the leaf, the
// parents, the walk, the table, the load, some 3 us); above, DRAM, in pieces of a
// token of a head (256 bytes; 512 in f32).  A row's 4 to 7 moves leave a warp few
// loads, so it takes those of several pairs together, but not of a layer or two (8
// rows of one layer 3.3 us, 4.0 together): 32 rows of 32 layers, 28.8 MB, 9.5 us
// in 1216 CTAs (9.9 in 304, 11.9 in 2048), with a pair at a time 10.7 (9.8 in 304,
// 13.6 in 2048); 192 rows of 16 layers in f32, 286 MB, 51.4 us, 5.6 TB/s (63 in
// 304 CTAs, 55.7 in 608).  In q8_0, 15.3 MB of the former rows, 13.3 us: the scales
// of a warp's pairs go one pair after the other, a trip to memory each.
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
  __shared__ int parents[PKV_MAX_TREE_TOKENS];
  __shared__ int line[PKV_MAX_TREE_TOKENS];  // the path, at the end
  __shared__ longlong2 moves[PKV_MAX_TREE_TOKENS];  // token rows of KV head 0 that move, and where to (-1: not)
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
      if (first && a.path && d < a.path_stride) a.path[static_cast<long long>(i) * a.path_stride + d] = x;
    }
    still += __syncthreads_count(x == d);
  }
  if (first && tid == 0) a.new_lens[i] = C + n;
  const int m = n - still;
  if (m == 0) return;
  for (int x = tid; x < m; x += blockDim.x) {
    const int src = C + line[PKV_MAX_TREE_TOKENS - m + x], dst = C + still + x;
    const int from = __ldg(bt + src / kPage), to = __ldg(bt + dst / kPage);
    const bool ok = from >= 0 && from < a.pool.num_pages && to >= 0 && to < a.pool.num_pages;
    if (!ok) record_status(status, PKV_DEV_BAD_PAGE);
    const long long step = static_cast<long long>(a.pool.n_kv) * kPage;
    moves[x] = make_longlong2(ok ? from * step + src % kPage : -1, ok ? to * step + dst % kPage : -1);
  }
  __syncthreads();

  // A unit is a layer's KV head and side.  A warp loads kBatch tokens before it
  // stores any: those of several units where they have few, else a unit's in turn.
  constexpr int kBatch = kTokens * kInFlight;
  const int pairs = 2 * a.pool.n_kv, units = a.layers * pairs;
  const int per = units >= 4 * kWarps ? max(1, kBatch / m) : 1;
  const int mine = lane / kLanes, vec = lane % kLanes;
  const int step = gridDim.y * kWarps * per;
  for (int u0 = (blockIdx.y * kWarps + warp) * per; u0 < units; u0 += step) {
    const int last = min(u0 + per, units), layer0 = u0 / pairs, pair0 = u0 - layer0 * pairs;
    for (int d0 = 0; d0 < m; d0 += kBatch) {
      uint4 w[kInFlight];
      uint8_t* to[kInFlight];
      int x = d0 + mine, unit = u0, layer = layer0, pair = pair0;  // this lane's move and its unit
#pragma unroll
      for (int e = 0; e < kInFlight; ++e, x += kTokens) {
        while (per > 1 && x >= m) {
          x -= m;
          ++unit;
          if (++pair == pairs) {
            pair = 0;
            ++layer;
          }
        }
        to[e] = nullptr;
        if (x < m && unit < last) {
          const longlong2 mv = moves[x];
          uint8_t* data = ((pair & 1) ? a.pool.v_data : a.pool.k_data) + layer * a.data_bytes +
                          (pair >> 1) * (kPage * kRow) + 16 * vec;
          if (mv.x >= 0) {
            w[e] = *reinterpret_cast<const uint4*>(data + mv.x * kRow);
            to[e] = data + mv.y * kRow;
          }
        }
      }
      __syncwarp();
#pragma unroll
      for (int e = 0; e < kInFlight; ++e)
        if (to[e]) *reinterpret_cast<uint4*>(to[e]) = w[e];
      __syncwarp();
    }
    if constexpr (DT == PKV_KV_Q8_0) {  // four f16 scales a token
      int layer = layer0, pair = pair0;
      for (int unit = u0; unit < last; ++unit) {
        uint8_t* scales = ((pair & 1) ? a.pool.v_scales : a.pool.k_scales) + layer * a.scale_bytes + (pair >> 1) * (kPage * 8);
        for (int d0 = 0; d0 < m; d0 += 32) {
          const longlong2 mv = d0 + lane < m ? moves[d0 + lane] : make_longlong2(-1, -1);
          uint2 w = make_uint2(0u, 0u);
          if (mv.x >= 0) w = *reinterpret_cast<const uint2*>(scales + mv.x * 8);
          __syncwarp();
          if (mv.x >= 0) *reinterpret_cast<uint2*>(scales + mv.y * 8) = w;
          __syncwarp();
        }
        if (++pair == pairs) {
          pair = 0;
          ++layer;
        }
      }
    }
  }
}

template <int DT>
cudaError_t launch(const CommitArgs& a, cudaStream_t st) {
  // Each CTA walks its row's path and looks its pages up before it moves anything: two waves of four an SM
  constexpr int kCtas = 2 * 4 * 152;
  const int groups = (a.layers * 2 * a.pool.n_kv + kWarps - 1) / kWarps;
  const int most = kCtas / a.rows.num_rows + 1;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(a.rows.num_rows, groups < 1 ? 1 : groups < most ? groups : most);
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
