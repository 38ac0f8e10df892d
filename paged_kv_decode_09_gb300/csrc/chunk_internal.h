// chunk_internal.h — argument blocks and launchers of the long-prompt operators
// (rope_append.cu, chunk_attention.cu, attention_mass.cu, evict.cu), shared
// with their C entries (chunk_api.cu).  Not installed.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "pkv_chunk.h"
#include "pkv_internal.h"

namespace pkv {

// One layer of a pool, as the C entries see it (api.cu).
struct PoolView {
  uint8_t* k_data;
  uint8_t* v_data;
  uint8_t* k_scales;  // q8_0 only
  uint8_t* v_scales;  // q8_0 only
  int num_pages;
  int n_kv;
  int dtype;
  int window;
  int32_t* status;
  unsigned long long test_stall_ns;  // test hook (kv_pool_set_test_stall); 0: off
};
pkv_status pool_layer_view(const pkv_pool* pool, int layer, PoolView* view);
pkv_status pool_layer_maps(const pkv_pool* pool, int layer, const TileMaps** maps);

// The rows of a chunk call.
struct ChunkRows {
  const int32_t* cu;  // [num_rows + 1]
  const int32_t* seq_lens;
  const int32_t* block_table;
  int bt_stride;
  int num_rows;
  int total_tokens;
};

struct RopeArgs {
  PoolView pool;
  ChunkRows rows;
  const uint8_t* q;
  const uint8_t* k;
  const uint8_t* v;
  long long q_stride, k_stride, v_stride;  // elements from token to token
  uint8_t* q_out;
  const int32_t* positions;  // [axes][total_tokens]
  const float* inv_freq;
  int in_dtype, q_dtype;
  int n_q;
  int half;                           // rot_dim / 2
  int axis_end[PKV_MAX_ROPE_AXES];    // pairs below axis_end[a] turn by axis a or an earlier one
  int interleaved;
};
cudaError_t launch_rope_append(const RopeArgs& a, cudaStream_t stream);

struct EvictArgs {
  PoolView pool;
  const float* mass;
  int mass_stride;
  const int32_t* block_table;
  int bt_stride;
  const int32_t* seq_lens;
  int num_rows;
  const int32_t* keep_lens;
  int first, recent;
  const int32_t* dst_block_table;
  int dst_bt_stride;
  int32_t* keep_idx;
  int keep_stride;
  float* dst_mass;
  int32_t* new_lens;
};
cudaError_t launch_evict(const EvictArgs& a, cudaStream_t stream);

// pkv_scores, as the kernels take them.
struct ScoreArgs {
  float scale;
  float softcap;
  const float* slopes;
  const int32_t* prefix_lens;
};

struct ChunkAttnArgs {
  PoolView pool;
  ChunkRows rows;
  const uint8_t* q;
  long long q_stride;
  int n_q;
  ScoreArgs sc;
  uint8_t* out;
  float* lse;  // or NULL
  uint8_t* workspace;
  int chunks;
};
size_t chunk_attention_workspace(int n_q, int n_kv, int chunks);
cudaError_t launch_chunk_attention(const ChunkAttnArgs& a, const TileMaps& maps, cudaStream_t stream);

// Tensor map of a call's queries (chunk_attention.cu).
cudaError_t encode_query_map(CUtensorMap* m, bool bf16, const void* q, long long stride, int heads, int group,
                             int tokens, int queries);

struct MassArgs {
  PoolView pool;
  ChunkRows rows;
  const uint8_t* q;
  long long q_stride;
  int n_q;
  ScoreArgs sc;
  const float* lse;
  int last_queries;
  const float* mass_in;
  float* mass_out;
  int mass_stride;
  uint8_t* workspace;
  int chunks;
};
size_t attention_mass_workspace(int chunks);
cudaError_t launch_attention_mass(const MassArgs& a, const TileMaps& maps, cudaStream_t stream);

}  // namespace pkv
