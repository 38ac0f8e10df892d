// chunk_attention.cu — chunk attention whose queries see a range of tokens, and
// what it shares with sparse_attention.cu.
#include "chunk_attention.cuh"

namespace pkv {

size_t chunk_attention_workspace(int n_q, int n_kv, int chunks) {
  (void)n_q;
  (void)n_kv;
  return rec_bytes(chunks) + 2 * static_cast<size_t>(chunks) * kSlotFull;
}

cudaError_t launch_chunk_attention(const ChunkAttnArgs& a, const TileMaps& maps, cudaStream_t st) {
  CUtensorMap qmap;
  cudaError_t e = encode_query_map(&qmap, a.pool.dtype == PKV_KV_BF16, a.q, a.q_stride, a.n_q, a.n_q / a.pool.n_kv,
                                   a.rows.total_tokens, 128 / (a.n_q / a.pool.n_kv));
  if (e != cudaSuccess) return e;
  if (a.parents || a.pool.sinks > 0) return launch_sparse_attention(a, maps, qmap, st);
  return launch_attention<false>(a, maps, qmap, st);
}

// The queries as a 4-D tensor {64 dims, heads, tokens, 2 halves of the dims},
// box {64, G, queries, 2}: a copy lands [half][query, head][64 dims] under the
// 128-byte swizzle, the K-major layout of a product's first operand.  Tokens
// behind the last read as zeros.
cudaError_t encode_query_map(CUtensorMap* m, bool bf16, const void* q, long long stride, int heads, int group,
                             int tokens, int queries) {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult r = cudaDriverEntryPointSymbolNotFound;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &r) != cudaSuccess ||
        r != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  }();
  if (!fn) return cudaErrorNotSupported;
  const cuuint64_t dims[4] = {64u, static_cast<cuuint64_t>(heads), static_cast<cuuint64_t>(tokens), 2u};
  const cuuint64_t strides[3] = {kD * 2, static_cast<cuuint64_t>(stride) * 2, 128u};
  const cuuint32_t box[4] = {64u, static_cast<cuuint32_t>(group), static_cast<cuuint32_t>(queries), 2u};
  const cuuint32_t estride[4] = {1u, 1u, 1u, 1u};
  const CUresult r = fn(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4,
                        const_cast<void*>(q), dims, strides, box, estride, CU_TENSOR_MAP_INTERLEAVE_NONE,
                        CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

}  // namespace pkv
