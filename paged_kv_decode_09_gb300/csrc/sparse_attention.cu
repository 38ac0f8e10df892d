// sparse_attention.cu — chunk attention on layers with sinks, and of trees.
#include "chunk_attention.cuh"

namespace pkv {

cudaError_t launch_sparse_attention(const ChunkAttnArgs& a, const TileMaps& maps, const CUtensorMap& qmap,
                                    cudaStream_t st) {
  return launch_attention<true>(a, maps, qmap, st);
}

}  // namespace pkv
