// kvq_chunk_attention on tcgen05, head_dim 320.
#include "kvq_chunk_tc.cuh"

namespace kvq {

ChunkTiles chunk_tc_tiles_d320(int parts) { return tc_tiles<320>(parts); }
cudaError_t launch_chunk_tc_d320(ChunkArgs& a, int parts, cudaStream_t st) { return launch_tc<320>(a, parts, st); }

}  // namespace kvq
