// kvq_chunk_attention on tcgen05, head_dim 64.
#include "kvq_chunk_tc.cuh"

namespace kvq {

ChunkTiles chunk_tc_tiles_d64(int parts) { return tc_tiles<64>(parts); }
cudaError_t launch_chunk_tc_d64(ChunkArgs& a, int parts, cudaStream_t st) { return launch_tc<64>(a, parts, st); }

}  // namespace kvq
