// kvq_chunk_attention on tcgen05, head_dim 256.
#include "kvq_chunk_tc.cuh"

namespace kvq {

ChunkTiles chunk_tc_tiles_d256(int parts) { return tc_tiles<256>(parts); }
cudaError_t launch_chunk_tc_d256(ChunkArgs& a, int parts, cudaStream_t st) { return launch_tc<256>(a, parts, st); }

}  // namespace kvq
