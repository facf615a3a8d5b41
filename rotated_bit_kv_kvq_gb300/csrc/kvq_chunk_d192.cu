// kvq_chunk_attention on tcgen05, head_dim 192.
#include "kvq_chunk_tc.cuh"

namespace kvq {

ChunkTiles chunk_tc_tiles_d192(int parts) { return tc_tiles<192>(parts); }
cudaError_t launch_chunk_tc_d192(ChunkArgs& a, int parts, cudaStream_t st) { return launch_tc<192>(a, parts, st); }

}  // namespace kvq
