// kvq_chunk_attention on tcgen05, head_dim 128.
#include "kvq_chunk_tc.cuh"

namespace kvq {

ChunkTiles chunk_tc_tiles_d128(int parts) { return tc_tiles<128>(parts); }
cudaError_t launch_chunk_tc_d128(ChunkArgs& a, int parts, cudaStream_t st) { return launch_tc<128>(a, parts, st); }

}  // namespace kvq
