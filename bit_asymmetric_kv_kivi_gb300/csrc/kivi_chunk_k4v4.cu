// Chunk attention for 4-bit keys and 4-bit values: the instantiations of kivi_chunk_impl.cuh
// for this pair of code widths.
#include "kivi_chunk_impl.cuh"

namespace kivi {

cudaError_t launch_chunk_k4v4(const ChunkArgs& a, cudaStream_t stream) { return launch_chunk_kv<4, 4>(a, stream); }

}  // namespace kivi
