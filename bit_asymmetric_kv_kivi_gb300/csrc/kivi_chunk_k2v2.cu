// Chunk attention for 2-bit keys and 2-bit values: the instantiations of kivi_chunk_impl.cuh
// for this pair of code widths.
#include "kivi_chunk_impl.cuh"

namespace kivi {

cudaError_t launch_chunk_k2v2(const ChunkArgs& a, cudaStream_t stream) { return launch_chunk_kv<2, 2>(a, stream); }

}  // namespace kivi
