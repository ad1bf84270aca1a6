// Extended decode kernels (a window with sinks, weights per group, any query group) for
// 4-bit keys and 4-bit values: the instantiations of kivi_decode_impl.cuh for this pair of code widths.
#include "kivi_decode_impl.cuh"

namespace kivi {

cudaError_t launch_ext_k4v4(const DecodeArgs& a, cudaStream_t stream) { return launch_ext_kv<4, 4>(a, stream); }

}  // namespace kivi
