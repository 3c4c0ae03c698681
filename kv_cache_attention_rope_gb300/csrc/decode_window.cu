// Windowed decode attention: one query per sequence over the last `window`
// tokens of its cache and the first `sinks` ones, with the split-KV kernels of
// decode_kernel.cuh over the tiles that hold them.
#include "decode_kernel.cuh"

namespace kvattn {

kvattn_status launch_decode_window(const DecodeArgs& a, cudaStream_t s) { return dispatch<true>(a, s); }

}  // namespace kvattn
