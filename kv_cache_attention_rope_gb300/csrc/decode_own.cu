// The part of a shared-prefix decode that is each sequence's own: the split-KV
// kernels of decode_kernel.cuh over the keys behind the prefix, and the merge with the
// prefix's partial results (decode_shared.cu).
#include "decode_kernel.cuh"

namespace kvattn {

kvattn_status launch_decode_own(const DecodeArgs& a, cudaStream_t s) { return dispatch<kOwn>(a, s); }

}  // namespace kvattn
