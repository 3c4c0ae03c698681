// Rotary append at positions that are the cache indexes (kernel and launch
// rules: rotary_kernel.cuh).
#include "rotary_kernel.cuh"

namespace kvattn {

kvattn_status launch_rotary_append(const RotaryArgs& a, cudaStream_t s) { return dispatch<false>(a, s); }

}  // namespace kvattn
