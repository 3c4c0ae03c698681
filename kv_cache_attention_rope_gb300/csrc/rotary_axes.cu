// Rotary append with several axes of positions and slots of their own (kernel
// and launch rules: rotary_kernel.cuh).
#include "rotary_kernel.cuh"

namespace kvattn {

kvattn_status launch_rotary_append_axes(const RotaryArgs& a, cudaStream_t s) { return dispatch<true>(a, s); }

}  // namespace kvattn
