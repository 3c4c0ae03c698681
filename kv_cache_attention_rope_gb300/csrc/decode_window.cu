// Windowed decode attention: one query per sequence over the last `window`
// tokens of its cache and the first `sinks` ones.  Calls of few keys, and those
// over fp8 pages whose window is not very long, take one launch
// (decode_direct.cu); the others, and those with a given number of splits, the
// split-KV kernels of decode_kernel.cuh over the tiles that hold seen keys.
#include "decode_kernel.cuh"

namespace kvattn {

kvattn_status launch_decode_window(const DecodeArgs& a, int32_t max_tiles, cudaStream_t s)
{
    kvattn_status st;
    if (max_tiles > 0 && launch_decode_direct(a, max_tiles, s, &st)) return st;
    return dispatch<true>(a, s);
}

}  // namespace kvattn
