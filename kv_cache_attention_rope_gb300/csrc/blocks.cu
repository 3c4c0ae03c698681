// Copies of whole cache blocks (copy on write of shared ones).
//
// "Nano-vLLM Part 2" page, section 05: the block manager keeps reference
// counts so that sequences with a common prefix share its blocks, and one
// block id names the same block in every layer's K and V area.  When a
// sequence appends into a partially filled block that another sequence still
// references, the block is first duplicated under a fresh id; this kernel
// makes those duplicates, for every K and V region (an fp8 cache: its one
// region of pages) at once.
//
// Bound by HBM: each block-region is one contiguous run (of Hkv x block_size x D
// elements, or Hkv x block_size / 16 pages), read once and written once.  A
// thread block copies chunks of a run, a chunk's vectors all under way before the first is
// stored; ids are looked up once per chunk.  A pair with an id outside the pool
// is skipped and recorded as KVATTN_ERR_BAD_INDEX.
#include <algorithm>

#include "kvattn_internal.cuh"

namespace kvattn {
namespace {

constexpr int kCopyThreads = 256;
constexpr int kVecs = 4;  // 16-byte vectors of a thread in a chunk

// Unit u: chunk u % chunks of region (u / chunks) % regions of pair u / (chunks regions).
__global__ void __launch_bounds__(kCopyThreads) copy_blocks_kernel(const __grid_constant__ CopyArgs a, const int chunks,
                                                                   const int chunk_vecs, const int64_t units)
{
    pdl_wait();
    const int vecs = (int)(a.block_bytes / 16);
    for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
        const int64_t pr = u / chunks;
        const int c = (int)(u - pr * chunks), pair = (int)(pr / a.regions), r = (int)(pr - (int64_t)pair * a.regions);
        const int32_t s = a.src[pair], d = a.dst[pair];
        if (s < 0 || s >= a.num_blocks || d < 0 || d >= a.num_blocks) {
            if (threadIdx.x == 0) record_error(a.status, KVATTN_ERR_BAD_INDEX);
            continue;
        }
        char* base = ((r & 1) ? a.v_base : a.k_base) + (r >> 1) * a.layer_stride;
        const uint4* from = reinterpret_cast<const uint4*>(base + (int64_t)s * a.block_bytes);
        uint4* to = reinterpret_cast<uint4*>(base + (int64_t)d * a.block_bytes);
        const int end = min(vecs, (c + 1) * chunk_vecs);
        uint4 v[kVecs];
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
            const int x = c * chunk_vecs + i * kCopyThreads + (int)threadIdx.x;
            if (x < end) v[i] = from[x];
        }
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
            const int x = c * chunk_vecs + i * kCopyThreads + (int)threadIdx.x;
            if (x < end) to[x] = v[i];
        }
    }
}

}  // namespace

kvattn_status launch_copy_blocks(const CopyArgs& a, cudaStream_t s)
{
    if (a.block_bytes / 16 > INT32_MAX / 2) return KVATTN_ERR_UNSUPPORTED;
    const int vecs = (int)(a.block_bytes / 16), most = kCopyThreads * kVecs;
    const int chunks = (vecs + most - 1) / most, chunk_vecs = (vecs + chunks - 1) / chunks;
    const int64_t units = (int64_t)a.n * a.regions * chunks;
    const int grid = (int)std::min<int64_t>(units, (int64_t)num_sms() * 8);
    return cuda_status(launch_pdl(copy_blocks_kernel, dim3(grid), dim3(kCopyThreads), 0, s, a, chunks, chunk_vecs, units));
}

}  // namespace kvattn
