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
// stored, ids being looked up once per chunk; or, where a run is at most half a chunk, several
// runs at a time.  A pair with an id outside the pool is skipped and recorded as
// KVATTN_ERR_BAD_INDEX.  (4000 blocks of 1 KV head of 64, bf16, 32 layers, 1.05 GB moved: 162 us,
// one run at a time 329; 500 blocks of 8 heads of 128: 337 us; 8192 fp8 blocks of 8 heads 84.)
#include <algorithm>

#include "kvattn_internal.cuh"

namespace kvattn {
namespace {

constexpr int kCopyThreads = 256;
constexpr int kVecs = 4;  // 16-byte vectors of a thread in a chunk
// Thread blocks per SM of a grid: with 4 and 8 the 8192 fp8 blocks took 84 and 91 us, the 500 blocks of 8 heads
// 337 and 341 (5: 86 and 335, but 9 heads of 64, in chunks of 576 vectors, 232 instead of 220).
constexpr int kBlocksPerSm = 4;

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

// Runs of at most half a chunk: unit u is `runs` of them, u runs .. , run x being region
// x % regions of pair x / regions, so that no thread goes without a vector.
__global__ void __launch_bounds__(kCopyThreads, kBlocksPerSm)
    copy_small_blocks_kernel(const __grid_constant__ CopyArgs a, const int runs, const int64_t total)
{
    pdl_wait();
    const int vecs = (int)(a.block_bytes / 16);
    for (int64_t first = (int64_t)blockIdx.x * runs; first < total; first += (int64_t)gridDim.x * runs) {
        const int64_t pair0 = first / a.regions;
        const int r0 = (int)(first - pair0 * a.regions), count = (int)min((int64_t)runs, total - first);
        uint4 v[kVecs];
        uint4* to[kVecs];
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
            const int x = i * kCopyThreads + (int)threadIdx.x, j = x / vecs;
            to[i] = nullptr;
            if (j >= count) continue;
            const unsigned rr = (unsigned)r0 + (unsigned)j, q = rr / (unsigned)a.regions, r = rr - q * (unsigned)a.regions;
            const int32_t s = a.src[pair0 + q], d = a.dst[pair0 + q];
            if (s < 0 || s >= a.num_blocks || d < 0 || d >= a.num_blocks) {
                if (x == j * vecs) record_error(a.status, KVATTN_ERR_BAD_INDEX);
                continue;
            }
            char* base = ((r & 1) ? a.v_base : a.k_base) + (int64_t)(r >> 1) * a.layer_stride;
            const int64_t off = (int64_t)(x - j * vecs) * 16;
            v[i] = *reinterpret_cast<const uint4*>(base + (int64_t)s * a.block_bytes + off);
            to[i] = reinterpret_cast<uint4*>(base + (int64_t)d * a.block_bytes + off);
        }
#pragma unroll
        for (int i = 0; i < kVecs; ++i)
            if (to[i]) *to[i] = v[i];
    }
}

}  // namespace

kvattn_status launch_copy_blocks(const CopyArgs& a, cudaStream_t s)
{
    if (a.block_bytes / 16 > INT32_MAX / 2) return KVATTN_ERR_UNSUPPORTED;
    const int vecs = (int)(a.block_bytes / 16), most = kCopyThreads * kVecs;
    const int64_t wave = (int64_t)num_sms() * kBlocksPerSm, total = (int64_t)a.n * a.regions;
    if (vecs <= most / 2) {
        const int runs = (int)std::max<int64_t>(1, std::min<int64_t>(most / vecs, (total + wave - 1) / wave));
        const int grid = (int)std::min<int64_t>((total + runs - 1) / runs, wave);
        return cuda_status(launch_pdl(copy_small_blocks_kernel, dim3(grid), dim3(kCopyThreads), 0, s, a, runs, total));
    }
    const int chunks = (vecs + most - 1) / most, chunk_vecs = (vecs + chunks - 1) / chunks;
    const int64_t units = total * chunks;
    const int grid = (int)std::min<int64_t>(units, wave);
    return cuda_status(launch_pdl(copy_blocks_kernel, dim3(grid), dim3(kCopyThreads), 0, s, a, chunks, chunk_vecs, units));
}

}  // namespace kvattn
