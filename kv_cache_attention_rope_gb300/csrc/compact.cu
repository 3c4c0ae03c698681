// Token compaction: a sequence's kept tokens move together in its cache.
//
// What it computes: token starts[s] + j of sequence s becomes a bit copy of its
// token keep[cu[s] + j] (K, V and an fp8 cache's scales), in every head and
// layer; the kept positions ascend, so keep[cu[s] + j] >= starts[s] + j.
// "Nano-vLLM Part 2" page, section 05 (tokens live in the slots that the block
// table names): a block is the unit of allocation, a slot that of a token, and
// tokens that leave in the middle (rejected drafts, evicted ones) leave holes
// that no block's release fills.
//
// How: bound by HBM, 2 rows of K and V per moved token and head, read once and
// written once, in place and without a workspace.  A thread block walks one
// sequence's list for some heads of one K or V region, a round of tokens at a
// time: all of a round's rows are loaded into registers, a barrier, all are
// stored.  That is a compaction in place: a round writes the places [j0, j1),
// and every row that a later round reads lies at keep[j] >= j >= j1.
#include <algorithm>
#include <climits>

#include "kvattn_internal.cuh"

namespace kvattn {
namespace {

constexpr int kThreads = 256;
constexpr int kVecs = 4;                       // 16-byte vectors that a thread holds
constexpr int kMaxRound = kThreads * kVecs / 8;  // tokens of a round: rows are 8 vectors at least

// The list of sequence s; one out of range counts as empty (recorded).
struct List {
    int first, n, start;
};
__device__ __forceinline__ List list_of(const CompactArgs& a, int s)
{
    List l{a.cu[s], 0, a.starts[s]};
    const int end = a.cu[s + 1];
    const int64_t room = min((int64_t)a.max_blocks * a.block_size, (int64_t)INT32_MAX);
    if (l.first < 0 || end < l.first || end > a.total_keep || l.start < 0 || (int64_t)l.start + (end - l.first) > room) {
        record_error(a.status, KVATTN_ERR_BAD_INDEX);
        return l;
    }
    l.n = end - l.first;
    return l;
}

// The block of sequence s that holds position pos, -1 (recorded) if the table or
// the pool has none.
__device__ __forceinline__ int block_of(const CompactArgs& a, int s, int pos)
{
    const int col = pos / a.block_size;
    const int b = col < a.max_blocks ? a.block_table[(int64_t)s * a.max_blocks + col] : -1;
    if (b >= 0 && b < a.num_blocks) return b;
    record_error(a.status, KVATTN_ERR_BAD_INDEX);
    return -1;
}

// Kept position j of the list, -1 (recorded) where the list does not ascend.
__device__ __forceinline__ int kept(const CompactArgs& a, const List& l, int j)
{
    const int p = a.keep[l.first + j];
    if ((int64_t)p >= (int64_t)l.start + j && (j == 0 || a.keep[l.first + j - 1] < p)) return p;
    record_error(a.status, KVATTN_ERR_BAD_INDEX);
    return -1;
}

// Block (s, region, part): region r = 2 layer + (0: K, 1: V), part p the heads
// p * heads ...  Rows of 2^row_log2 vectors.
__global__ void __launch_bounds__(kThreads) compact_rows_kernel(const __grid_constant__ CompactArgs a, const int heads,
                                                                const int parts, const int row_log2)
{
    pdl_wait();
    const int regions = 2 * a.layers;
    const int s = blockIdx.x / (regions * parts), rest = blockIdx.x - s * regions * parts;
    const int r = rest / parts, h0 = (rest - r * parts) * heads;
    const int nh = min(heads, a.hkv - h0);
    const List l = list_of(a, s);
    const int round = (kThreads * kVecs >> row_log2) / heads;  // tokens
    uint4* pool = reinterpret_cast<uint4*>(((r & 1) ? a.v_base : a.k_base) + (r >> 1) * a.layer_stride);
    __shared__ int64_t rows[2][kMaxRound];  // first vector of a token's row of head h0: source (-1: stays), place
    const int64_t head_vecs = (int64_t)a.block_size << row_log2;
    int token[kVecs];  // of this thread's vectors: token of the round, -1 past its heads
    int64_t off[kVecs];
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
        const int x = i * kThreads + threadIdx.x, row = x >> row_log2;
        const int h = row / round;
        token[i] = h < nh ? row - h * round : INT_MAX;
        off[i] = h * head_vecs + (x & ((1 << row_log2) - 1));
    }
    for (int j0 = 0; j0 < l.n; j0 += round) {
        const int cnt = min(round, l.n - j0);
        __syncthreads();  // the round before has read `rows`
        if ((int)threadIdx.x < cnt) {
            const int j = j0 + threadIdx.x, to = l.start + j, from = kept(a, l, j);
            int64_t src = -1, dst = -1;
            if (from >= 0 && from != to) {
                const int bs = block_of(a, s, from), bd = block_of(a, s, to);
                if (bs >= 0 && bd >= 0) {
                    src = (((int64_t)bs * a.hkv + h0) * a.block_size + from % a.block_size) << row_log2;
                    dst = (((int64_t)bd * a.hkv + h0) * a.block_size + to % a.block_size) << row_log2;
                }
            }
            rows[0][threadIdx.x] = src;
            rows[1][threadIdx.x] = dst;
        }
        __syncthreads();
        uint4 v[kVecs];
        bool moves[kVecs];
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
            moves[i] = token[i] < cnt && rows[0][token[i]] >= 0;
            if (moves[i]) v[i] = pool[rows[0][token[i]] + off[i]];
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kVecs; ++i)
            if (moves[i]) pool[rows[1][token[i]] + off[i]] = v[i];
    }
}

// An fp8 cache.  A warp makes one destination page (16 tokens of a head): K rows
// as vectors, and since V stands transposed, its bytes one at a time, 16 of a
// dim for a lane, from whichever pages hold them.  Tokens of the page that no
// kept one is moved to stay as they are.  Block (s, head); a round is a page for
// each warp, all loaded before any is stored.
constexpr int kPageWarps = 4;
__global__ void __launch_bounds__(kPageWarps * 32) compact_pages_kernel(const __grid_constant__ CompactArgs a)
{
    pdl_wait();
    const int s = blockIdx.x / a.hkv, h = blockIdx.x - s * a.hkv;
    const List l = list_of(a, s);
    if (l.n == 0) return;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int bpages = a.block_size / 16;
    unsigned char* pool = reinterpret_cast<unsigned char*>(a.k_base);
    auto page_of = [&](int blk, int pos) {
        return (((int64_t)blk * a.hkv + h) * bpages + pos % a.block_size / 16) * kF8Page;
    };
    const int last = (int)(((int64_t)l.start + l.n - 1) / 16);
    for (int p0 = l.start / 16; p0 <= last; p0 += kPageWarps) {
        const int p = p0 + warp;
        // lane e < 16: token e of the page comes from byte offset `src` of the pool
        // (a page) and its token `from`
        int64_t dst = -1, src = -1;
        int from = lane & 15;
        bool moved = false;
        if (p <= last) {
            const int bd = block_of(a, s, p * 16);
            if (bd >= 0) {
                src = dst = page_of(bd, p * 16);
                const int64_t j = (int64_t)p * 16 + (lane & 15) - l.start;
                if (j >= 0 && j < l.n) {
                    const int k = kept(a, l, (int)j);
                    if (k >= 0 && k != l.start + j) {
                        const int bs = block_of(a, s, k);
                        if (bs >= 0) {
                            src = page_of(bs, k);
                            from = k & 15;
                            moved = true;
                        }
                    }
                }
            }
        }
        const bool work = __any_sync(0xffffffffu, moved);
        const unsigned which = __ballot_sync(0xffffffffu, moved);
        uint4 kv[4];
        uint32_t vw[4][4];  // dims lane + 32 i, tokens 4 w .. 4 w + 3
        float scale = 0.f;
        if (work) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int e = (lane >> 3) + 4 * i, c = lane & 7;
                const int64_t sp = __shfl_sync(0xffffffffu, src, e);
                const int fr = __shfl_sync(0xffffffffu, from, e);
                kv[i] = *reinterpret_cast<const uint4*>(pool + sp + fr * 128 + ((c ^ f8_swz(fr)) << 4));
            }
            scale = *reinterpret_cast<const float*>(pool + src + (lane < 16 ? kF8KsOff : kF8VsOff) + 4 * from);
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int w = 0; w < 4; ++w) vw[i][w] = 0;
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                const int64_t sp = __shfl_sync(0xffffffffu, src, e);
                const int fr = __shfl_sync(0xffffffffu, from, e);
                const unsigned char* v = pool + sp + kF8VOff + 16 * lane + fr;
#pragma unroll
                for (int i = 0; i < 4; ++i) vw[i][e >> 2] |= (uint32_t)v[512 * i] << (8 * (e & 3));
            }
        }
        __syncthreads();
        if (work) {
            unsigned char* pg = pool + dst;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int e = (lane >> 3) + 4 * i, c = lane & 7;
                if (which >> e & 1u) *reinterpret_cast<uint4*>(pg + e * 128 + ((c ^ f8_swz(e)) << 4)) = kv[i];
                *reinterpret_cast<uint4*>(pg + kF8VOff + 16 * (lane + 32 * i)) =
                    make_uint4(vw[i][0], vw[i][1], vw[i][2], vw[i][3]);
            }
            *reinterpret_cast<float*>(pg + (lane < 16 ? kF8KsOff : kF8VsOff) + 4 * (lane & 15)) = scale;
        }
    }
}

}  // namespace

kvattn_status launch_compact(const CompactArgs& a, cudaStream_t s)
{
    if (a.fp8) {
        const int64_t grid = (int64_t)a.num_seqs * a.hkv;
        if (grid > INT32_MAX) return KVATTN_ERR_UNSUPPORTED;
        return cuda_status(launch_pdl(compact_pages_kernel, dim3((unsigned)grid), dim3(kPageWarps * 32), 0, s, a));
    }
    int row_log2 = 0;
    while ((16 << row_log2) < a.row_bytes) ++row_log2;
    // heads of a block: as many as fill a round with the tokens of an average list
    const int64_t mean = std::max<int64_t>(1, a.total_keep / a.num_seqs);
    int heads = 1;
    while (heads * 2 <= a.hkv && (heads * 2 * mean << row_log2) <= kThreads * kVecs) heads *= 2;
    const int parts = (a.hkv + heads - 1) / heads;
    const int64_t grid = (int64_t)a.num_seqs * 2 * a.layers * parts;
    if (grid > INT32_MAX) return KVATTN_ERR_UNSUPPORTED;
    return cuda_status(launch_pdl(compact_rows_kernel, dim3((unsigned)grid), dim3(kThreads), 0, s, a, heads, parts, row_log2));
}

}  // namespace kvattn
