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
// written once, in place and without a workspace.  A cluster of thread blocks walks one
// sequence's list for some (region, head) slices, a round of tokens at a
// time: all of a round's rows are loaded into registers, a barrier, all are
// stored.  That is a compaction in place: a round writes the places [j0, j1),
// and every row that a later round reads lies at keep[j] >= j >= j1.  The barrier's
// wait is covered by the other clusters of the SM, so a long list is spread
// over as many blocks as fill the GPU.
#include <algorithm>
#include <climits>

#include "kvattn_internal.cuh"

namespace kvattn {
namespace {

constexpr int kThreads = 256, kWide = 512;     // of a block, where many and where few lists are moved
constexpr int kVecs = 4;                       // 16-byte vectors that a thread holds
constexpr int kMaxRound = kWide * kVecs / 8;   // tokens of a block's round: rows are 8 vectors at least
constexpr int kMaxCluster = 8;
// Blocks per SM that a grid may have by clusters.  Evicting half of 16 bf16 lists of up to 32768
// tokens took 354 us with 6, 269 with 8, 232 with 16 and more; a quarter of 32 fp8 lists of up to
// 8192 (as above) 243, 158 (12) and 144.
constexpr int kFill = 16;

// Every load of the cluster's threads so far has its value, before any of them goes on.
__device__ __forceinline__ void cluster_sync(int cluster)
{
    if (cluster == 1)
        __syncthreads();
    else
        asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

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

// Cluster (s, part): slices part * slices ... of the 2 layers Hkv (region, head)
// ones, region 2 layer + (0: K, 1: V), head fastest.  Rows of 2^row_log2 vectors.
__global__ void __launch_bounds__(kWide, 3)
    compact_rows_kernel(const __grid_constant__ CompactArgs a, const int cluster, const int slices, const int parts,
                        const int row_log2)
{
    pdl_wait();
    const int unit = blockIdx.x / cluster, rank = blockIdx.x - unit * cluster;
    const int s = unit / parts, first = (unit - s * parts) * slices;
    const int ns = min(slices, 2 * a.layers * a.hkv - first);
    const List l = list_of(a, s);
    if (l.n == 0) return;
    const int round = ((int)blockDim.x * kVecs >> row_log2) / slices;  // tokens of a block
    // tokens: first vector of a row of head 0, source (-1: stays) and place; of this
    // round, the next, and the one before, whose stores may be under way
    __shared__ int64_t rows[3][2][kMaxRound];
    const int64_t head_vecs = (int64_t)a.block_size << row_log2;
    int token[kVecs];  // of this thread's vectors: token of the round, INT_MAX past its slices
    uint4* base[kVecs];
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
        const int x = i * (int)blockDim.x + threadIdx.x, row = x >> row_log2, sl = row / round;
        const int r = (first + sl) / a.hkv, h = first + sl - r * a.hkv;
        token[i] = sl < ns ? row - sl * round : INT_MAX;
        base[i] = reinterpret_cast<uint4*>(((r & 1) ? a.v_base : a.k_base) + (r >> 1) * a.layer_stride) + h * head_vecs +
                  (x & ((1 << row_log2) - 1));
    }
    auto place = [&](unsigned j0, int buf) {
        if ((int)threadIdx.x < min(round, (int)((unsigned)l.n - j0))) {
            const int j = (int)j0 + threadIdx.x, to = l.start + j, from = kept(a, l, j);
            int64_t src = -1, dst = -1;
            if (from >= 0 && from != to) {
                const int bs = block_of(a, s, from), bd = block_of(a, s, to);
                if (bs >= 0 && bd >= 0) {
                    src = ((int64_t)bs * a.hkv * a.block_size + from % a.block_size) << row_log2;
                    dst = ((int64_t)bd * a.hkv * a.block_size + to % a.block_size) << row_log2;
                }
            }
            rows[buf][0][threadIdx.x] = src;
            rows[buf][1][threadIdx.x] = dst;
        }
    };
    const unsigned step = round * cluster;
    place(rank * round, 0);
    __syncthreads();
    int buf = 0;
    for (unsigned j0 = 0; j0 < (unsigned)l.n; j0 += step) {
        const int cnt = min(round, (int)((unsigned)l.n - j0 - rank * round));
        const int next = buf == 2 ? 0 : buf + 1;
        uint4 v[kVecs];
        bool moves[kVecs];
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
            const int64_t src = token[i] < cnt ? rows[buf][0][token[i]] : -1;
            moves[i] = src >= 0;
            if (moves[i]) v[i] = base[i][src];
        }
        place(j0 + step + rank * round, next);
        cluster_sync(cluster);
#pragma unroll
        for (int i = 0; i < kVecs; ++i)
            if (moves[i]) base[i][rows[buf][1][token[i]]] = v[i];
        buf = next;
    }
}

// An fp8 cache.  A warp makes one destination page (16 tokens of a head): K rows
// as vectors.  V stands transposed, 4 tokens of a dim in a 32-bit word; those that four
// kept tokens come from are at most four, mostly two: a word of the destination is one
// byte permutation of two words, or the merge of two.  Tokens of the page
// that no kept one is moved to stay as they are.  Cluster (s, head); a round is a page
// for each warp, all loaded before any is stored.  (Words are read several times, from L1:
// no page is read after its own round's stores.  Copying one byte at a time took 263 us, picking
// bytes out of whole 16-byte rows 144, this 108, for a quarter evicted of 32 lists of up to 8192 tokens.)
constexpr int kPageWarps = 4, kPageWide = 8;
__global__ void __launch_bounds__(kPageWide * 32, 4)
    compact_pages_kernel(const __grid_constant__ CompactArgs a, const int cluster)
{
    pdl_wait();
    const int unit = blockIdx.x / cluster, rank = blockIdx.x - unit * cluster;
    const int s = unit / a.hkv, h = unit - s * a.hkv;
    const List l = list_of(a, s);
    if (l.n == 0) return;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int bpages = a.block_size / 16;
    unsigned char* pool = reinterpret_cast<unsigned char*>(a.k_base);
    auto page_of = [&](int blk, int pos) { return (blk * a.hkv + h) * bpages + pos % a.block_size / 16; };
    const int last = (int)(((int64_t)l.start + l.n - 1) / 16);
    // page p is page `dst` of the pool; lane e (and e + 16): its token e comes from page
    // `src` and is token `from` there.  (Pages of 4224 bytes are counted in 32 bits.)
    struct Page {
        unsigned dst, src;
        int from;
        bool moved;
    };
    auto plan = [&](int p) {
        Page g{0, 0, lane & 15, false};
        if (p <= last) {
            const int bd = block_of(a, s, p * 16);
            const int64_t j = (int64_t)p * 16 + (lane & 15) - l.start;
            const int k = j >= 0 && j < l.n ? kept(a, l, (int)j) : -1;
            if (bd >= 0) {
                g.src = g.dst = page_of(bd, p * 16);
                if (k >= 0 && k != l.start + j) {
                    const int bs = block_of(a, s, k);
                    if (bs >= 0) {
                        g.src = page_of(bs, k);
                        g.from = k & 15;
                        g.moved = true;
                    }
                }
            }
        }
        return g;
    };
    const int warps = blockDim.x >> 5, step = warps * cluster, at = rank * warps + warp;
    Page next = plan(l.start / 16 + at);
    for (int p0 = l.start / 16; p0 <= last; p0 += step) {
        const Page g = next;
        const unsigned which = __ballot_sync(0xffffffffu, g.moved);
        uint4 kv[4];
        uint32_t vw[4][4];  // dims lane + 32 i, tokens 4 w .. 4 w + 3
        float scale = 0.f;
        if (which) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int e = (lane >> 3) + 4 * i, c = lane & 7;
                const unsigned sp = __shfl_sync(0xffffffffu, g.src, e);
                const int fr = __shfl_sync(0xffffffffu, g.from, e);
                if (which >> e & 1u)
                    kv[i] = *reinterpret_cast<const uint4*>(pool + (int64_t)sp * kF8Page + fr * 128 + ((c ^ f8_swz(fr)) << 4));
            }
            scale = *reinterpret_cast<const float*>(pool + (int64_t)g.src * kF8Page + (lane < 16 ? kF8KsOff : kF8VsOff) +
                                                    4 * g.from);
            // the word that token e is in, how many others the tokens before it in its
            // word of the destination are in, and the byte of the pair (word, other)
            const unsigned word = g.src * 4 + (g.from >> 2), quad = lane & ~3u, below = (1u << (lane & 3)) - 1u;
            const unsigned same = __match_any_sync(0xffffffffu, word) >> quad;
            const unsigned firsts = __ballot_sync(0xffffffffu, (same & below) == 0) >> quad & 0xfu;
            const int nth = __popc(firsts & (2u * (1u << (__ffs(same) - 1)) - 1u)) - 1;
            unsigned sel = (unsigned)((nth & 1) * 4 + (g.from & 3)) << (4 * (lane & 3));
            sel |= __shfl_xor_sync(0xffffffffu, sel, 1);
            sel |= __shfl_xor_sync(0xffffffffu, sel, 2);
            auto word_at = [&](int e) {  // token e's, of this lane's dims
                const unsigned x = __shfl_sync(0xffffffffu, word, e);
                return pool + (int64_t)(x >> 2) * kF8Page + kF8VOff + (x & 3) * 4 + 16 * lane;
            };
            const unsigned second = firsts & (firsts - 1), third = second & (second - 1), fourth = third & (third - 1);
            const int b1 = quad + (second ? __ffs(second) - 1 : 0), b2 = quad + (third ? __ffs(third) - 1 : 0),
                      b3 = quad + (fourth ? __ffs(fourth) - 1 : 0);
            uint32_t x[4][2][4];
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                const unsigned char* p0w = word_at(4 * w);
                const unsigned char* p1w = word_at(__shfl_sync(0xffffffffu, b1, 4 * w));
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    x[w][0][i] = *reinterpret_cast<const uint32_t*>(p0w + 512 * i);
                    x[w][1][i] = *reinterpret_cast<const uint32_t*>(p1w + 512 * i);
                }
            }
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                const unsigned z = __shfl_sync(0xffffffffu, sel, 4 * w);
#pragma unroll
                for (int i = 0; i < 4; ++i) vw[i][w] = __byte_perm(x[w][0][i], x[w][1][i], z);
            }
            const unsigned more = __ballot_sync(0xffffffffu, nth >= 2);
            if (more) {
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    const unsigned char* p2w = word_at(__shfl_sync(0xffffffffu, b2, 4 * w));
                    const unsigned char* p3w = word_at(__shfl_sync(0xffffffffu, b3, 4 * w));
                    const unsigned z = __shfl_sync(0xffffffffu, sel, 4 * w), m = more >> 4 * w & 0xfu;
                    if (m == 0) continue;
                    // bytes of `m` from the third and fourth word
                    const unsigned keep = __byte_perm(0u, 0xffffffffu, (m & 1u) * 4 | (m & 2u) << 5 | (m & 4u) << 8 | (m & 8u) << 11);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint32_t y = __byte_perm(*reinterpret_cast<const uint32_t*>(p2w + 512 * i),
                                                       *reinterpret_cast<const uint32_t*>(p3w + 512 * i), z);
                        vw[i][w] = (y & keep) | (vw[i][w] & ~keep);
                    }
                }
            }
        }
        next = plan(p0 + step + at);
        cluster_sync(cluster);
        if (which) {
            unsigned char* pg = pool + (int64_t)g.dst * kF8Page;
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

// Blocks of a unit's cluster: more of them while the grid is not above kFill blocks per
// SM and each has work for a round.
int cluster_of(int64_t units, int64_t rounds)
{
    int c = 1;
    while (c < kMaxCluster && units * c * 2 <= (int64_t)kFill * num_sms() && 2 * c <= rounds) c *= 2;
    return c;
}

// Whether blocks of twice the threads are wanted besides: one list of 16384 tokens and
// 8 heads 50.7 -> 35.1 us, 16 such lists 232 -> 239.  (fp8 pages, when V was still picked out of whole
// rows: 94.9 -> 56.3, and 32 lists of 6144 tokens 144 -> 156.)
bool wide(int64_t units, int cluster, int64_t rounds)
{
    return cluster == kMaxCluster && units * cluster * 4 <= (int64_t)kFill * num_sms() && 2 * cluster <= rounds;
}

template <typename... KArgs, typename... Args>
kvattn_status run(void (*kern)(KArgs...), int64_t units, int threads, int cluster, cudaStream_t s, Args... args)
{
    if (units * cluster > INT32_MAX) return KVATTN_ERR_UNSUPPORTED;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(units * cluster));
    cfg.blockDim = dim3(threads);
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cuda_status(cudaLaunchKernelEx(&cfg, kern, args...));
}

}  // namespace

// Laid out for the mean list, which is all that the host knows: a long one among many short ones
// gets as few blocks as these (half of 16384 tokens, 8 heads of 128, bf16: 30 us alone, 209
// beside 127 empty lists).
kvattn_status launch_compact(const CompactArgs& a, cudaStream_t s)
{
    const int64_t mean = std::max<int64_t>(1, a.total_keep / a.num_seqs);
    if (a.fp8) {
        const int64_t units = (int64_t)a.num_seqs * a.hkv, rounds = mean / (16 * kPageWarps);
        const int cluster = cluster_of(units, rounds), warps = wide(units, cluster, rounds) ? kPageWide : kPageWarps;
        return run(compact_pages_kernel, units, warps * 32, cluster, s, a, cluster);
    }
    int row_log2 = 0;
    while ((16 << row_log2) < a.row_bytes) ++row_log2;
    // slices of a block: as many as fill a round with the tokens of an average list
    const int64_t rows = kThreads * kVecs >> row_log2, all = 2 * (int64_t)a.layers * a.hkv;
    const int slices = (int)std::max<int64_t>(1, std::min(all, rows / mean));
    const int64_t parts = (all + slices - 1) / slices, units = a.num_seqs * parts;
    const int64_t rounds = mean / (rows / slices);
    const int cluster = cluster_of(units, rounds), threads = wide(units, cluster, rounds) ? kWide : kThreads;
    if (parts > INT32_MAX) return KVATTN_ERR_UNSUPPORTED;
    return run(compact_rows_kernel, units, threads, cluster, s, a, cluster, slices, (int)parts, row_log2);
}

}  // namespace kvattn
