// Decode attention for a batch in which groups of sequences share their first
// tokens: a prefix is read once for every 256 queries of its group.
//
// What it computes: kvattn_decode's out[b][j], an online softmax over every key of
// sequence b ("From-scratch AI inference engine" page, section 3.3: a query sees
// all cached keys), as the merge of partial states
//     m = max_i s_i,  l = sum_i 2^(s_i - m),  O = sum_i 2^(s_i - m) V[i],
//     s_i = q[b][j] . K[i][j / G] * scale * log2(e)
// over pieces of the prefix that b's group shares and of its own keys behind it
// (section 3.4 of the same page: states over parts of the keys merge by their
// maxima and sums; "Nano-vLLM Part 2" page, section 05: sequences with a common
// prefix share its blocks).  Only whole 16-token pages of a prefix are shared, and a
// sequence that is shorter takes no part, so no row has a mask of its own.  A page whose block
// is not in the pool is seen by nobody: its scores are -infinity, its V is zero.
//
// What bounds it.  A KV head's queries over a prefix are (sequences of the group) x
// G rows of one matrix product, so the prefix's K and V are read once for up to 256 of
// them, 4 D e bytes a key and KV head, for 4 D FLOPs a key and row: up to about 128 rows HBM
// has the longer part, from 256 rows on the tensor cores and the softmax beside them.  (More
// rows are more segments, each with its own pass over the pages, from L2 at best: one document
// and 512 rows are loaded, and in fp8 converted, twice.)  Own keys have G rows and are HBM's.
//
// How.  One launch, a CTA per SM, some of them on prefixes and the others on own
// keys, as many of each as make both end together; decode_shared_merge_kernel then
// merges a row's pieces.
//
// Prefixes (prefix_cta): rows come in blocks of 256 / G sequences.  The pages of all
// (row block, KV head) segments form one stream, cut into equal ranges, one per CTA,
// segments being cut where ranges meet.  A piece is worked on in tiles of up to 8
// pages on the tcgen05 tensor cores.  One of more than 128 rows has two row tiles by
// turns over the same K and V tiles; any other has one.  Either way the steps (S, softmax,
// P.V) alternate between two S buffers, so that the softmax of one runs beside the products
// of the other; a piece of one row tile has one of the two O buffers, the next
// piece the other.  Roles (four warpgroups): warp 0 copies K and Q tiles, warp 2 V
// tiles (a page a lane, straight from the block table); warp 1 issues the MMAs, P.V
// of a step and then S of the second one after it, from piece to piece without a gap;
// warps 4-11 the softmax (columns 0-63 and 64-127), P overwriting the first half
// of S in TMEM; warps 12-15 the outputs.  TMEM: S_0, S_1, O_0, O_1, 128 columns each.
//
// Own keys (own_warp): the pages of all (sequence, KV head) segments form a stream
// too, cut into equal ranges, one per warp.  A warp loads its pages straight from
// global memory into mma.sync fragments (bf16_tile.cuh), a page ahead and prefetched into
// L2 a page before that, and writes a
// state where a segment ends: no warp waits for another, and nothing is paid per
// segment but its state.  That takes 230 registers, so eight warps of the CTA do it
// and the others give theirs up.  (Twelve warps with rings in shared memory: a page took
// 1500 cycles of work and 2000 to issue its cp.async copies, or as long for its two TMA
// boxes; own parts of 64 sequences of up to 4096, 537 MB, behind 2048 shared tokens: 123 and 113 us,
// now 105, without the prefetch 134.)
//
// fp8 pages.  On prefixes, warp 0 copies whole pages and others make the operands of
// them: warps 2 and 3 K's codes exactly in f16 (and Q in f16 over 16), the output warps, which
// have time, V's, in the transposed order that the page has, exactly in bf16.  K's scales multiply the
// scores' columns, V's the weights before they are rounded to bf16, whose range is the scales'
// own.  Own keys go as in decode_direct.cu, pages through two buffers per warp.
//
// Every wait on a barrier is bounded: a timeout records KVATTN_ERR_TIMEOUT, the
// roles stop waiting, drain their copies and MMAs, free TMEM and return.
#include <algorithm>
#include <climits>
#include <cmath>
#include <cstring>

#include "bf16_tile.cuh"
#include "fp8_tile.cuh"
#include "tc_roles.cuh"

namespace kvattn {
namespace {

constexpr int kBM = 128;       // rows per tile
constexpr int kBN = 128;       // keys per tile
constexpr int kPage = 16;      // tokens per TMA copy of one block
constexpr int kPages = kBN / kPage;
constexpr int kThreads = 512;
constexpr int kStages = 2;     // of K, of V and of Q tiles
constexpr int kPanel = kBM * 128;  // 16 KB: 128 rows x 64 columns (one 128-byte swizzle panel of Q)
constexpr int kMinShared = 128;  // tokens of a prefix that is worth pieces of its own
constexpr int kMinPer = 8;     // fewest shared pages of a CTA's range
constexpr int kMinOwn = 2;     // fewest own pages of a warp's range
constexpr float kSetUpBytes = 180000.f, kSegmentBytes = 80000.f;  // of K and V that take as long (ranges_of)
constexpr int kOwnAhead = 1;  // bf16: pages between the one a warp loads and the one it prefetches into L2
constexpr int kPast = 4;       // pieces whose sums may be waiting for the output warps
constexpr int kRaw = 2;        // fp8: stages of pages
// Tiles whose pages' presence is kept.  It is written before the wait for the tile's stage and read by the
// tile's softmax: the stage of the tile before was free after S of three tiles before, which was issued after
// the P.V, and so after the softmax, of five tiles before; fp8's conversion may be a tile behind that.
constexpr int kHave = 8;
static_assert(kSharedRows == 2 * kBM, "a prefix piece's rows");
static_assert(kMaxGroups <= kThreads, "a thread per group");
// Registers per thread of the warpgroups (the block starts with 128 each:
// 112 + 2 x 152 + 96 = 4 x 128).  With 96, 168 and 80 some spill, 105.3 us for the 12 prompts, not 103.3.
constexpr int kRegsIssue = 112, kRegsSoftmax = 152, kRegsOutput = 96;
constexpr int kRegsOwn = 232, kRegsIdle = 24;  // 2 x 232 + 2 x 24 = 4 x 128
// Warps of a CTA on own keys: 4 .. 11, or all of them (fp8).
template <bool kF8>
__host__ __device__ constexpr int own_warps() { return kF8 ? kThreads / 32 : 8; }

// Barriers of a CTA on prefixes.
struct Bars {
    uint64_t q_full[kStages], q_empty[kStages];  // of a Q tile: loaded; every S MMA that reads it is done
    uint64_t k_full[kStages], k_empty[kStages], v_full[kStages], v_empty[kStages];
    uint64_t s_full[2], p_full[2];
    uint64_t o_done[2], o_free[2];   // the piece's last P.V into O_z has completed; O_z has been read
    uint64_t l_full[kPast];          // maxima and row sums of a piece
    // fp8: pages loaded, read; scales and Q converted (K and V: k_full[0], v_full[0] then)
    uint64_t raw_full[kRaw], raw_empty[kRaw], scales[kPast], q_f16[kStages];
    uint64_t drain;
    uint32_t have[kHave];  // bit i: page i of the tile is there
    uint32_t tmem;
    int abort_flag;
};
static_assert(sizeof(Bars) <= 384, "the barriers fit before the exchange area");

// The call's groups and sequences, and the streams of pages: group g's shared ones are
// first[g] .. first[g+1] - 1 (segments: KV heads outermost, then row blocks; their rows
// rows[g] ..), sequence b's own Hkv own[b] .. Hkv own[b+1] - 1.
struct Plan {
    int cu[kMaxGroups + 1];
    int tokens[kMaxGroups];   // shared, whole pages; 0: shares nothing
    int leader[kMaxGroups];   // a sequence of the group that has them
    int members[kMaxGroups];  // how many have them
    int first[kMaxGroups + 1], rows[kMaxGroups + 1];
    int own[kMaxSharedBatch + 1];
    int segments;  // of all groups
    int two_rows;  // shared pages of segments of two row tiles
    int sums[3][kThreads / 32];
};

template <int kD, bool kF8>
struct Geo {
    static constexpr int kPanels = kD / 64;
    static constexpr int kTileBytes = kBM * kD * 2;    // a Q tile, a K stage or a V stage
    static constexpr int kGroup = 8 * kD * 2;          // one 8-key group of a stage (all panels)
    static constexpr int kPageBytes = kPage * kD * 2;  // one page of K or V
    static constexpr int kCost = kF8 ? kF8Page : 2 * kPageBytes;  // bytes of a page of both
    static constexpr int kRawBytes = kPages * kF8Page;
    static constexpr int kKV = kF8 ? 1 : kStages;      // stages of K and of V
    static constexpr int kOffQ = 0;
    static constexpr int kOffK = kStages * kTileBytes;
    static constexpr int kOffV = kOffK + kKV * kTileBytes;
    static constexpr int kOffRaw = kOffV + kKV * kTileBytes;
    static constexpr int kOffScales = kOffRaw + (kF8 ? kRaw * kRawBytes : 0);  // of kPast tiles: K's [128], V's [128]
    static constexpr int kOffBar = kOffScales + (kF8 ? kPast * 1024 : 0);
    // fp32: row maxima of a tile [2][2 halves][128]; of kPast pieces, row sums [2 halves][2][128] and maxima [2][128]
    static constexpr int kOffX = kOffBar + 384;
    static constexpr int kOffPlan = kOffX + 2048 + kPast * 768 * 4;
    static constexpr int kSmemBytes = kOffPlan + (int)sizeof(Plan) + 1024;  // + slack to align the base to 1 KB
    static constexpr int kOffRing = 4 * kMaxSharedBatch;  // own keys, fp8: pages of the warps, behind the lengths
    static_assert(kD == 64 || kD == 128, "head dim");
    static_assert(!kF8 || kOffRing + kThreads / 32 * 2 * kF8Page <= kOffBar, "the rings");
};

struct Maps {
    CUtensorMap q;  // 3-D: (D, Hq, batch), box (64, G, 128 / G)
    CUtensorMap k;  // 4-D: (64 columns, 8 rows, 2 panels, rows / 8), box (64, 8, 2, 2); D = 64: 2-D, box (64, 16)
    CUtensorMap v;
};

template <int kHD>
__device__ __forceinline__ void copy_page(void* dst, const CUtensorMap* m, int row, uint64_t* full, uint64_t policy)
{
    if constexpr (kHD == 128) tma_load_4d(dst, m, 0, 0, 0, row >> 3, full, policy);
    else tma_load_2d(dst, m, 0, row, full, policy);
}

// Pages of `len` tokens, which may be up to INT_MAX.
__device__ __forceinline__ int pages_of(int len) { return (int)(((unsigned)len + (kPage - 1)) / kPage); }

__device__ __forceinline__ int blocks_of(int seqs, int lg) { return ((seqs << lg) + kSharedRows - 1) / kSharedRows; }

// The last group g of n with cu[g] <= b: the one b is in.
__device__ __forceinline__ int group_of(const Plan& P, int n, int b)
{
    int g = 0;
    for (int m = n; m > 1;) {
        const int half = m >> 1;
        if (P.cu[g + half] <= b) g += half;
        m -= half;
    }
    return g;
}

// Fills the plan from the call's arguments (every CTA does), and `len` with the
// sequences' lengths, 0 for one out of range.  Groups that are out of order or out of
// range share nothing, nor does a prefix of fewer than kMinShared tokens, or of which
// fewer than two sequences have it all.
__device__ __forceinline__ void make_plan(const SharedArgs& a, Plan& P, int* len, int lg)
{
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, n = a.num_groups;
    const int per = (a.d.batch + kThreads - 1) / kThreads;  // sequences of a thread, mostly one
    const int b0 = tid * per, b1 = min(b0 + per, a.d.batch);
    const int64_t room = (int64_t)a.d.max_blocks * a.d.block_size;
    bool ok = true;
    if (tid < n) {
        const int c0 = a.cu_groups[tid], c1 = a.cu_groups[tid + 1], s = a.shared_lens[tid];
        ok = c0 >= 0 && c1 >= c0 && c1 <= a.d.batch && s >= 0 && s <= a.max_shared && (tid > 0 || c0 == 0) && s <= room;
        P.cu[tid] = c0;
        if (tid == n - 1) P.cu[n] = c1;
        P.tokens[tid] = s >= kMinShared ? s & ~(kPage - 1) : 0;
        P.leader[tid] = INT_MAX;
        P.members[tid] = 0;
    }
    if (tid == 0) P.segments = P.two_rows = 0;
    // (loops are not unrolled: the instructions of this are fetched once per call, which is
    // what it waits for)
#pragma unroll 1
    for (int b = b0; b < b1; ++b) {
        int L = a.d.seq_lens[b];
        if (L < 0 || L > a.d.max_seq_len || L > room) {
            if (blockIdx.x == 0) record_error(a.d.status, KVATTN_ERR_BAD_INDEX);
            L = 0;
        }
        len[b] = L;
    }
    ok = __syncthreads_and(ok);
    if (!ok && blockIdx.x == 0 && tid == 0) record_error(a.d.status, KVATTN_ERR_BAD_INDEX);
    auto has = [&](int b) {  // the group whose shared tokens sequence b has, -1: none
        if (!ok || b >= P.cu[n]) return -1;
        const int g = group_of(P, n, b);
        return P.tokens[g] > 0 && len[b] >= P.tokens[g] ? g : -1;
    };
#pragma unroll 1
    for (int b = b0; b < b1; ++b) {
        const int g = has(b);
        P.own[b + 1] = g;
        if (g >= 0) {
            atomicMin(&P.leader[g], b);
            atomicAdd(&P.members[g], 1);
        }
    }
    __syncthreads();
    auto shared = [&](int g) { return ok && P.members[g] >= 2 ? P.tokens[g] / kPage : 0; };  // pages
    int v[3] = {0, 0, 0};  // pages of a group, rows of its segments; own pages of this thread's sequences
    int tokens = 0;
    if (tid < n && (tokens = shared(tid) * kPage) > 0) {
        const int seqs = P.cu[tid + 1] - P.cu[tid], rows = seqs << lg, segments = blocks_of(seqs, lg) * a.d.hkv;
        v[0] = segments * (tokens / kPage);
        v[1] = rows * a.d.hkv;
        atomicAdd(&P.segments, segments);
        atomicAdd(&P.two_rows, (rows + kSharedRows - kBM - 1) / kSharedRows * a.d.hkv * (tokens / kPage));
    }
#pragma unroll 1
    for (int b = b0; b < b1; ++b) {
        const int g = P.own[b + 1];
        P.own[b + 1] = v[2] += pages_of(len[b]) - (g >= 0 ? shared(g) : 0);
    }
    const int mine = v[2];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1)
#pragma unroll
        for (int i = 0; i < 3; ++i) {
            const int x = __shfl_up_sync(0xffffffffu, v[i], o);
            if (lane >= o) v[i] += x;
        }
    if (lane == 31)
#pragma unroll
        for (int i = 0; i < 3; ++i) P.sums[i][warp] = v[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 3; ++i) v[i] += __reduce_add_sync(0xffffffffu, lane < warp ? P.sums[i][lane] : 0);
    if (tid < n) {
        P.first[tid + 1] = v[0];
        P.rows[tid + 1] = v[1];
        P.tokens[tid] = tokens;
    }
#pragma unroll 1
    for (int b = b0; b < b1; ++b) P.own[b + 1] += v[2] - mine;
    if (tid == 0) P.first[0] = P.rows[0] = P.own[0] = 0;
    __syncthreads();
}

// How many CTAs are on prefixes, and the pages of a CTA's and of an own warp's range.
struct Ranges {
    int ctas, per, own_per;
};
// In times of a shared page of one row tile: one of two takes 1 + kTwo (fp8, whose conversion and
// softmax bound it; bf16 pages are HBM's), an own page kPage + kMore x^2, x the prefixes' part of the
// work (a CTA on a prefix has more of its copies under way, so own bf16 pages take longer the
// more such CTAs share HBM with them), an own segment kSegment besides (state, queries), a prefix CTA `set_up`
// besides its pages (tensor memory, the pipeline's filling) and `segment` for each of its
// segments (256 rows of output); so with t for all,
// p / (t - set_up) + o / t = ctas.
// Measured with inputs that change from call to call, us of this kernel alone (the merge has 4.5 to 6.5 besides;
// 64 sequences but for two): bf16 (kPage, kMore), 2048 shared and up to 512 own
// tokens | 12 prompts of up to 8191, 192 sequences, 1024 own | 32 x (65536, 256): 0.6, 1: 23.4 | 104 |
// 55; 0.85, 1: 26.5 | 127 | 55; 0.4, 1.2: 26.4 | 112 | 55; 0.95, 0.8: 26.7 | 136 | 55; before own pages came
// by way of L2, 1, 0: 27.2 | 129 | 72.  fp8 (kPage, kSegment, kTwo), 16384
// and 1024 | 8192 and 2048 | 16 x (8192, 2048): 1, 4, 1.4: 72 | 77 | 29; 1, 4, 1: 75 | 83 | 29; 0.8, 4, 1.2: 71 | 73 | 26;
// 0.8, 4, 2: 70 | 64 | -; 1, 4, 2.4: 69 | 67 | -; 0.6, 3, 1.6: 83 | 68 | -; 1.2, 4, 1.6: 74 | 78 | 28; a page of two row tiles counted as of one: 1, 2: 89 and 0.4, 2: 71 | 69 | -,
// but 16 x 8192 shared by 4s, with 32 own, 56 instead of 40.  As the code is now: 22.6 | 101 | 54.5, and fp8 16384
// and 1024 69.5.  The bf16 constants were chosen at 32 / 8 heads of 128 and serve D = 64 and groups of 1, 2 and 8
// untuned (figures of those: prefixes_once in api.cu).
template <bool kF8>
struct OwnCost {
    static constexpr float kPage = kF8 ? 0.8f : 0.6f, kMore = kF8 ? 0.f : 1.0f, kSegment = kF8 ? 4.f : 1.f,
                           kTwo = kF8 ? 2.0f : 0.f;
};
template <bool kF8>
__device__ __forceinline__ Ranges ranges_of(int shared, int two_rows, int segments, int own, int own_segments, int ctas,
                                            float set_up, float segment)
{
    using C = OwnCost<kF8>;
    constexpr int warps = own_warps<kF8>();
    Ranges r{0, 0, 0};
    if (shared > 0) {
        const float c = (float)ctas, p = (float)shared + C::kTwo * (float)two_rows + segment * (float)segments,
                    part = p / (p + (float)own),
                    o = (C::kPage + C::kMore * part * part) * (float)own + C::kSegment * (float)own_segments,
                    u = set_up * c + p + o;
        const float t = (u + sqrtf(fmaxf(u * u - 4.f * c * set_up * o, 0.f))) / (2.f * c);
        r.ctas = min((int)ceilf(p / fmaxf(t - set_up, 1.f)), (shared + kMinPer - 1) / kMinPer);
        r.ctas = max(1, min(r.ctas, own > 0 ? ctas - 1 : ctas));
        r.per = (shared + r.ctas - 1) / r.ctas;
    }
    if (own > 0) {
        const int n = (ctas - r.ctas) * warps;
        r.own_per = max((own + n - 1) / n, kMinOwn);
    }
    return r;
}

// ---------------------------------------------------------------- prefixes

// A piece: pages p0 .. p1 - 1 of row `row` of the table for KV head h and `rows`
// rows: head r % G of sequence b0 + r / G.  Its results go to rows `out` ...
struct Piece {
    int row, b0, rows, h, p0, p1, out;
    __device__ __forceinline__ bool two() const { return rows > kBM; }
    __device__ __forceinline__ int tiles() const { return (p1 - p0 + kPages - 1) / kPages; }
    // Steps of S, softmax and P.V: step j is of key tile tile(j), and of the first or second
    // row tile by turns if there are two.
    __device__ __forceinline__ int steps() const { return two() ? 2 * tiles() : tiles(); }
    __device__ __forceinline__ int tile(int j) const { return two() ? j >> 1 : j; }
    __device__ __forceinline__ int pages(int t) const { return min(kPages, p1 - p0 - t * kPages); }
};

// Walks the pieces of a CTA's range.
struct Walk {
    int r, end, g;
    __device__ __forceinline__ bool next(const SharedArgs& a, const Plan& P, int lg, Piece& p)
    {
        if (r >= end) return false;
        while (P.first[g + 1] <= r) ++g;
        const int pages = P.tokens[g] / kPage, seqs = P.cu[g + 1] - P.cu[g], blocks = blocks_of(seqs, lg);
        const int off = r - P.first[g], seg = off / pages;
        p.p0 = off - seg * pages;
        p.p1 = min(pages, p.p0 + end - r);
        p.h = seg / blocks;
        const int rb = seg - p.h * blocks;
        p.row = P.leader[g];
        p.b0 = P.cu[g] + rb * (kSharedRows >> lg);
        p.rows = min(kSharedRows, (seqs << lg) - rb * kSharedRows);
        p.out = (int)blockIdx.x * kSharedRows + P.rows[g] + p.h * (seqs << lg) + rb * kSharedRows;
        r += p.p1 - p.p0;
        return true;
    }
};

// fp8: Q tile `q` of the CTA, as loaded, to f16 over 16 in place, by 64 threads r.
__device__ __forceinline__ bool convert_q(Bars& B, unsigned char* tile, int q, int r, volatile int* abort_flag, int* status)
{
    if (!long_wait(&B.q_full[q % kStages], (q / kStages) & 1, 0, abort_flag, status)) return false;
    uint4* p = reinterpret_cast<uint4*>(tile);
#pragma unroll 4
    for (int i = r; i < kBM * 128 * 2 / 16; i += 64) {
        const uint4 v = p[i];
        auto half2 = [](uint32_t u) { return pack_f16_rn(bf16lo(u) * 0.0625f, bf16hi(u) * 0.0625f); };
        p[i] = make_uint4(half2(v.x), half2(v.y), half2(v.z), half2(v.w));
    }
    fence_async_smem();
    mbar_arrive(&B.q_f16[q % kStages]);
    return true;
}

// Tile g of the CTA, `pages` pages: K's codes to f16 (exact), in 64-column panels of 128
// rows (keys) with 128-byte swizzle, and the scales, K's times `mul`, by 64 threads r.
__device__ __forceinline__ bool convert_k(Bars& B, unsigned char* smem, float mul, int pages, int g, int r,
                                          volatile int* abort_flag, int* status)
{
    using GE = Geo<128, true>;
    const int s = g % kRaw;
    if (!long_wait(&B.raw_full[s], (g / kRaw) & 1, 1, abort_flag, status)) return false;
    const unsigned char* raw = smem + GE::kOffRaw + s * GE::kRawBytes;
    if (g > 0 && !long_wait(&B.k_empty[0], (g - 1) & 1, 1, abort_flag, status)) return false;
    // (S of tile g - 1 was issued after the P.V of tile g - 3, whose softmax has read the
    // scales of tile g - kPast)
    float* sc = reinterpret_cast<float*>(smem + GE::kOffScales + (g % kPast) * 1024);
    for (int i = r; i < pages * kPage; i += 64) {
        const unsigned char* pg = raw + (i >> 4) * kF8Page;
        sc[i] = reinterpret_cast<const float*>(pg + kF8KsOff)[i & 15] * mul;
        sc[128 + i] = reinterpret_cast<const float*>(pg + kF8VsOff)[i & 15];
    }
    mbar_arrive(&B.scales[g % kPast]);
    // thread r has chunk place r % 8 of tokens r / 8 and r / 8 + 8 of each page
    const int t0 = r >> 3;
    unsigned char* dst = smem + GE::kOffK + t0 * 128;
    const int c0 = (r & 7) ^ f8_swz(t0), c1 = (r & 7) ^ f8_swz(t0 + 8);  // their dims' chunks
    auto put = [&](unsigned char* row, int c, const uint4& w) {
        unsigned char* at = row + (c >> 2) * kPanel;
        const int i0 = ((2 * (c & 3)) ^ (t0 & 7)) << 4;
        *reinterpret_cast<uint4*>(at + i0) = make_uint4(e4m3x2_to_f16x2(w.x), e4m3x2_to_f16x2(w.x >> 16),
                                                        e4m3x2_to_f16x2(w.y), e4m3x2_to_f16x2(w.y >> 16));
        *reinterpret_cast<uint4*>(at + (i0 ^ 16)) = make_uint4(e4m3x2_to_f16x2(w.z), e4m3x2_to_f16x2(w.z >> 16),
                                                               e4m3x2_to_f16x2(w.w), e4m3x2_to_f16x2(w.w >> 16));
    };
#pragma unroll 2
    for (int p = 0; p < pages; ++p) {
        const uint4 x = *reinterpret_cast<const uint4*>(raw + p * kF8Page + 16 * r);
        const uint4 y = *reinterpret_cast<const uint4*>(raw + p * kF8Page + 16 * r + 1024);
        put(dst + p * (kPage * 128), c0, x);
        put(dst + p * (kPage * 128) + 1024, c1, y);
    }
    fence_async_smem();
    mbar_arrive(&B.k_full[0]);
    mbar_arrive(&B.raw_empty[s]);
    return true;
}

// ... and V's to bf16 (exact), in panels of 128 rows (dims) of 64 keys, by 128 threads r.
__device__ __forceinline__ bool convert_v(Bars& B, unsigned char* smem, int pages, int g, int r, volatile int* abort_flag,
                                          int* status)
{
    using GE = Geo<128, true>;
    const int s = g % kRaw;
    if (!long_wait(&B.raw_full[s], (g / kRaw) & 1, 1, abort_flag, status)) return false;
    if (g > 0 && !long_wait(&B.v_empty[0], (g - 1) & 1, 1, abort_flag, status)) return false;
    const unsigned char* raw = smem + GE::kOffRaw + s * GE::kRawBytes + kF8VOff + 16 * r;  // dim r
    unsigned char* dst = smem + GE::kOffV + r * 128;
    auto bf16x2 = [](uint32_t two) {
        const uint32_t h = e4m3x2_to_f16x2(two);
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
        return pack_bf16_rn(f.x, f.y);
    };
#pragma unroll 2
    for (int p = 0; p < pages; ++p) {
        const uint4 w = *reinterpret_cast<const uint4*>(raw + p * kF8Page);
        unsigned char* at = dst + (p >> 2) * kPanel;
        const int i0 = ((2 * (p & 3)) ^ (r & 7)) << 4;
        *reinterpret_cast<uint4*>(at + i0) = make_uint4(bf16x2(w.x), bf16x2(w.x >> 16), bf16x2(w.y), bf16x2(w.y >> 16));
        *reinterpret_cast<uint4*>(at + (i0 ^ 16)) = make_uint4(bf16x2(w.z), bf16x2(w.z >> 16), bf16x2(w.w), bf16x2(w.w >> 16));
    }
    fence_async_smem();
    mbar_arrive(&B.v_full[0]);
    mbar_arrive(&B.raw_empty[s]);
    return true;
}

template <int kHD, bool kF8>
__device__ __forceinline__ void prefix_cta(const SharedArgs& a, const Maps& maps, const Plan& P, const Walk walk0, int lg,
                                           unsigned char* smem)
{
    using GE = Geo<kHD, kF8>;
    constexpr int kTileBytes = GE::kTileBytes, kPageBytes = GE::kPageBytes, kGroup = GE::kGroup, kKV = GE::kKV;
    constexpr int kOffQ = GE::kOffQ, kOffK = GE::kOffK, kOffV = GE::kOffV;
    Bars& B = *reinterpret_cast<Bars*>(smem + GE::kOffBar);
    volatile int* abort_flag = &B.abort_flag;
    int* const status = a.d.status;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int x = 0; x < 2; ++x) {
            mbar_init(&B.q_full[x], 1);
            mbar_init(&B.q_empty[x], 1);
            mbar_init(&B.k_full[x], kF8 ? 64 : 1);
            mbar_init(&B.k_empty[x], 1);
            mbar_init(&B.v_full[x], kF8 ? 128 : 1);
            mbar_init(&B.v_empty[x], 1);
            mbar_init(&B.s_full[x], 1);
            mbar_init(&B.p_full[x], 256);
            mbar_init(&B.o_done[x], 1);
            mbar_init(&B.o_free[x], 128);
        }
        for (int x = 0; x < kPast; ++x) {
            mbar_init(&B.l_full[x], 256);
            mbar_init(&B.scales[x], 64);
        }
        for (int x = 0; x < kRaw; ++x) {
            mbar_init(&B.raw_full[x], 1);
            mbar_init(&B.raw_empty[x], 192);
            mbar_init(&B.q_f16[x], 64);
        }
        mbar_init(&B.drain, 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 1) tmem_alloc(&B.tmem, 512);
    fence_async_smem();  // (the lengths were where copies go now)
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = B.tmem;  // S_0 at +0, S_1 at +128, O_0 at +256, O_1 at +384

    if (warp < 4) {
        setmaxnreg_dec<kRegsIssue>();
        if (warp == 0 || (warp == 2 && !kF8)) {
            // ====================== TMA producers: K and Q, V ======================
            const uint64_t pol = l2_evict_normal_policy();
            const bool is_k = warp == 0;
            if (lane == 0) {
                if (is_k) tma_prefetch_map(&maps.q);
                if (!kF8) tma_prefetch_map(is_k ? &maps.k : &maps.v);
            }
            bool go = true;
            // lane 0 waits for `empty` (unless the buffer is new) and arms `full`
            auto arm = [&](uint64_t* full, uint64_t* empty, int use, uint32_t bytes) -> bool {
                if (lane == 0) {
                    go = use == 0 ? !*abort_flag : wait_or_abort(empty, (use - 1) & 1, abort_flag, status);
                    if (go) mbar_arrive_expect_tx(full, bytes);
                }
                return go = __shfl_sync(0xffffffffu, go, 0);
            };
            // ... of a tile without all its pages, with zeros in their places: V's weights are 0 (and
            // 0 * NaN would not be), and fp8 pages have scales.
            auto arm_gaps = [&](uint64_t* full, uint64_t* empty, int use, uint32_t bytes, unsigned char* stage, int page_bytes,
                                int pages, uint32_t have) -> bool {
                if (lane == 0) go = use == 0 ? !*abort_flag : wait_or_abort(empty, (use - 1) & 1, abort_flag, status);
                if (!(go = __shfl_sync(0xffffffffu, go, 0))) return false;
                for (int i = 0; i < pages; ++i)
                    if (!(have >> i & 1u))
                        for (int x = lane; x < page_bytes / 16; x += 32)
                            reinterpret_cast<uint4*>(stage + i * page_bytes)[x] = make_uint4(0, 0, 0, 0);
                fence_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive_expect_tx(full, bytes);
                __syncwarp();
                return true;
            };
            // Lane i < 8 copies page i of a tile; its block's id comes from the table a
            // tile ahead (lanes without a page read their row's first entry).
            auto block_id = [&](const Piece& p, int t) -> int32_t {
                const int col = lane < p.pages(t) ? (p.p0 + t * kPages + lane) * kPage / a.d.block_size : 0;
                return a.d.block_table[(int64_t)p.row * a.d.max_blocks + col];
            };
            auto pool_row = [&](const Piece& p, int t, int32_t blk) -> int {
                if (lane >= p.pages(t)) return -1;
                if (blk < 0 || blk >= a.d.num_blocks) {
                    if (is_k) record_error(status, KVATTN_ERR_BAD_INDEX);
                    return -1;
                }
                return (int)(((int64_t)blk * a.d.hkv + p.h) * a.d.block_size) +
                       (p.p0 + t * kPages + lane) * kPage % a.d.block_size;
            };
            int g = 0, qg = 0;  // K (or V) and Q tiles armed so far
            Walk w = walk0;
            Piece p, ahead;
            bool more = w.next(a, P, lg, ahead);
            int32_t blk_next = block_id(ahead, 0);
            while (go && more) {
                p = ahead;
                const int n = p.tiles();
                for (int t = 0; t < n; ++t) {
                    const int row = pool_row(p, t, blk_next);
                    const uint32_t have = __ballot_sync(0xffffffffu, row >= 0);
                    constexpr int kBytes = kF8 ? kF8Page : kPageBytes;
                    const uint32_t bytes = (uint32_t)__popc(have) * (uint32_t)kBytes;
                    const bool gaps = (kF8 || !is_k) && have != (1u << p.pages(t)) - 1u;
                    if (is_k && lane == 0) B.have[g % kHave] = have;
                    static_assert(kRaw == kStages, "stages of pages as of tiles");
                    const int s = g % kStages;
                    uint64_t* full = kF8 ? &B.raw_full[s] : is_k ? &B.k_full[s] : &B.v_full[s];
                    uint64_t* empty = kF8 ? &B.raw_empty[s] : is_k ? &B.k_empty[s] : &B.v_empty[s];
                    unsigned char* stage = smem + (kF8 ? GE::kOffRaw + s * GE::kRawBytes : kOffV + s * kTileBytes);
                    if (__builtin_expect(gaps, 0)
                            ? !arm_gaps(full, empty, g / kStages, bytes, stage, kBytes, p.pages(t), have)
                            : !arm(full, empty, g / kStages, bytes))
                        break;
                    if (kF8 && row >= 0)
                        bulk_load(smem + GE::kOffRaw + s * GE::kRawBytes + lane * kF8Page,
                                  (const char*)a.d.k_pool + (int64_t)(row / kPage) * kF8Page, kF8Page, full, pol);
                    else if (row >= 0)
                        copy_page<kHD>(smem + (is_k ? kOffK : kOffV) + s * kTileBytes + lane * kPageBytes,
                                       is_k ? &maps.k : &maps.v, row, full, pol);
                    ++g;
                    if (t + 1 == n) {
                        more = w.next(a, P, lg, ahead);
                        if (more) blk_next = block_id(ahead, 0);
                    } else {
                        blk_next = block_id(p, t + 1);
                    }
                    if (is_k && t == 0) {
                        const int tiles = p.two() ? 2 : 1;
                        for (int x = 0; x < tiles; ++x) {
                            const int qs = qg % kStages;
                            if (!arm(&B.q_full[qs], &B.q_empty[qs], qg / kStages, (uint32_t)kTileBytes)) break;
                            if (lane < GE::kPanels)
                                tma_load_3d(smem + kOffQ + qs * kTileBytes + lane * kPanel, &maps.q, 64 * lane, p.h << lg,
                                            p.b0 + x * (kBM >> lg), &B.q_full[qs], pol);
                            ++qg;
                        }
                        if (!go) break;
                    }
                }
            }
            // After an abort, let every armed copy land before the CTA can exit.
            __syncwarp();
            if (lane == 0 && *abort_flag) {
                for (int t = max(0, g - kStages); t < g; ++t)
                    mbar_wait(kF8 ? &B.raw_full[t % kStages] : is_k ? &B.k_full[t % kStages] : &B.v_full[t % kStages],
                              (t / kStages) & 1, status);
                for (int t = max(0, qg - kStages); t < qg; ++t) mbar_wait(&B.q_full[t % kStages], (t / kStages) & 1, status);
            }
        } else if (warp == 1) {
            // ============================== MMA issuer ==============================
            // The whole warp runs the schedule (waits agreed by the warp) and one
            // elected lane issues.  Operand descriptors are built once: a stage or
            // k-step only adds (byte offset >> 4) to the start-address field, which
            // cannot carry out of it (shared-memory offsets stay below 256 KB).
            // (converted fp8 operands have 64-column panels of 128 rows, as Q; V's rows are dims)
            constexpr uint32_t idesc_s = kF8 ? idesc_f16_f32(kBM, 0, false) : idesc_bf16_f32(kBM, 0, false);  // N: the tile's keys
            constexpr uint32_t idesc_o = idesc_bf16_f32(kBM, kHD, !kF8);
            const uint32_t sbase = smem_addr(smem);
            const uint64_t dQ = umma_desc_sw128(sbase + kOffQ, 16, 1024);
            const uint64_t dK = umma_desc_sw128(sbase + kOffK, 16, kF8 ? 1024 : kGroup);
            const uint64_t dV = kF8 ? umma_desc_sw128(sbase + kOffV, 16, 1024) : umma_desc_sw128(sbase + kOffV, 1024, kGroup);
            uint64_t* const q_ready = kF8 ? B.q_f16 : B.q_full;
            constexpr uint64_t kTileStep = kTileBytes >> 4;
            auto wait = [&](uint64_t* b, uint32_t parity) {
                if (__all_sync(0xffffffffu, mbar_try_wait(b, parity))) return true;
                return warp_wait(b, parity, abort_flag, status);
            };
            // Steps through the pieces: the S and the P.V of each.
            struct Steps {
                Walk w;
                Piece p;
                bool more;
                int j, n;    // of the piece p
                int x;       // S_x is this step's, the next step's the other
                int z;       // O_z is the piece's (two row tiles: O_0 and O_1)
                int kv, q;   // K (or V) and Q tiles of the pieces before
            };
            auto start = [&](Steps& s) {
                s.j = 0;
                s.n = (s.more = s.w.next(a, P, lg, s.p)) ? s.p.steps() : 0;
            };
            auto advance = [&](Steps& s) {
                s.x ^= 1;
                if (++s.j < s.n) return;
                if (!s.p.two()) s.z ^= 1;
                s.kv += s.p.tiles();
                s.q += s.p.two() ? 2 : 1;
                start(s);
            };
            // The K stage is free after the last S that reads it, the Q tile after the
            // piece's last.
            auto do_s = [&](const Steps& s) -> bool {
                const bool two = s.p.two();
                const int y = s.j & 1, x = s.x, t = s.p.tile(s.j), k = s.kv + t, q = s.q + (two ? y : 0);
                const uint32_t idesc = idesc_s | ((uint32_t)(s.p.pages(t) * kPage >> 3) << 17);
                if (t == 0 && !wait(&q_ready[q % kStages], (q / kStages) & 1)) return false;
                if (!wait(&B.k_full[k % kKV], (k / kKV) & 1)) return false;
                tc_fence_after();
                if (elect_one()) {
                    const uint64_t qd = dQ + (q % kStages) * kTileStep, kd = dK + (k % kKV) * kTileStep;
                    const uint32_t d = tmem + x * 128;
#pragma unroll
                    for (int i = 0; i < kHD / 16; ++i)  // k-step: 16 columns, 32 B inside the 128-byte atom
                        tc_mma_f16(d, qd + (uint64_t)(((i >> 2) * kPanel + (i & 3) * 32) >> 4),
                                   kd + (uint64_t)(((i >> 2) * (kF8 ? kPanel : 1024) + (i & 3) * 32) >> 4), idesc, i > 0);
                    tc_commit(&B.s_full[x]);
                    if (!two || y == 1) tc_commit(&B.k_empty[k % kKV]);
                    if (s.j + (two ? 2 : 1) >= s.n) tc_commit(&B.q_empty[q % kStages]);
                }
                __syncwarp();
                return true;
            };
            // O_z += P_x V, P_x in S_x's first 64 columns, over the tile's pages; a piece's
            // first overwrites O_z (o_free: the piece before on it has been read)
            uint32_t seen = 0;    // bit x: parity of the P_x so far
            uint32_t pieces = 0;  // bits z, 2 + z: parity of the pieces on O_z so far, whether there are any
            auto do_pv = [&](const Steps& s) -> bool {
                const bool two = s.p.two(), first = s.j < (two ? 2 : 1);
                const int y = s.j & 1, x = s.x, z = two ? y : s.z, t = s.p.tile(s.j), v = s.kv + t;
                if (!wait(&B.v_full[v % kKV], (v / kKV) & 1) || !wait(&B.p_full[x], seen >> x & 1u)) return false;
                seen ^= 1u << x;
                if (first) {
                    if ((pieces >> (2 + z) & 1u) && !wait(&B.o_free[z], ~pieces >> z & 1u)) return false;
                    pieces = (pieces ^ 1u << z) | 4u << z;
                }
                tc_fence_after();
                if (elect_one()) {
                    const uint64_t vd = dV + (v % kKV) * kTileStep;
                    const uint32_t d = tmem + 256 + z * 128, pa = tmem + x * 128;
                    const int pages = s.p.pages(t);
#pragma unroll
                    for (int i = 0; i < kPages; ++i)  // k-step: 16 keys = two 8-key groups
                        if (i < pages)
                            tc_mma_f16_ts(d, pa + i * 8,
                                          vd + (uint64_t)((kF8 ? (i >> 2) * kPanel + (i & 3) * 32 : i * 2 * kGroup) >> 4), idesc_o,
                                          (!first || i > 0));
                    if (!two || y == 1) tc_commit(&B.v_empty[v % kKV]);
                    if (s.j + (two ? 2 : 1) >= s.n) tc_commit(&B.o_done[z]);
                }
                __syncwarp();
                return true;
            };
            // P.V of a step, then S of the second step after it, whichever piece that is
            // of: it overwrites S_x's columns after P.V has read P_x from them (tensor
            // operations of one thread run in issue order).
            Steps fs{walk0, {}, false, 0, 0, 0, 0, 0, 0}, fo = fs;
            start(fs);
            start(fo);
            bool ok = true;
            for (int ahead = 0; ok && fo.more;) {
                if (ahead < 2 && fs.more) {
                    ok = do_s(fs);
                    advance(fs);
                    ++ahead;
                } else {
                    ok = do_pv(fo);
                    advance(fo);
                    --ahead;
                }
            }
            // every MMA this warp issued has completed once `drain` flips
            if (elect_one()) tc_commit(&B.drain);
            __syncwarp();
            mbar_wait(&B.drain, 0, status);
        } else if (kF8) {
            // ============================= K and Q to f16 =============================
            const int r = threadIdx.x - 64;
            int g = 0, q = 0;
            Walk w = walk0;
            Piece p;
            bool ok = true;
            while (ok && w.next(a, P, lg, p)) {
                for (int x = 0; ok && x < (p.two() ? 2 : 1); ++x, ++q)
                    ok = convert_q(B, smem + kOffQ + q % kStages * kTileBytes, q, r, abort_flag, status);
                const int n = p.tiles();
                for (int t = 0; ok && t < n; ++t, ++g)
                    ok = convert_k(B, smem, a.d.scale_log2 * 16.f, p.pages(t), g, r, abort_flag, status);
            }
        }
    } else if (warp < 12) {
        setmaxnreg_inc<kRegsSoftmax>();
        // ================================= softmax ==================================
        // All eight warps work on whichever S is due: thread (quarter, lane) owns row
        // r = 32 quarter + lane of the tile, warps 4-7 its columns 0..63 (half hf =
        // 0) and warps 8-11 its columns 64..127 (hf = 1).  The halves of a row agree on
        // the row max through shared memory, with a named barrier of that pair of
        // warps per tile.  These warps never stop early: after an abort their waits return
        // at once and they run on to the end (nothing of it is reported good).  The states
        // of two row tiles change places after each step.
        const int hf = (warp - 4) >> 2;
        const int quarter = warp & 3;        // TMEM lanes 32*quarter .. +31
        const int r = quarter * 32 + lane;   // row of the tile
        const uint32_t lane_base = (uint32_t)(quarter * 32) << 16;
        float* xchg = reinterpret_cast<float*>(smem + GE::kOffX);
        const float sl2 = kF8 ? 1.f : a.d.scale_log2;  // (fp8: in K's scales)
        uint32_t steps = 0;  // bit x: parity of the S_x seen so far
        int ii = 0, x = 0, z = 0, v = 0;  // v: V tiles of the pieces before
        Walk w = walk0;
        Piece p;
        while (w.next(a, P, lg, p)) {
            const bool two = p.two();
            const int n = p.steps();
            float m_now = -INFINITY, l_now = 0.f, m_other = -INFINITY, l_other = 0.f;
#pragma unroll 1
            for (int j = 0; j < n; ++j, x ^= 1) {
                const int y = j & 1;
                const uint32_t tS = tmem + lane_base + x * 128 + hf * 64;
                const uint32_t tO = tmem + lane_base + 256 + (two ? y : z) * 128 + hf * (kHD / 2);
                const int u = v + p.tile(j);
                wait_or_abort(&B.s_full[x], steps >> x & 1u, abort_flag, status);
                __syncwarp();
                steps ^= 1u << x;
                const int rows = p.rows - (two ? y * kBM : 0);  // of the tile (P of others may be anything)
                if (quarter * 32 < rows) {
                    const uint32_t have = B.have[u % kHave] >> (4 * hf) & 0xfu;  // pages of this half's columns
                    uint32_t sv[64];
                    tc_fence_after();
                    tmem_ld32(tS, *reinterpret_cast<uint32_t(*)[32]>(&sv[0]));
                    tmem_ld32(tS + 32, *reinterpret_cast<uint32_t(*)[32]>(&sv[32]));
                    tmem_ld_wait();
                    [[maybe_unused]] const float4* vs = nullptr;  // V's scales of this half's columns
                    if constexpr (kF8) {
                        const float4* ks = reinterpret_cast<const float4*>(smem + GE::kOffScales + (u % kPast) * 1024) + hf * 16;
                        vs = ks + 32;
                        wait_or_abort(&B.scales[u % kPast], (u / kPast) & 1, abort_flag, status);
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            const float4 k = ks[e];
                            sv[4 * e] = __float_as_uint(__uint_as_float(sv[4 * e]) * k.x);
                            sv[4 * e + 1] = __float_as_uint(__uint_as_float(sv[4 * e + 1]) * k.y);
                            sv[4 * e + 2] = __float_as_uint(__uint_as_float(sv[4 * e + 2]) * k.z);
                            sv[4 * e + 3] = __float_as_uint(__uint_as_float(sv[4 * e + 3]) * k.w);
                        }
                    }
                    if (have != 0xfu) {
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if (!(have >> i & 1u)) {
#pragma unroll
                                for (int e = 0; e < kPage; ++e) sv[kPage * i + e] = __float_as_uint(-INFINITY);
                            }
                    }
                    float m4[4];
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        m4[q] = fmaxf(__uint_as_float(sv[2 * q]), __uint_as_float(sv[2 * q + 1]));
#pragma unroll
                    for (int e = 8; e < 64; e += 8)
#pragma unroll
                        for (int q = 0; q < 4; ++q)
                            m4[q] = max3(m4[q], __uint_as_float(sv[e + 2 * q]), __uint_as_float(sv[e + 2 * q + 1]));
                    const float hm = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
                    float* slot = xchg + x * 256;
                    slot[hf * 128 + r] = hm;
                    bar_sync(1 + quarter, 64);
                    const float m_tile = fmaxf(hm, slot[(1 - hf) * 128 + r]) * sl2;
                    const bool none = m_now == -INFINITY;  // no score above -infinity so far
                    const bool rescale = !none && m_tile > m_now + 8.f && r < rows;
                    const float m_new = none || rescale ? m_tile : m_now;
                    const float alpha = none || r >= rows ? 1.f : fast_exp2(m_now - m_new);
                    m_now = m_new;
                    // P = 2^(s*scale*log2e - m) in bf16, into columns 32hf..32hf+31 of S_x
                    // (both halves have read their S before the barrier); scores that are
                    // all -infinity so far subtract +inf so every p is 0.  The row sum adds the
                    // fp32 p, whose rounding to bf16 is off by at most 2^-8 relative, at random.
                    uint32_t pw[32];
                    const float msub = m_now == -INFINITY ? INFINITY : m_now;
                    const uint64_t scale2 = pk(sl2, sl2), msub2 = pk(-msub, -msub);
                    uint64_t sum2[2] = {0, 0};
#pragma unroll
                    for (int e = 0; e < 32; ++e) {
                        const uint64_t xx =
                            ffma2(pk(__uint_as_float(sv[2 * e]), __uint_as_float(sv[2 * e + 1])), scale2, msub2);
                        const uint64_t pp = pk(fast_exp2(pk_lo(xx)), fast_exp2(pk_hi(xx)));
                        if constexpr (kF8) {
                            const float2 w = reinterpret_cast<const float2*>(vs)[e];
                            pw[e] = pack_bf16_rn(pk_lo(pp) * w.x, pk_hi(pp) * w.y);
                        } else {
                            pw[e] = pack_bf16_rn(pk_lo(pp), pk_hi(pp));
                        }
                        sum2[e & 1] = fadd2(sum2[e & 1], pp);
                    }
                    tmem_st32(tmem + lane_base + x * 128 + hf * 32, pw);
                    l_now = l_now * alpha + ((pk_lo(sum2[0]) + pk_hi(sum2[0])) + (pk_lo(sum2[1]) + pk_hi(sum2[1])));
                    // O (this half's columns): the P.V of two steps ago completed before this
                    // S_x was reported; the last step's, if it was of this O too, before its V
                    // stage was free.  The whole warp rescales if any of its rows must (alpha is 1
                    // for the others).
                    if (__any_sync(0xffffffffu, rescale && j > (two ? 1 : 0))) {
                        if (!two) {  // (tile u - 1)
                            wait_or_abort(&B.v_empty[(u - 1) % kKV], ((u - 1) / kKV) & 1, abort_flag, status);
                            __syncwarp();
                            tc_fence_after();
                        }
#pragma unroll 1
                        for (int q = 0; q < kHD / 64; ++q) {
                            uint32_t o[32];
                            tmem_ld32(tO + q * 32, o);
                            tmem_ld_wait();
#pragma unroll
                            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
                            tmem_st32(tO + q * 32, o);
                        }
                    }
                    tmem_st_wait();
                    tc_fence_before();
                }
                mbar_arrive(&B.p_full[x]);
                if (two) {
                    const float m = m_now, l = l_now;
                    m_now = m_other;
                    l_now = l_other;
                    m_other = m;
                    l_other = l;
                }
            }
            // This piece's maxima and sums to the output warps.  Those of piece ii - kPast
            // have been read: this piece's last S came after the P.V of two steps before, of
            // piece ii - 2 at least, whose first waited until the piece before it on its O, ii -
            // 4 at least, had been read, which its sums are before.
            float* lx = xchg + 512 + (ii % kPast) * 768;  // [2 halves][2 tiles][128 rows], then maxima [2][128]
            lx[(hf * 2 + 0) * 128 + r] = l_now;
            lx[(hf * 2 + 1) * 128 + r] = l_other;
            if (hf == 0) {
                lx[512 + r] = m_now;
                lx[640 + r] = m_other;
            }
            mbar_arrive(&B.l_full[ii % kPast]);
            ++ii;
            v += p.tiles();
            if (!two) z ^= 1;
        }
    } else {
        setmaxnreg_dec<kRegsOutput>();
        // ================================== output ==================================
        // Thread (quarter, lane) owns row r of a tile.  Rows go out of registers in
        // whole 32-byte sectors.
        const int quarter = warp & 3;
        const int r = quarter * 32 + lane;
        const uint32_t tO = tmem + ((uint32_t)(quarter * 32) << 16) + 256;
        const float* xchg = reinterpret_cast<const float*>(smem + GE::kOffX);
        uint32_t done = 0;  // bit z: parity of the pieces on O_z so far
        int ii = 0, z0 = 0;
        Walk w = walk0;
        Piece p, ahead;
        bool ok = true, more = w.next(a, P, lg, ahead);
        [[maybe_unused]] int g = 0;  // fp8: tiles converted so far
        auto convert = [&](const Piece& c, int t) {
            return !kF8 || convert_v(B, smem, c.pages(t), g++, r, abort_flag, status);
        };
        ok = convert(ahead, 0);
        while (ok && more) {
            p = ahead;
            const bool two = p.two();
            if constexpr (kF8) {
                const int n = p.tiles();
                for (int t = 1; ok && t < n; ++t) ok = convert(p, t);
            }
            more = w.next(a, P, lg, ahead);
            if (ok && more) ok = convert(ahead, 0);  // (the next piece's P.V do not wait for this one's output)
            if (!ok) break;
            if (!long_wait(&B.l_full[ii % kPast], (ii / kPast) & 1, p.tiles(), abort_flag, status)) break;
            const float* lx = xchg + 512 + (ii % kPast) * 768;
            const float l0 = lx[r] + lx[256 + r], l1 = lx[128 + r] + lx[384 + r], m0 = lx[512 + r], m1 = lx[640 + r];
            ++ii;
#pragma unroll 1
            for (int y = 0; y < (two ? 2 : 1); ++y) {
                const int z = two ? y : z0;
                if (!(ok = warp_wait(&B.o_done[z], done >> z & 1u, abort_flag, status))) break;
                done ^= 1u << z;
                tc_fence_after();
                const bool write = y * kBM + r < p.rows;
                const int64_t row = (int64_t)p.out + y * kBM + r;
                if (write) *reinterpret_cast<float2*>(a.ml + row * 2) = y ? make_float2(m1, l1) : make_float2(m0, l0);
                float* o = a.o + row * kHD;
#pragma unroll 1
                for (int q = 0; q < kHD / 32; ++q) {
                    uint32_t u[32];
                    tmem_ld32(tO + z * 128 + q * 32, u);
                    tmem_ld_wait();
                    if (q + 1 == kHD / 32) {
                        tc_fence_before();
                        mbar_arrive(&B.o_free[z]);
                    }
                    if (write) {
#pragma unroll
                        for (int c = 0; c < 4; ++c) store_256(o + q * 32 + 8 * c, u + 8 * c);
                    }
                }
            }
            if (!two) z0 ^= 1;
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// ---------------------------------------------------------------- own keys

// Lane i looks up page i of a batch of 32, from `first` on, of a range that ends at `end`:
// its segment b Hkv + h, its row in the pool, how many of its tokens are keys (0: its
// block is not there), and, as 32, whether its segment or the range ends.
struct OwnPage {
    int seg, row, info;
    __device__ __forceinline__ OwnPage(const SharedArgs& a, const Plan& P, const int* lens, int first, int end)
        : seg(0), row(0), info(0)
    {
        const int r = first + (threadIdx.x & 31), hkv = a.d.hkv;
        if (r >= end) return;
        int b = 0;  // the last sequence with Hkv own[b] <= r
        for (int m = a.d.batch; m > 1;) {
            const int half = m >> 1;
            if (hkv * P.own[b + half] <= r) b += half;
            m -= half;
        }
        const int pages = P.own[b + 1] - P.own[b], in = r - hkv * P.own[b], h = in / pages, len = lens[b];
        const int left = pages - (in - h * pages);  // pages up to the segment's end
        const int tok = (pages_of(len) - left) * kPage;
        const int32_t blk = a.d.block_table[(int64_t)b * a.d.max_blocks + tok / a.d.block_size];
        seg = b * hkv + h;
        info = left == 1 || r + 1 == end ? 32 : 0;
        if (blk < 0 || blk >= a.d.num_blocks) {
            record_error(a.d.status, KVATTN_ERR_BAD_INDEX);
        } else {
            row = (int)(((int64_t)blk * hkv + h) * a.d.block_size) + tok % a.d.block_size;
            info |= min(kPage, len - tok);
        }
    }
};
__device__ __forceinline__ uint32_t seen_of(int info) { return (1u << (info & 31)) - 1u; }

// Range `c` of the own pages, begin .. end - 1, by this warp.
template <int kHD>
__device__ __forceinline__ void own_warp(const SharedArgs& a, const Plan& P, const int* lens, int c, int begin, int end, int lg)
{
    const int lane = threadIdx.x & 31, g4 = lane >> 2, q4 = lane & 3;
    const int G = 1 << lg, n = end - begin;
    OwnPage page(a, P, lens, begin, end);
    // the group's queries as B fragments: head g4, the dims in the order of K's chunks
    uint32_t q[kHD / 16][2], qn[kHD / 16][2];
    auto load_q = [&](int seg) {
        const __nv_bfloat16* qh = reinterpret_cast<const __nv_bfloat16*>(a.d.q) + (((int64_t)seg << lg) + g4) * kHD;
#pragma unroll
        for (int i = 0; i < kHD / 32; ++i) {
            const uint4 w = g4 < G ? ldg16(qh + 8 * (q4 + 4 * i)) : make_uint4(0, 0, 0, 0);
            qn[2 * i][0] = w.x;
            qn[2 * i][1] = w.y;
            qn[2 * i + 1][0] = w.z;
            qn[2 * i + 1][1] = w.w;
        }
    };
    const char *kp = (const char*)a.d.k_pool, *vp = (const char*)a.d.v_pool;
    Bf16Tile<kHD> t;
    uint4 v[2][4][kHD / 64];
    int seg = __shfl_sync(0xffffffffu, page.seg, 0), info = __shfl_sync(0xffffffffu, page.info, 0);
    auto load = [&](int j, uint4 (&vv)[4][kHD / 64]) {
        const int64_t row = __shfl_sync(0xffffffffu, page.row, j & 31);
        t.load_k(kp + row * (kHD * 2), seen_of(info), g4, q4);
        t.load_v(vv, vp + row * (kHD * 2), seen_of(info), g4, q4);
    };
    // Page j on its way to L2, if it is of the looked up batch: a page is loaded one page's
    // time ahead, less than memory takes while all SMs read.  (One, two, three, five pages before
    // its load: 114, 120, 124, 137 us for 64 sequences of up to 4096 own tokens, without 134.)
    auto prefetch = [&](int j) {
        if ((j & 31) < kOwnAhead || j >= n) return;
        const int64_t row = __shfl_sync(0xffffffffu, page.row, j & 31);
        constexpr int kLines = kPage * kHD * 2 / 128;
#pragma unroll
        for (int i = 0; i < 2 * kLines / 32; ++i) {
            const int line = lane + 32 * i;
            const char* at = (line < kLines ? kp : vp) + row * (kHD * 2) + line % kLines * 128;
            asm volatile("prefetch.global.L2 [%0];" ::"l"(at));
        }
    };
    load(0, v[0]);
    load_q(seg);
    prefetch(kOwnAhead);
    Softmax st;
    float o[kHD / 16][4];
    bool fresh = true;
    auto step = [&](int j, const uint4 (&vnow)[4][kHD / 64], uint4 (&vnext)[4][kHD / 64]) {
        if (fresh) {
#pragma unroll
            for (int i = 0; i < kHD / 16; ++i) {
                q[i][0] = qn[i][0];
                q[i][1] = qn[i][1];
                o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
            }
            st.init();
        }
        float s[4] = {0.f, 0.f, 0.f, 0.f};
        t.scores(s, q);
        // the next page flies during this page's softmax and P.V, and so do the next
        // segment's queries
        const uint32_t now = seen_of(info);
        const int seg_now = seg;
        fresh = info & 32;
        if (j + 1 < n) {
            if (((j + 1) & 31) == 0) page = OwnPage(a, P, lens, begin + j + 1, end);
            seg = __shfl_sync(0xffffffffu, page.seg, (j + 1) & 31);
            info = __shfl_sync(0xffffffffu, page.info, (j + 1) & 31);
            load(j + 1, vnext);
            prefetch(j + 1 + kOwnAhead);
            if (fresh) load_q(seg);
        }
        const float sl2 = a.d.scale_log2;
        const float x[4] = {now >> g4 & 1u ? s[0] * sl2 : -INFINITY, now >> g4 & 1u ? s[1] * sl2 : -INFINITY,
                            now >> (g4 + 8) & 1u ? s[2] * sl2 : -INFINITY,
                            now >> (g4 + 8) & 1u ? s[3] * sl2 : -INFINITY};
        float p[4];
        st.step(x, o, p);
        // P in bf16, the type of V that the MMA takes it with: off by at most 2^-8 relative,
        // at random; the sum adds the fp32 p
        t.add(vnow, o, movmatrix_trans(pack_bf16_rn(p[0], p[1])), movmatrix_trans(pack_bf16_rn(p[2], p[3])));
        if (fresh) {  // the segment's end, or the range's: its state
#pragma unroll
            for (int i = 4; i < 32; i <<= 1) {
                st.l[0] += __shfl_xor_sync(0xffffffffu, st.l[0], i);
                st.l[1] += __shfl_xor_sync(0xffffffffu, st.l[1], i);
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int g = 2 * q4 + e;
                if (g >= G) continue;
                const int64_t row = (((int64_t)c + seg_now) << lg) + g;
                float* out = a.own_o + row * kHD;
                // the lane's dims dim_of(i, half) are neighbours in i
#pragma unroll
                for (int half = 0; half < 2; ++half)
#pragma unroll
                    for (int i = 0; i < kHD / 16; i += 4)
                        *reinterpret_cast<float4*>(out + Bf16Tile<kHD>::dim_of(i, half, g4)) =
                            make_float4(o[i][2 * half + e], o[i + 1][2 * half + e], o[i + 2][2 * half + e],
                                        o[i + 3][2 * half + e]);
                if (g4 == 0) *reinterpret_cast<float2*>(a.own_ml + row * 2) = make_float2(st.m[e], st.l[e]);
            }
        }
    };
    for (int j = 0; j < n; j += 2) {
        step(j, v[0], v[1]);
        if (j + 1 < n) step(j + 1, v[1], v[0]);
    }
}

// ... of fp8 pages, through two places of `ring` (fp8_tile.cuh has the fragments).
__device__ __forceinline__ void own_warp_fp8(const SharedArgs& a, const Plan& P, const int* lens, int c, int begin, int end,
                                             int lg, unsigned char* ring)
{
    constexpr int kRing = 2;
    const int lane = threadIdx.x & 31, g4 = lane >> 2, q4 = lane & 3;
    const int rk0 = (g4 >> 1) * 4 + (g4 & 1), rk1 = rk0 + 2;
    const int G = 1 << lg, n = end - begin;
    OwnPage now(a, P, lens, begin, end), next(a, P, lens, begin + 32, end);  // batches `batch` and the one after
    int batch = 0;
    auto seg_of = [&](int j) { return __shfl_sync(0xffffffffu, j >> 5 == batch ? now.seg : next.seg, j & 31); };
    auto info_of = [&](int j) { return __shfl_sync(0xffffffffu, j >> 5 == batch ? now.info : next.info, j & 31); };
    auto row_of = [&](int j) { return __shfl_sync(0xffffffffu, j >> 5 == batch ? now.row : next.row, j & 31); };
    auto fetch = [&](int j) {  // page j on its way to its place: one group of copies, empty past the end
        if (j < n) {
            const unsigned char* src = (const unsigned char*)a.d.k_pool + (int64_t)(row_of(j) / kPage) * kF8Page + 16 * lane;
            const uint32_t dst = smem_addr(ring + j % kRing * kF8Page + 16 * lane);
            auto copy = [](uint32_t to, const void* from) {
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
            };
#pragma unroll
            for (int i = 0; i < kF8Page / 512; ++i) copy(dst + 512 * i, src + 512 * i);
            if (lane < kF8Page % 512 / 16) copy(dst + kF8Page / 512 * 512, src + kF8Page / 512 * 512);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll
    for (int j = 0; j < kRing; ++j) fetch(j);
    uint32_t q[8][2];
    uint4 qn[4];  // the next segment's queries, as they are
    auto load_q = [&](int seg) {
        const __nv_bfloat16* qh = reinterpret_cast<const __nv_bfloat16*>(a.d.q) + (((int64_t)seg << lg) + g4) * 128;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            qn[i] = g4 < G ? ldg16(qh + 16 * (q4 + 4 * (i >> 1)) + 8 * (i & 1)) : make_uint4(0, 0, 0, 0);
    };
    load_q(seg_of(0));
    Fp8Softmax st;
    float o[8][4];
    bool fresh = true;
    for (int j = 0; j < n; ++j) {
        if (j >> 5 != batch) {
            ++batch;
            now = next;
            next = OwnPage(a, P, lens, begin + 32 * (batch + 1), end);
        }
        if (fresh) {  // scaled by 2^-4 into f16's range (the scores are scaled back)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t u[4] = {qn[i].x, qn[i].y, qn[i].z, qn[i].w};
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    q[2 * i + (k >> 1)][k & 1] = pack_f16_rn(bf16lo(u[k]) * 0.0625f, bf16hi(u[k]) * 0.0625f);
            }
            st.init();
#pragma unroll
            for (int i = 0; i < 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
        }
        const int seg = seg_of(j), info = info_of(j);
        fresh = info & 32;
        if (fresh && j + 1 < n) load_q(seg_of(j + 1));
        asm volatile("cp.async.wait_group %0;" ::"n"(kRing - 1) : "memory");
        __syncwarp();  // every lane's copies of page j are there
        Fp8Tile t;
        t.load(ring + j % kRing * kF8Page, rk0, g4, q4);
        __syncwarp();  // and every lane has read it
        fetch(j + kRing);
        float s[4] = {0.f, 0.f, 0.f, 0.f};
        t.scores(s, q);
        const uint32_t seen = seen_of(info);
        const float sl2 = a.d.scale_log2 * 16.f, k0 = t.ks[0] * sl2, k1 = t.ks[1] * sl2;
        const bool in0 = seen >> rk0 & 1u, in1 = seen >> rk1 & 1u;
        float x[4] = {in0 ? s[0] * k0 : -INFINITY, in0 ? s[1] * k0 : -INFINITY, in1 ? s[2] * k1 : -INFINITY,
                            in1 ? s[3] * k1 : -INFINITY};
        const float sv0 = in0 ? t.vs[0] : 0.f, sv1 = in1 ? t.vs[1] : 0.f;
        uint32_t vmask = 0xffffffffu;  // the bytes of this lane's words whose tokens are seen
        if (seen != (1u << kPage) - 1u) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (!(seen >> (4 * q4 + i) & 1u)) vmask &= ~(0xffu << (8 * i));
        }
        float w[4];
        st.step(x, sv0, sv1, lane, [&](int i) { return t.v[i] & vmask; }, o, w);
        t.add(o, movmatrix_trans(pack_f16_rn(w[0], w[1])), movmatrix_trans(pack_f16_rn(w[2], w[3])), vmask);
        if (fresh) {  // the segment's end, or the range's: its state
#pragma unroll
            for (int i = 4; i < 32; i <<= 1) {
                st.l[0] += __shfl_xor_sync(0xffffffffu, st.l[0], i);
                st.l[1] += __shfl_xor_sync(0xffffffffu, st.l[1], i);
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int g = 2 * q4 + e;
                if (g >= G) continue;
                const int64_t row = (((int64_t)c + seg) << lg) + g;
                float* out = a.own_o + row * 128 + g4;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    out[16 * i] = o[i][e] * st.ref[e];
                    out[16 * i + 8] = o[i][2 + e] * st.ref[e];
                }
                if (g4 == 0) *reinterpret_cast<float2*>(a.own_ml + row * 2) = make_float2(st.m[e], st.l[e]);
            }
        }
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
}

template <int kHD, bool kF8>
__global__ void __launch_bounds__(kThreads, 1)
    decode_shared_kernel(const __grid_constant__ SharedArgs a, const __grid_constant__ Maps maps)
{
    pdl_wait();
    using GE = Geo<kHD, kF8>;
    extern __shared__ unsigned char smem_raw[];
    unsigned char* smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
    Plan& P = *reinterpret_cast<Plan*>(smem + GE::kOffPlan);
    const int lg = __ffs(a.d.hq / a.d.hkv) - 1;  // row r of a prefix piece: sequence r >> lg, head r & (G - 1)
    int* len = reinterpret_cast<int*>(smem);  // (where Q will be)
    make_plan(a, P, len, lg);
    const int shared = P.first[a.num_groups], own = a.d.hkv * P.own[a.d.batch];
    const Ranges ranges = ranges_of<kF8>(shared, P.two_rows, P.segments, own, a.d.hkv * a.d.batch, gridDim.x,
                                         kSetUpBytes / GE::kCost, kSegmentBytes / GE::kCost);
    // where the merge finds each sequence's partial results
    for (int b = (int)blockIdx.x + (int)gridDim.x * threadIdx.x; b < a.d.batch; b += (int)gridDim.x * kThreads) {
        SharedOf o{};
        o.per = ranges.per;
        o.own_per = ranges.own_per;
        o.own_first = a.d.hkv * P.own[b];
        o.own_pages = P.own[b + 1] - P.own[b];
        if (shared > 0 && b < P.cu[a.num_groups]) {
            const int g = group_of(P, a.num_groups, b), pages = P.tokens[g] / kPage;
            if (pages > 0 && len[b] >= P.tokens[g]) {
                const int seqs = P.cu[g + 1] - P.cu[g], r = (b - P.cu[g]) << lg;
                o.pages = pages;
                o.first = P.first[g] + r / kSharedRows * pages;
                o.head_pages = blocks_of(seqs, lg) * pages;
                o.row = P.rows[g] + r;
                o.head_rows = seqs << lg;
            }
        }
        a.of[b] = o;
    }
    if ((int)blockIdx.x < ranges.ctas) {
        const int r = min(shared, (int)blockIdx.x * ranges.per), end = min(shared, r + ranges.per);
        if (r < end) prefix_cta<kHD, kF8>(a, maps, P, Walk{r, end, 0}, lg, smem);
    } else {
        const int warp = threadIdx.x >> 5;
        constexpr int kWarps = own_warps<kF8>(), kFirst = kF8 ? 0 : 4;
        if constexpr (!kF8) {
            if (warp < kFirst || warp >= kFirst + kWarps) {
                setmaxnreg_dec<kRegsIdle>();
                return;
            }
            setmaxnreg_inc<kRegsOwn>();
        }
        const int c = ((int)blockIdx.x - ranges.ctas) * kWarps + warp - kFirst;
        const int r = min(own, c * ranges.own_per), end = min(own, r + ranges.own_per);
        if (r >= end) return;
        if constexpr (kF8) own_warp_fp8(a, P, len, c, r, end, lg, smem + GE::kOffRing + warp * 2 * kF8Page);
        else own_warp<kHD>(a, P, len, c, r, end, lg);
    }
}

// Merges the pieces of a row (sequence, query head): kWarps warps a row, each the pieces
// of every kWarps-th chunk of 4 (a lane's loads of their outputs and the maxima and sums are under
// way together), then the warps' states.
template <int kHD, int kWarps>
__global__ void __launch_bounds__(128) decode_shared_merge_kernel(const __grid_constant__ SharedArgs a)
{
    pdl_wait();
    constexpr int kV = kHD / 32, kChunk = 4;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, share = warp % kWarps;
    const int wid = blockIdx.x * (4 / kWarps) + warp / kWarps;
    if (kWarps < 4 && wid >= a.d.batch * a.d.hq) return;
    const int G = a.d.hq / a.d.hkv, b = wid / a.d.hq, qh = wid - b * a.d.hq, h = qh / G, g = qh - h * G;
    const SharedOf s = a.of[b];
    int np = 0, no = 0;
    int64_t shared0 = 0, own0 = 0;  // rows of the first pieces
    if (s.pages > 0) {
        const int first = s.first + h * s.head_pages, c = first / s.per;
        np = (first + s.pages - 1) / s.per - c + 1;
        shared0 = (int64_t)c * kSharedRows + s.row + h * s.head_rows + g;
    }
    if (s.own_pages > 0) {
        const int first = s.own_first + h * s.own_pages, c = first / s.own_per;
        no = (first + s.own_pages - 1) / s.own_per - c + 1;
        own0 = (int64_t)(c + b * a.d.hkv + h) * G + g;
    }
    float acc[kV] = {}, den = 0.f, top = -INFINITY;
    for (int c0 = share * kChunk; c0 < np + no; c0 += kWarps * kChunk) {
        auto row_of = [&](int c) { return c < np ? shared0 + (int64_t)c * kSharedRows : own0 + (int64_t)(c - np) * G; };
        float2 ml = make_float2(-INFINITY, 0.f);
        if (lane < kChunk && c0 + lane < np + no)
            ml = *reinterpret_cast<const float2*>((c0 + lane < np ? a.ml : a.own_ml) + row_of(c0 + lane) * 2);
        float o[kChunk][kV];
#pragma unroll
        for (int i = 0; i < kChunk; ++i) {
            if (c0 + i < np + no) {
                const float* p = (c0 + i < np ? a.o : a.own_o) + row_of(c0 + i) * kHD + kV * lane;
                if constexpr (kV == 4) *reinterpret_cast<float4*>(o[i]) = *reinterpret_cast<const float4*>(p);
                else *reinterpret_cast<float2*>(o[i]) = *reinterpret_cast<const float2*>(p);
            }
        }
        // (a piece's sum is 0 without a score above -infinity, NaN with NaN scores)
        float m = ml.y == 0.f ? -INFINITY : ml.x;
#pragma unroll
        for (int x = 1; x < kChunk; x <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, x));
        m = fmaxf(top, __shfl_sync(0xffffffffu, m, 0));
        const float f0 = den == 0.f ? 0.f : exp2f(top - m), w = ml.y == 0.f ? 0.f : exp2f(ml.x - m);
        top = m;
        float sum = ml.y == 0.f ? 0.f : w * ml.y;
#pragma unroll
        for (int x = 1; x < kChunk; x <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
        den = den * f0 + __shfl_sync(0xffffffffu, sum, 0);
#pragma unroll
        for (int k = 0; k < kV; ++k) acc[k] *= f0;
#pragma unroll
        for (int i = 0; i < kChunk; ++i) {
            const float wi = __shfl_sync(0xffffffffu, w, i);
            if (wi != 0.f) {
#pragma unroll
                for (int k = 0; k < kV; ++k) acc[k] += wi * o[i][k];
            }
        }
    }
    if constexpr (kWarps > 1) {
        __shared__ float part[kWarps][kHD], stat[kWarps][2];
#pragma unroll
        for (int k = 0; k < kV; ++k) part[warp][kV * lane + k] = acc[k];
        if (lane == 0) {
            stat[warp][0] = top;
            stat[warp][1] = den;
        }
        __syncthreads();
        if (warp > 0) return;
        float m = -INFINITY;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) m = fmaxf(m, stat[w][1] == 0.f ? -INFINITY : stat[w][0]);
        den = 0.f;
#pragma unroll
        for (int k = 0; k < kV; ++k) acc[k] = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            if (stat[w][1] == 0.f) continue;
            const float f = exp2f(stat[w][0] - m);
            den += f * stat[w][1];
#pragma unroll
            for (int k = 0; k < kV; ++k) acc[k] += f * part[w][kV * lane + k];
        }
    }
    const float inv = den == 0.f ? 0.f : 1.f / den;
    uint32_t* out = reinterpret_cast<uint32_t*>(a.d.out) + ((int64_t)wid * kHD + kV * lane) / 2;
    if constexpr (kV == 4)
        *reinterpret_cast<uint2*>(out) = make_uint2(pack_bf16_rn(acc[0] * inv, acc[1] * inv), pack_bf16_rn(acc[2] * inv, acc[3] * inv));
    else
        *out = pack_bf16_rn(acc[0] * inv, acc[1] * inv);
}

template <int kHD, bool kF8>
bool make_maps(const DecodeArgs& a, Maps& m)
{
    std::memset(&m, 0, sizeof(m));
    const cuuint32_t G = a.hq / a.hkv;
    const cuuint64_t dims[3] = {(cuuint64_t)kHD, (cuuint64_t)a.hq, (cuuint64_t)a.batch};
    const cuuint64_t strides[2] = {(cuuint64_t)kHD * 2, (cuuint64_t)a.hq * kHD * 2};
    const cuuint32_t qbox[3] = {64, G, (cuuint32_t)kBM / G};
    if (!encode(&m.q, a.q, 3, dims, strides, qbox)) return false;
    const int64_t rows = (int64_t)a.num_blocks * a.hkv * a.block_size;
    if constexpr (kF8) return true;  // (pages are copied whole)
    else if constexpr (kHD == 128) return pool_maps(a.k_pool, a.v_pool, rows, false, &m.k, &m.v);
    // (64 columns, rows): a box of (64, 16) is one 16-row page, [16 rows][128 B]
    const cuuint64_t pdims[2] = {64, (cuuint64_t)rows};
    const cuuint64_t pstrides[1] = {64 * 2};
    const cuuint32_t pbox[2] = {64, 16};
    return encode(&m.k, a.k_pool, 2, pdims, pstrides, pbox) && encode(&m.v, a.v_pool, 2, pdims, pstrides, pbox);
}

template <int kHD, bool kF8>
kvattn_status launch(const SharedArgs& a, cudaStream_t s)
{
    Maps maps;
    if (!make_maps<kHD, kF8>(a.d, maps)) return KVATTN_ERR_CUDA;
    constexpr int kSmem = Geo<kHD, kF8>::kSmemBytes;
    static_assert(kSmem <= 232448, "shared memory of a block");
    static SmemLimit limit;
    if (limit.ensure(reinterpret_cast<const void*>(decode_shared_kernel<kHD, kF8>), kSmem) != cudaSuccess) return KVATTN_ERR_CUDA;
    const cudaError_t e = launch_pdl(decode_shared_kernel<kHD, kF8>, dim3((unsigned)num_sms()), dim3(kThreads), kSmem, s, a, maps);
    if (e != cudaSuccess) return KVATTN_ERR_CUDA;
    const int rows = a.d.batch * a.d.hq;
    // four warps a row where that leaves the GPU's warps room (rows 512, 1024, 2048 and 6144: 4.6, 5.8,
    // 6.4 and 14.3 us with four, 7.2, 7.9, 4.5 and 6.2 with one)
    return cuda_status(rows <= 1024 ? launch_pdl(decode_shared_merge_kernel<kHD, 4>, dim3((unsigned)rows), dim3(128), 0, s, a)
                                    : launch_pdl(decode_shared_merge_kernel<kHD, 1>, dim3((unsigned)((rows + 3) / 4)),
                                                 dim3(128), 0, s, a));
}

}  // namespace

kvattn_status launch_decode_shared(const SharedArgs& a, cudaStream_t s)
{
    if (a.d.fp8) return a.d.d == 128 ? launch<128, true>(a, s) : KVATTN_ERR_UNSUPPORTED;
    return a.d.d == 128 ? launch<128, false>(a, s) : a.d.d == 64 ? launch<64, false>(a, s) : KVATTN_ERR_UNSUPPORTED;
}

}  // namespace kvattn
