// Decode attention over the prefixes that groups of sequences share, on the
// tcgen05 tensor cores: a prefix is read once for all the queries of its group.
//
// What it computes: for a group of sequences whose first S tokens are the same
// (S rounded down to whole 16-token pages), and every query head j of every
// sequence b of it, the partial softmax state
//     m = max_{i < S} s_i,  l = sum_i 2^(s_i - m),  O = sum_i 2^(s_i - m) V[i],
//     s_i = q[b][j] . K[i][j / G] * scale * log2(e)
// in pieces over ranges of keys ("From-scratch AI inference engine" page, section
// 3.4: states over parts of the keys merge by their maxima and sums;
// "Nano-vLLM Part 2" page, section 05: sequences with a common prefix share its
// blocks).  decode_own.cu then does each sequence's other keys and the merge.
//
// What bounds it.  A KV head's queries are (sequences of the group) x G rows of one
// matrix product, so the prefix's K and V are read once, 4 D e bytes a key and KV
// head, for 4 D FLOPs a key and row: up to about 128 rows HBM has the longer
// part, from 256 rows on the tensor cores and the softmax beside them.
//
// How.  Rows come in blocks of 256 / G sequences.  The (row block, KV head) segments'
// tiles of 128 keys form one stream that is cut into equal ranges, one per SM
// (persistent CTAs), segments being cut where ranges meet.  A piece of more than
// 128 rows works on two row tiles A and B in turn over the same K and V tiles;
// one of up to 128 rows has A and B over the even and the odd key tiles, with states of
// their own that the output warps merge.  Either way the softmax of one runs beside the
// products of the other.  A row sees every key of the prefix (shorter sequences
// take no part), so only a prefix's last tile is masked, beyond its whole pages.
//
// Roles (four warpgroups): warp 0 copies K and Q tiles, warp 2 V tiles (a page a
// lane, straight from the block table); warp 1 issues the MMAs in the order PV_A(t)
// S_A(t+1) PV_B(t) S_B(t+1), from piece to piece without a gap; warps 4-11 the
// softmax (columns 0-63 and 64-127), P overwriting the first half of S in
// TMEM; warps 12-15 the outputs.  TMEM: S_A, S_B, O_A, O_B, 128 columns each.
// Every wait on a barrier is bounded: a timeout records KVATTN_ERR_TIMEOUT, the
// roles stop waiting, drain their copies and MMAs, free TMEM and return.
#include <algorithm>
#include <climits>
#include <cstring>

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
constexpr int kMinPer = 2;     // fewest tiles of a CTA's range
static_assert(kPrefixRows == 2 * kBM, "a piece's rows");
static_assert(kMaxGroups <= kThreads, "a thread per group");
// Registers per thread of the warpgroups (the block starts with 128 each:
// 96 + 2 x 168 + 80 = 4 x 128).
constexpr int kRegsIssue = 96, kRegsSoftmax = 168, kRegsOutput = 80;

// Barriers, in shared memory.
struct Bars {
    uint64_t q_full[kStages], q_empty[kStages];  // of a Q tile: loaded; every S MMA that reads it is done
    uint64_t k_full[kStages], k_empty[kStages], v_full[kStages], v_empty[kStages];
    uint64_t s_full[2], p_full[2];
    uint64_t o_done[2], o_free[2];   // the piece's last P.V into O_x has completed; O_x has been read
    uint64_t l_full[2];              // maxima and row sums of the even and of the odd pieces
    uint64_t drain;
    uint32_t tmem;
    int abort_flag;
};

// The groups of the call, and the stream of their tiles (group g: tiles first[g] ..
// first[g+1] - 1, segments segment[g] .., KV heads outermost, then row blocks).
struct Groups {
    int cu[kMaxGroups + 1];
    int tokens[kMaxGroups];   // shared, whole pages; 0: shares nothing
    int leader[kMaxGroups];   // a sequence of the group that has them
    int members[kMaxGroups];  // how many have them
    int first[kMaxGroups + 1], segment[kMaxGroups + 1];
    int sums[2][kThreads / 32];
};

template <int kD>
struct Geo {
    static constexpr int kPanels = kD / 64;
    static constexpr int kTileBytes = kBM * kD * 2;    // a Q tile, a K stage or a V stage
    static constexpr int kGroup = 8 * kD * 2;          // one 8-key group of a stage (all panels)
    static constexpr int kPageBytes = kPage * kD * 2;  // one page of K or V
    static constexpr int kOffQ = 0;
    static constexpr int kOffK = kStages * kTileBytes;
    static constexpr int kOffV = kOffK + kStages * kTileBytes;
    static constexpr int kOffBar = kOffV + kStages * kTileBytes;
    // fp32: row maxima of a tile [2][2 halves][128]; of two pieces, row sums [2][2 halves][2][128] and maxima [2][2][128]
    static constexpr int kOffX = kOffBar + 256;
    static constexpr int kOffGroups = kOffX + 8192;
    static constexpr int kSmemBytes = kOffGroups + (int)sizeof(Groups) + 1024;  // + slack to align the base to 1 KB
    static_assert(kD == 64 || kD == 128, "head dim");
};
static_assert(sizeof(Bars) <= 256, "the barriers fit before the exchange area");

struct Maps {
    CUtensorMap q;  // 3-D: (D, Hq, batch), box (64, G, 128 / G)
    CUtensorMap k;  // 4-D: (64 columns, 8 rows, 2 panels, rows / 8), box (64, 8, 2, 2); D = 64: 2-D, box (64, 16)
    CUtensorMap v;
};

// A piece: tiles t0 .. t1 - 1 of the `tokens` keys of the row `leader` of the table,
// for KV head h and `rows` rows: head r % G of sequence b0 + r / G.
struct Piece {
    int b0, rows, h, t0, t1, tokens, leader, id;
    __device__ __forceinline__ bool two() const { return rows > kBM; }
    // A's and B's tiles: the x-th's t-th is key tile t0 + (two ? t : 2 t + x)
    __device__ __forceinline__ int tiles(int x) const { return two() ? t1 - t0 : (t1 - t0 + 1 - x) >> 1; }
};

__device__ __forceinline__ bool len_ok(int L, const DecodeArgs& a)
{
    return L >= 0 && L <= a.max_seq_len && (int64_t)L <= (int64_t)a.max_blocks * a.block_size;
}

// Fills G from the call's arguments; every CTA does.  Groups that are out of order
// or out of range share nothing, nor does a group of which fewer than two sequences
// have the prefix.
__device__ __forceinline__ void plan_groups(const DecodeArgs& a, Groups& G, int lg)
{
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, n = a.num_groups;
    bool ok = true;
    if (tid < n) {
        const int c0 = a.cu_groups[tid], c1 = a.cu_groups[tid + 1], s = a.shared_lens[tid];
        ok = c0 >= 0 && c1 >= c0 && c1 <= a.batch && s >= 0 && s <= a.max_shared && (tid > 0 || c0 == 0) &&
             (int64_t)s <= (int64_t)a.max_blocks * a.block_size;
        G.cu[tid] = c0;
        if (tid == n - 1) G.cu[n] = c1;
        G.tokens[tid] = s & ~(kPage - 1);
        G.leader[tid] = INT_MAX;
        G.members[tid] = 0;
    }
    ok = __syncthreads_and(ok);
    if (!ok && blockIdx.x == 0 && tid == 0) record_error(a.status, KVATTN_ERR_BAD_INDEX);
    if (ok) {
        for (int b = tid; b < G.cu[n]; b += kThreads) {
            int g = 0;  // the last group with cu[g] <= b: the one b is in
            for (int m = n; m > 1;) {
                const int half = m >> 1;
                if (G.cu[g + half] <= b) g += half;
                m -= half;
            }
            const int L = a.seq_lens[b];
            if (len_ok(L, a) && L >= G.tokens[g]) {
                atomicMin(&G.leader[g], b);
                atomicAdd(&G.members[g], 1);
            }
        }
    }
    __syncthreads();
    int tiles = 0, segs = 0;
    if (tid < n) {
        if (!ok || G.members[tid] < 2) G.tokens[tid] = 0;
        if (G.tokens[tid] > 0) {
            const int seqs = G.cu[tid + 1] - G.cu[tid];
            segs = (((seqs << lg) + kPrefixRows - 1) / kPrefixRows) * a.hkv;
            tiles = segs * ((G.tokens[tid] + kBN - 1) / kBN);
        }
    }
    int ti = tiles, si = segs;  // up to this lane's
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, ti, o), y = __shfl_up_sync(0xffffffffu, si, o);
        if (lane >= o) {
            ti += x;
            si += y;
        }
    }
    if (lane == 31) {
        G.sums[0][warp] = ti;
        G.sums[1][warp] = si;
    }
    __syncthreads();
    for (int w = 0; w < warp; ++w) {
        ti += G.sums[0][w];
        si += G.sums[1][w];
    }
    if (tid < n) {
        G.first[tid + 1] = ti;
        G.segment[tid + 1] = si;
    }
    if (tid == 0) G.first[0] = G.segment[0] = 0;
    __syncthreads();
}

template <int kHD>
__global__ void __launch_bounds__(kThreads, 1)
    decode_prefix_kernel(const __grid_constant__ DecodeArgs a, const __grid_constant__ Maps maps)
{
    pdl_wait();
    using GE = Geo<kHD>;
    constexpr int kTileBytes = GE::kTileBytes, kPageBytes = GE::kPageBytes, kGroup = GE::kGroup;
    constexpr int kOffQ = GE::kOffQ, kOffK = GE::kOffK, kOffV = GE::kOffV;
    extern __shared__ unsigned char smem_raw[];
    unsigned char* smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
    Bars& B = *reinterpret_cast<Bars*>(smem + GE::kOffBar);
    Groups& G = *reinterpret_cast<Groups*>(smem + GE::kOffGroups);
    volatile int* abort_flag = &B.abort_flag;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int lg = __ffs(a.hq / a.hkv) - 1;  // row r of a piece: sequence r >> lg, head r & (G - 1)
    plan_groups(a, G, lg);
    const int total = G.first[a.num_groups];
    const int per = max((total + (int)gridDim.x - 1) / (int)gridDim.x, kMinPer);
    // where the merge finds each sequence's partial results
    for (int b = (int)blockIdx.x * kThreads + threadIdx.x; b < a.batch; b += (int)gridDim.x * kThreads) {
        PrefixOf p{0, 0, 0, 0, 0, 0, 0, per};
        int g = 0;
        for (int m = a.num_groups; m > 1;) {
            const int half = m >> 1;
            if (G.cu[g + half] <= b) g += half;
            m -= half;
        }
        const int L = a.seq_lens[b];
        if (total > 0 && b < G.cu[a.num_groups] && G.tokens[g] > 0 && len_ok(L, a) && L >= G.tokens[g]) {
            const int seqs = G.cu[g + 1] - G.cu[g], blocks = ((seqs << lg) + kPrefixRows - 1) / kPrefixRows;
            const int r = (b - G.cu[g]) << lg, rb = r / kPrefixRows;
            p.tokens = G.tokens[g];
            p.tiles = (p.tokens + kBN - 1) / kBN;
            p.first = G.first[g] + rb * p.tiles;
            p.head_tiles = blocks * p.tiles;
            p.segment = G.segment[g] + rb;
            p.head_segments = blocks;
            p.row = r - rb * kPrefixRows;
        }
        a.prefix[b] = p;
    }
    const int r_begin = min(total, (int)blockIdx.x * per), r_end = min(total, r_begin + per);
    if (r_begin >= r_end) return;

    if (threadIdx.x == 0) {
        for (int x = 0; x < 2; ++x) {
            mbar_init(&B.q_full[x], 1);
            mbar_init(&B.q_empty[x], 1);
            mbar_init(&B.k_full[x], 1);
            mbar_init(&B.k_empty[x], 1);
            mbar_init(&B.v_full[x], 1);
            mbar_init(&B.v_empty[x], 1);
            mbar_init(&B.s_full[x], 1);
            mbar_init(&B.p_full[x], 256);
            mbar_init(&B.o_done[x], 1);
            mbar_init(&B.o_free[x], 128);
            mbar_init(&B.l_full[x], 256);
        }
        mbar_init(&B.drain, 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 1) tmem_alloc(&B.tmem, 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = B.tmem;  // S_A at +0, S_B at +128, O_A at +256, O_B at +384

    // Walks this CTA's pieces.
    struct Walk {
        int r, g;
    };
    const Walk walk0{r_begin, 0};
    auto next_piece = [&](Walk& w, Piece& p) -> bool {
        if (w.r >= r_end) return false;
        while (G.first[w.g + 1] <= w.r) ++w.g;
        p.tokens = G.tokens[w.g];
        p.leader = G.leader[w.g];
        const int tiles = (p.tokens + kBN - 1) / kBN, seqs = G.cu[w.g + 1] - G.cu[w.g];
        const int blocks = ((seqs << lg) + kPrefixRows - 1) / kPrefixRows;
        const int off = w.r - G.first[w.g], seg = off / tiles;
        p.t0 = off - seg * tiles;
        p.t1 = min(tiles, p.t0 + r_end - w.r);
        p.h = seg / blocks;
        const int rb = seg - p.h * blocks;
        p.b0 = G.cu[w.g] + rb * (kPrefixRows >> lg);
        p.rows = min(kPrefixRows, (seqs << lg) - rb * kPrefixRows);
        p.id = (int)blockIdx.x + G.segment[w.g] + seg;
        w.r += p.t1 - p.t0;
        return true;
    };

    if (warp < 4) {
        setmaxnreg_dec<kRegsIssue>();
        if (warp == 0 || warp == 2) {
            // ====================== TMA producers: K and Q, V ======================
            const uint64_t pol = l2_evict_normal_policy();
            const bool is_k = warp == 0;
            if (lane == 0) {
                if (is_k) tma_prefetch_map(&maps.q);
                tma_prefetch_map(is_k ? &maps.k : &maps.v);
            }
            bool go = true;
            // lane 0 waits for `empty` (unless the buffer is new) and arms `full`
            auto arm = [&](uint64_t* full, uint64_t* empty, int use, uint32_t bytes) -> bool {
                if (lane == 0) {
                    go = use == 0 ? !*abort_flag : wait_or_abort(empty, (use - 1) & 1, abort_flag, a.status);
                    if (go) mbar_arrive_expect_tx(full, bytes);
                }
                return go = __shfl_sync(0xffffffffu, go, 0);
            };
            // Lane p < 8 copies page p of a tile; its block's id comes from the table a
            // tile ahead (lanes without a page read their row's first entry).
            auto has_page = [&](const Piece& p, int t) { return lane < kPages && t * kBN + lane * kPage < p.tokens; };
            auto block_id = [&](const Piece& p, int t) -> int32_t {
                const int col = has_page(p, t) ? (t * kBN + lane * kPage) / a.block_size : 0;
                return a.block_table[(int64_t)p.leader * a.max_blocks + col];
            };
            auto page_row = [&](const Piece& p, int t, int32_t blk) -> int {
                if (!has_page(p, t)) return -1;
                if (blk < 0 || blk >= a.num_blocks) {
                    if (is_k) record_error(a.status, KVATTN_ERR_BAD_INDEX);
                    return -1;
                }
                return (int)(((int64_t)blk * a.hkv + p.h) * a.block_size) + (t * kBN + lane * kPage) % a.block_size;
            };
            int g = 0, qg = 0;  // K (or V) and Q tiles armed so far
            Walk w = walk0;
            Piece p, ahead;
            bool more = next_piece(w, ahead);
            int32_t blk_next = block_id(ahead, ahead.t0);
            while (go && more) {
                p = ahead;
                for (int t = p.t0; t < p.t1; ++t) {
                    const int row = page_row(p, t, blk_next);
                    const uint32_t bytes = (uint32_t)__popc(__ballot_sync(0xffffffffu, row >= 0)) * (uint32_t)kPageBytes;
                    const int s = g % kStages;
                    if (!arm(is_k ? &B.k_full[s] : &B.v_full[s], is_k ? &B.k_empty[s] : &B.v_empty[s], g / kStages, bytes)) break;
                    if (row >= 0) {
                        unsigned char* dst = smem + (is_k ? kOffK : kOffV) + s * kTileBytes + lane * kPageBytes;
                        const CUtensorMap* m = is_k ? &maps.k : &maps.v;
                        uint64_t* full = is_k ? &B.k_full[s] : &B.v_full[s];
                        if constexpr (kHD == 128) tma_load_4d(dst, m, 0, 0, 0, row >> 3, full, pol);
                        else tma_load_2d(dst, m, 0, row, full, pol);
                    }
                    ++g;
                    const bool first = t == p.t0;
                    if (t + 1 == p.t1) {
                        more = next_piece(w, ahead);
                        if (more) blk_next = block_id(ahead, ahead.t0);
                    } else {
                        blk_next = block_id(p, t + 1);
                    }
                    if (is_k && first) {
                        for (int x = 0; x < (p.two() ? 2 : 1); ++x) {
                            const int qs = qg % kStages;
                            if (!arm(&B.q_full[qs], &B.q_empty[qs], qg / kStages, kTileBytes)) break;
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
                    mbar_wait(is_k ? &B.k_full[t % kStages] : &B.v_full[t % kStages], (t / kStages) & 1, a.status);
                for (int t = max(0, qg - kStages); t < qg; ++t) mbar_wait(&B.q_full[t % kStages], (t / kStages) & 1, a.status);
            }
        } else if (warp == 1) {
            // ============================== MMA issuer ==============================
            // The whole warp runs the schedule (waits agreed by the warp) and one
            // elected lane issues.  Operand descriptors are built once: a stage or
            // k-step only adds (byte offset >> 4) to the start-address field, which
            // cannot carry out of it (shared-memory offsets stay below 256 KB).
            constexpr uint32_t idesc_s = idesc_bf16_f32(kBM, kBN, false);
            constexpr uint32_t idesc_o = idesc_bf16_f32(kBM, kHD, true);
            const uint32_t sbase = smem_addr(smem);
            const uint64_t dQ = umma_desc_sw128(sbase + kOffQ, 16, 1024);
            const uint64_t dK = umma_desc_sw128(sbase + kOffK, 16, kGroup);
            const uint64_t dV = umma_desc_sw128(sbase + kOffV, 1024, kGroup);
            constexpr uint64_t kTileStep = kTileBytes >> 4;
            auto wait = [&](uint64_t* b, uint32_t parity) {
                if (__all_sync(0xffffffffu, mbar_try_wait(b, parity))) return true;
                return warp_wait(b, parity, abort_flag, a.status);
            };
            int kb = 0, vb = 0, qb = 0;      // K, V and Q tiles of the pieces before
            uint32_t steps[2] = {0, 0};      // P_x that have been read so far
            uint32_t pieces[2] = {0, 0};     // pieces with an O_x before this one
            // S_x of the t-th tile of A or B.  The K stage is free after the last S that
            // reads it, the Q tile after the piece's last.
            auto do_s = [&](const Piece& p, int x, int t) -> bool {
                const bool two = p.two();
                const int kt = two ? t : 2 * t + x, k = kb + kt, q = qb + (two ? x : 0), n = p.t1 - p.t0;
                if (t == 0 && !wait(&B.q_full[q % kStages], (q / kStages) & 1)) return false;
                if (!wait(&B.k_full[k % kStages], (k / kStages) & 1)) return false;
                tc_fence_after();
                if (elect_one()) {
                    const uint64_t qd = dQ + (q % kStages) * kTileStep, kd = dK + (k % kStages) * kTileStep;
                    const uint32_t d = tmem + x * 128;
#pragma unroll
                    for (int i = 0; i < kHD / 16; ++i)  // k-step: 16 columns, 32 B inside the 128-byte atom
                        tc_mma_f16(d, qd + (uint64_t)(((i >> 2) * kPanel + (i & 3) * 32) >> 4),
                                   kd + (uint64_t)(((i >> 2) * 1024 + (i & 3) * 32) >> 4), idesc_s, i > 0);
                    tc_commit(&B.s_full[x]);
                    if (!two || x == 1) tc_commit(&B.k_empty[k % kStages]);
                    if (kt == n - 1) tc_commit(&B.q_empty[q % kStages]);
                }
                __syncwarp();
                return true;
            };
            // O_x += P_x V, P_x in S_x's first 64 columns, over the tile's whole pages; a
            // piece's first overwrites O_x (o_free: the piece before has been read)
            auto do_pv = [&](const Piece& p, int x, int t) -> bool {
                const bool two = p.two();
                const int kt = two ? t : 2 * t + x, v = vb + kt;
                if (!wait(&B.v_full[v % kStages], (v / kStages) & 1) || !wait(&B.p_full[x], steps[x] & 1)) return false;
                ++steps[x];
                if (t == 0) {
                    if (pieces[x] > 0 && !wait(&B.o_free[x], (pieces[x] - 1) & 1)) return false;
                    ++pieces[x];
                }
                tc_fence_after();
                if (elect_one()) {
                    const uint64_t vd = dV + (v % kStages) * kTileStep;
                    const uint32_t d = tmem + 256 + x * 128, pa = tmem + x * 128;
                    const int pages = min(kPages, (p.tokens - (p.t0 + kt) * kBN) / kPage);
#pragma unroll
                    for (int i = 0; i < kPages; ++i)  // k-step: 16 keys = two 8-key groups
                        if (i < pages)
                            tc_mma_f16_ts(d, pa + i * 8, vd + (uint64_t)((i * 2 * kGroup) >> 4), idesc_o, (t > 0 || i > 0));
                    if (!two || x == 1) tc_commit(&B.v_empty[v % kStages]);
                    if (t + 1 == p.tiles(x)) tc_commit(&B.o_done[x]);
                }
                __syncwarp();
                return true;
            };
            // Order per t: PV_A(t) S_A(t+1) PV_B(t) S_B(t+1); S_x(t+1) overwrites S_x's
            // columns after PV_x(t) has read P_x(t) from them (tensor operations of
            // one thread run in issue order).
            Walk w = walk0;
            Piece p, next;
            bool more = next_piece(w, p);
            bool ok = do_s(p, 0, 0) && (p.tiles(1) == 0 || do_s(p, 1, 0));
            while (ok && more) {
                const int n0 = p.tiles(0), n1 = p.tiles(1);
                for (int t = 0; ok && t + 1 < n0; ++t) {
                    ok = do_pv(p, 0, t) && do_s(p, 0, t + 1) && do_pv(p, 1, t) && (t + 1 >= n1 || do_s(p, 1, t + 1));
                }
                if (!ok) break;
                // the piece's last, and the next piece's first S
                if (!(ok = do_pv(p, 0, n0 - 1))) break;
                more = next_piece(w, next);
                const int kb0 = kb, vb0 = vb, qb0 = qb;
                const int kb1 = kb + p.t1 - p.t0, qb1 = qb + (p.two() ? 2 : 1);
                if (more) {
                    kb = kb1;
                    qb = qb1;
                    ok = do_s(next, 0, 0);
                    kb = kb0;
                    qb = qb0;
                }
                if (ok && n1 == n0) ok = do_pv(p, 1, n1 - 1);
                kb = kb1;
                qb = qb1;
                vb = vb0 + p.t1 - p.t0;
                if (ok && more && next.tiles(1) > 0) ok = do_s(next, 1, 0);
                p = next;
            }
            // every MMA this warp issued has completed once `drain` flips
            if (elect_one()) tc_commit(&B.drain);
            __syncwarp();
            mbar_wait(&B.drain, 0, a.status);
        }
    } else if (warp < 12) {
        setmaxnreg_inc<kRegsSoftmax>();
        // ================================= softmax ==================================
        // All eight warps work on whichever S is due: thread (quarter, lane) owns row
        // r = 32 quarter + lane of the tile, warps 4-7 its columns 0..63 (half hf =
        // 0) and warps 8-11 its columns 64..127 (hf = 1).  The halves of a row agree on
        // the row max through shared memory, with a named barrier of that pair of
        // warps per tile.  These warps never stop early: after an abort their waits return
        // at once and they run on to the end (nothing of it is reported good).  One
        // body for A and B, whose states change places after each.
        const int hf = (warp - 4) >> 2;
        const int quarter = warp & 3;        // TMEM lanes 32*quarter .. +31
        const int r = quarter * 32 + lane;   // row of the tile
        const uint32_t lane_base = (uint32_t)(quarter * 32) << 16;
        float* xchg = reinterpret_cast<float*>(smem + GE::kOffX);
        const float sl2 = a.scale_log2;
        uint32_t steps = 0;  // bit x: parity of the S_x seen so far
        int ii = 0;
        Walk w = walk0;
        Piece p;
        while (next_piece(w, p)) {
            const bool two = p.two();
            const int n0 = p.tiles(0), n1 = p.tiles(1);
            float m_now = -INFINITY, l_now = 0.f, m_other = -INFINITY, l_other = 0.f;  // of A and B in turn
#pragma unroll 1
            for (int st = 0; st < n0 + n1; ++st) {
                const int t = st >> 1, x = st & 1;
                const uint32_t tS = tmem + lane_base + x * 128 + hf * 64;
                const uint32_t tO = tmem + lane_base + 256 + x * 128 + hf * (kHD / 2);
                const int keys = p.tokens - (p.t0 + (two ? t : st)) * kBN - hf * 64;  // of this half's columns
                wait_or_abort(&B.s_full[x], steps >> x & 1u, abort_flag, a.status);
                __syncwarp();
                steps ^= 1u << x;
                if ((two ? x * kBM : 0) + quarter * 32 < p.rows) {  // (P of other rows may be anything)
                    uint32_t sv[64];
                    tc_fence_after();
                    tmem_ld32(tS, *reinterpret_cast<uint32_t(*)[32]>(&sv[0]));
                    tmem_ld32(tS + 32, *reinterpret_cast<uint32_t(*)[32]>(&sv[32]));
                    tmem_ld_wait();
                    if (keys < 64) {
#pragma unroll
                        for (int e = 0; e < 64; ++e)
                            if (e >= keys) sv[e] = __float_as_uint(-INFINITY);
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
                    const bool rescale = !none && m_tile > m_now + 8.f;
                    const float m_new = none || rescale ? m_tile : m_now;
                    const float alpha = none ? 1.f : fast_exp2(m_now - m_new);
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
                        pw[e] = pack_bf16_rn(pk_lo(pp), pk_hi(pp));
                        sum2[e & 1] = fadd2(sum2[e & 1], pp);
                    }
                    tmem_st32(tmem + lane_base + x * 128 + hf * 32, pw);
                    l_now = l_now * alpha + ((pk_lo(sum2[0]) + pk_hi(sum2[0])) + (pk_lo(sum2[1]) + pk_hi(sum2[1])));
                    // O_x (this half's columns): PV_x(t-1) completed before S_x(t) was
                    // reported.  The whole warp rescales if any of its rows must (alpha
                    // is 1 for the others).
                    if (__any_sync(0xffffffffu, rescale && t > 0)) {
#pragma unroll 1
                        for (int q = 0; q < kHD / 64; ++q) {
                            uint32_t v[32];
                            tmem_ld32(tO + q * 32, v);
                            tmem_ld_wait();
#pragma unroll
                            for (int e = 0; e < 32; ++e) v[e] = __float_as_uint(__uint_as_float(v[e]) * alpha);
                            tmem_st32(tO + q * 32, v);
                        }
                    }
                    tmem_st_wait();
                    tc_fence_before();
                }
                mbar_arrive(&B.p_full[x]);
                const float m = m_now, l = l_now;
                m_now = m_other;
                l_now = l_other;
                m_other = m;
                l_other = l;
            }
            if ((n0 + n1) & 1) {  // A was last
                const float m = m_now, l = l_now;
                m_now = m_other;
                l_now = l_other;
                m_other = m;
                l_other = l;
            }
            // this piece's maxima and sums to the output warps (two pieces' worth: those of
            // piece ii - 2 were read before S_A of this piece was issued)
            float* lx = xchg + 512 + (ii & 1) * 512;  // [2 halves][2 tiles][128 rows]
            float* mx = xchg + 1536 + (ii & 1) * 256;
            lx[(hf * 2 + 0) * 128 + r] = l_now;
            lx[(hf * 2 + 1) * 128 + r] = l_other;
            if (hf == 0) {
                mx[r] = m_now;
                mx[128 + r] = m_other;
            }
            mbar_arrive(&B.l_full[ii & 1]);
            ++ii;
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
        uint32_t done[2] = {0, 0};  // pieces with an O_x so far
        int ii = 0;
        Walk w = walk0;
        Piece p;
        bool ok = true;
        while (ok && next_piece(w, p)) {
            const bool two = p.two();
            const int n1 = p.tiles(1);
            if (!long_wait(&B.l_full[ii & 1], (ii >> 1) & 1, p.t1 - p.t0, abort_flag, a.status)) break;
            const float* lx = xchg + 512 + (ii & 1) * 512;
            const float* mx = xchg + 1536 + (ii & 1) * 256;
            const float l0 = lx[r] + lx[256 + r], l1 = lx[128 + r] + lx[384 + r], m0 = mx[r], m1 = mx[128 + r];
            ++ii;
            const int64_t row0 = (int64_t)p.id * kPrefixRows + r;
            // 16 columns of O at a time into row `row`; merged: f0 O_A + f1 O_B
            auto put = [&](int64_t row, bool write, float m, float l) {
                if (write) *reinterpret_cast<float2*>(a.prefix_ml + row * 2) = make_float2(m, l);
            };
            if (two || n1 == 0) {
#pragma unroll 1
                for (int x = 0; x < (two ? 2 : 1); ++x) {
                    if (!(ok = warp_wait(&B.o_done[x], done[x] & 1, abort_flag, a.status))) break;
                    ++done[x];
                    tc_fence_after();
                    const bool write = x * kBM + r < p.rows;
                    put(row0 + x * kBM, write, x ? m1 : m0, x ? l1 : l0);
                    float* o = a.prefix_o + (row0 + x * kBM) * kHD;
#pragma unroll 1
                    for (int q = 0; q < kHD / 32; ++q) {
                        uint32_t v[32];
                        tmem_ld32(tO + x * 128 + q * 32, v);
                        tmem_ld_wait();
                        if (q + 1 == kHD / 32) {
                            tc_fence_before();
                            mbar_arrive(&B.o_free[x]);
                        }
                        if (write) {
#pragma unroll
                            for (int c = 0; c < 4; ++c) store_256(o + q * 32 + 8 * c, v + 8 * c);
                        }
                    }
                }
            } else {
                ok = warp_wait(&B.o_done[0], done[0] & 1, abort_flag, a.status) &&
                     warp_wait(&B.o_done[1], done[1] & 1, abort_flag, a.status);
                if (!ok) break;
                ++done[0];
                ++done[1];
                tc_fence_after();
                const bool write = r < p.rows;
                // (a sum of 0: no score above -infinity, no weight)
                const float m = fmaxf(l0 == 0.f ? -INFINITY : m0, l1 == 0.f ? -INFINITY : m1);
                const float f0 = l0 == 0.f ? 0.f : fast_exp2(m0 - m), f1 = l1 == 0.f ? 0.f : fast_exp2(m1 - m);
                put(row0, write, m, f0 * l0 + f1 * l1);
                float* o = a.prefix_o + row0 * kHD;
#pragma unroll 1
                for (int q = 0; q < kHD / 16; ++q) {
                    uint32_t u[16], v[16];
                    tmem_ld16(tO + q * 16, u);
                    tmem_ld16(tO + 128 + q * 16, v);
                    tmem_ld_wait();
                    if (q + 1 == kHD / 16) {
                        tc_fence_before();
                        mbar_arrive(&B.o_free[0]);
                        mbar_arrive(&B.o_free[1]);
                    }
                    if (write) {
#pragma unroll
                        for (int e = 0; e < 16; ++e)
                            u[e] = __float_as_uint(f0 * __uint_as_float(u[e]) + f1 * __uint_as_float(v[e]));
                        store_256(o + q * 16, u);
                        store_256(o + q * 16 + 8, u + 8);
                    }
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

template <int kHD>
bool make_maps(const DecodeArgs& a, Maps& m)
{
    std::memset(&m, 0, sizeof(m));
    const cuuint32_t G = a.hq / a.hkv;
    const cuuint64_t dims[3] = {(cuuint64_t)kHD, (cuuint64_t)a.hq, (cuuint64_t)a.batch};
    const cuuint64_t strides[2] = {(cuuint64_t)kHD * 2, (cuuint64_t)a.hq * kHD * 2};
    const cuuint32_t qbox[3] = {64, G, (cuuint32_t)kBM / G};
    if (!encode(&m.q, a.q, 3, dims, strides, qbox)) return false;
    const int64_t rows = (int64_t)a.num_blocks * a.hkv * a.block_size;
    if constexpr (kHD == 128) return pool_maps(a.k_pool, a.v_pool, rows, false, &m.k, &m.v);
    // (64 columns, rows): a box of (64, 16) is one 16-row page, [16 rows][128 B]
    const cuuint64_t pdims[2] = {64, (cuuint64_t)rows};
    const cuuint64_t pstrides[1] = {64 * 2};
    const cuuint32_t pbox[2] = {64, 16};
    return encode(&m.k, a.k_pool, 2, pdims, pstrides, pbox) && encode(&m.v, a.v_pool, 2, pdims, pstrides, pbox);
}

template <int kHD>
kvattn_status launch(const DecodeArgs& a, cudaStream_t s)
{
    Maps maps;
    if (!make_maps<kHD>(a, maps)) return KVATTN_ERR_CUDA;
    constexpr int kSmem = Geo<kHD>::kSmemBytes;
    static_assert(kSmem <= 232448, "shared memory of a block");
    static SmemLimit limit;
    if (limit.ensure(reinterpret_cast<const void*>(decode_prefix_kernel<kHD>), kSmem) != cudaSuccess) return KVATTN_ERR_CUDA;
    return cuda_status(launch_pdl(decode_prefix_kernel<kHD>, dim3((unsigned)num_sms()), dim3(kThreads), kSmem, s, a, maps));
}

}  // namespace

kvattn_status launch_decode_shared(const DecodeArgs& a, cudaStream_t s)
{
    return a.d == 128 ? launch<128>(a, s) : a.d == 64 ? launch<64>(a, s) : KVATTN_ERR_UNSUPPORTED;
}

}  // namespace kvattn
