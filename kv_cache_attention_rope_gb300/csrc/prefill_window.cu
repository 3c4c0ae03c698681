// Chunked-prefill attention with a sliding window and sink tokens on the
// tcgen05 tensor cores.
//
// What it computes: for chunk c with prefix P and query row r at position
// p = P + r,
//     out[r] = softmax_k(q[r] . K[k] * scale) V[k],  k <= p and (k > p - window or k < sinks)
// over the chunk's sequence in the paged cache, which already holds the
// chunk's own keys ("From-scratch AI inference engine" page, sections 3.3, the
// mask, and 3.4, the online softmax over key tiles).
//
// How: persistent CTAs, one per SM, over work items of one KV head and 256 / G
// tokens of a chunk: the G query heads of the KV head's group make them 256
// rows (row r: head r % G of token r / G), two 128-row tiles A and B that share
// one K/V stream.  With a window the keys that an item reads are window - 1 +
// its tokens, so few tokens of many heads read least: at a window of 1024 and
// G = 4, 64 tokens take 9 tiles of 128 keys for 8 tiles' worth of seen keys
// (256 tokens of one head: 11), and A and B see nearly the same columns.  16
// chunks of 512 queries: 152 us with items of one head, 125 us with the group.
//
// Columns.  An item's pages (16 keys) are its sink_pages first ones and those
// from the page of its first row's first window key on, `gap` pages apart;
// its tiles are cut from that list.  The row at position p then sits at column
// p' = p - 16 gap and sees the columns v <= p' with v > p' - window or v <
// sinks: with gap > 0 every column of the first part lies below the first
// row's window, and every column of the second is a key past the sinks.
//
// Roles (four warpgroups):
//  - warp 0: TMA copies of Q tiles and of 128-key K tiles, warp 2 of V tiles,
//    one 4 KB box per page, straight from the block table; warp 1: the MMAs, in
//    the order PV_A(t) S_A(t+1) PV_B(t) S_B(t+1), through the items without a
//    gap (tile t+1 of an item's last is the next item's first); warp 3: zeros in
//    V rows that no row sees;
//  - warps 4-7 and 8-11: the softmax of columns 0-63 and 64-127 of whichever
//    tile is due; P, in V's type (bf16, or f16 over an fp8 cache's copy),
//    overwrites the first half of S in TMEM;
//  - warps 12-15: O / row sums -> bf16 rows of out, while the others are at
//    the next item (and, over an fp8 cache's copy, q -> f16 as it arrives).
// TMEM: S_A, S_B, O_A, O_B, 128 columns each.  Every wait on a barrier is
// bounded (1 s, and more where many tiles go by meanwhile): a timeout records
// KVATTN_ERR_TIMEOUT, the roles stop waiting, drain their copies and MMAs, free TMEM
// and return.
#include <algorithm>
#include <cstring>
#include <mutex>

#include "tc_roles.cuh"

namespace kvattn {
namespace {

constexpr int kBM = 128;       // rows per tile (two tiles per item: A and B)
constexpr int kBN = 128;       // keys per KV tile
constexpr int kPage = 16;      // tokens per TMA copy of one block
constexpr int kThreads = 512;
constexpr int kStages = 2;     // of K and of V
constexpr int kPanel = kBM * 128;  // 16 KB: 128 rows x 64 columns (one 128-byte swizzle panel of Q)
constexpr int kMaxPairs = 512;     // more (chunk, token block) pairs than this are taken unsorted
constexpr int kMaxChunks = 4 * kMaxPairs - 1;  // of a launch: their pair counts fit where the sorted pairs go
// Registers per thread of the warpgroups (the block starts with 128 each:
// 96 + 2 x 168 + 80 = 4 x 128).
constexpr int kRegsIssue = 96, kRegsSoftmax = 168, kRegsOutput = 80;

// Shared-memory geometry for head dim kD (64 or 128): a row of Q, K or V is
// kD / 64 panels of 128 bytes; a K/V stage is [8-key group][panel][8 keys]
// [128 B], so a 16-token page is one contiguous block of the stage.
template <int kD>
struct Geo {
    static constexpr int kPanels = kD / 64;
    static constexpr int kTileBytes = kBM * kD * 2;    // a Q tile, a K stage or a V stage
    static constexpr int kGroup = 8 * kD * 2;          // one 8-key group of a stage (all panels)
    static constexpr int kPageBytes = kPage * kD * 2;  // one page of K or V
    static constexpr int kOffQ = 0;                    // Q_A, Q_B
    static constexpr int kOffK = 2 * kTileBytes;
    static constexpr int kOffV = kOffK + kStages * kTileBytes;
    static constexpr int kOffBar = kOffV + kStages * kTileBytes;
    static constexpr int kOffX = kOffBar + 256;        // fp32: row maxima [2][2][128], row sums of two items [2][2][2][128]
    static constexpr int kOffPairs = kOffX + 6144;     // sorted pairs (or `before`)
    static constexpr int kOffScratch = kOffPairs + kMaxPairs * 16;  // tiles per pair
    static constexpr int kSmemBytes = kOffScratch + kMaxPairs * 4 + 1024;  // + slack to align the base to 1 KB
    static_assert(kD == 64 || kD == 128, "head dim");
};

struct Maps {
    CUtensorMap q;  // 3-D: (D, Hq, total_q), box (64, G, 128 / G)
    CUtensorMap k;  // 4-D: (64 columns, 8 rows, 2 panels, rows / 8), box (64, 8, 2, 2); D = 64: 2-D, box (64, 16)
    CUtensorMap v;
};

// Barriers, in shared memory.
struct Bars {
    uint64_t q_full[2], q_empty[2];  // of Q_x: loaded; every S_x MMA of the item is done
    uint64_t q_f16[2];               // kF16: converted
    uint64_t k_full[kStages], k_empty[kStages], v_full[kStages], v_empty[kStages];
    uint64_t v_raw[kStages];         // V loaded, with rows to zero before it counts as v_full
    uint64_t s_full[2], p_full[2];
    uint64_t o_done[2], o_free[2];   // the item's last P.V into O_x has completed; O_x has been read
    uint64_t l_full[2];              // row sums of the even and of the odd items
    uint64_t drain;
    uint32_t tmem;
    int abort_flag;
};
static_assert(sizeof(Bars) <= 256, "the barriers fit before the exchange area");

// A token block of a chunk: rows (tokens) row0 .. row0 + rows - 1 of q, at
// positions pos0 ...
struct Pair {
    int row0, pos0, rows, c;
};

// Tokens of chunk c; metadata out of range gives none (recorded when `report`).
__device__ __forceinline__ int chunk_rows(const PrefillArgs& a, int c, bool report)
{
    const int q0 = a.cu_q_lens[c], qlen = a.cu_q_lens[c + 1] - q0, P = a.prefix_lens[c];
    if (qlen < 0 || P < 0 || qlen > a.max_q_len || q0 < 0 || (int64_t)q0 + qlen > a.total_q ||
        (int64_t)P + qlen > (int64_t)a.max_blocks * a.block_size ||
        (qlen > 0 && !window_keys_ok(P, qlen, a.window, a.sinks))) {
        if (report) record_error(a.status, KVATTN_ERR_BAD_INDEX);
        return 0;
    }
    return qlen;
}

// Pair i of a call: before[c] pairs belong to the chunks before chunk c.
__device__ __forceinline__ Pair make_pair(const PrefillArgs& a, const int* before, int step, int i)
{
    int c = 0;  // the last chunk with before[c] <= i: the one pair i is in
    for (int n = a.num_chunks; n > 1;) {
        const int half = n >> 1;
        if (before[c + half] <= i) c += half;
        n -= half;
    }
    const int first = (i - before[c]) * step;
    const int q0 = a.cu_q_lens[c];
    return {q0 + first, a.prefix_lens[c] + first, min(step, a.cu_q_lens[c + 1] - q0 - first), c};
}

struct Divisors {
    Divisor hkv, block_pages;  // KV heads; 16-token pages of a block
};

// The pages of a pair (see the top of the file) and its tiles.
struct Pages {
    int n, sink, gap, tiles;
};
__device__ __forceinline__ Pages pages_of(const PrefillArgs& a, const Pair& p)
{
    Pages g;
    const int all = (p.pos0 + p.rows - 1) / kPage + 1;
    g.sink = a.sinks > 0 ? min(all, (a.sinks - 1) / kPage + 1) : 0;
    g.gap = max(0, max(0, p.pos0 - a.window + 1) / kPage - g.sink);
    g.n = all - g.gap;
    g.tiles = (g.n + kBN / kPage - 1) / (kBN / kPage);
    return g;
}

// Columns of an item that no row of it sees: from `end` on, and sinks .. low.
struct Unseen {
    int end, low;
};
__device__ __forceinline__ Unseen unseen_of(const PrefillArgs& a, const Pair& p, const Pages& g)
{
    const int tok = p.pos0 - g.gap * kPage;  // column of the item's first token
    return {tok + p.rows, tok - a.window};
}
// Whether tile t has any.
__device__ __forceinline__ bool has_unseen(const PrefillArgs& a, const Unseen& u, int t)
{
    return (t + 1) * kBN > u.end || (t * kBN <= u.low && (t + 1) * kBN > a.sinks);
}

// Persistent CTAs.  Items are (pair, KV head), KV heads innermost, with up to
// kMaxPairs pairs in descending order of tiles (every CTA ranks them identically
// in shared memory; ties by index) and more in the order of their chunks.
// CTA k takes, in round r, item r G + k for even r and r G + G - 1 - k for odd r
// (G CTAs).  Pipeline state (stages, phases) runs on across items.
// kF16: K and V (and so q and P, which the MMAs take in their types) in f16,
// scaled per (chunk, KV head) as a.kv_scale says.  q arrives in bf16, and the
// output warps, which have time, convert it in place to q / 16 (f16's 11 bits
// hold bf16's 8; from 2^20 on it is infinite, and under 2^-10 it loses bits).
template <int kHD, bool kF16>
__global__ void __launch_bounds__(kThreads, 1)
    prefill_window_kernel(const __grid_constant__ PrefillArgs a, const __grid_constant__ Maps maps,
                          const __grid_constant__ Divisors div)
{
    pdl_wait();
    using GE = Geo<kHD>;
    constexpr int kTileBytes = GE::kTileBytes, kPageBytes = GE::kPageBytes, kGroup = GE::kGroup;
    constexpr int kOffQ = GE::kOffQ, kOffK = GE::kOffK, kOffV = GE::kOffV;
    extern __shared__ unsigned char smem_raw[];
    unsigned char* smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
    Bars& B = *reinterpret_cast<Bars*>(smem + GE::kOffBar);
    volatile int* abort_flag = &B.abort_flag;
    Pair* sorted_pairs = reinterpret_cast<Pair*>(smem + GE::kOffPairs);
    int* before = reinterpret_cast<int*>(smem + GE::kOffPairs);
    int* scratch = reinterpret_cast<int*>(smem + GE::kOffScratch);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int lg = __ffs(a.hq / a.hkv) - 1;  // row r of a tile: token r >> lg, head r & (G - 1)
    const int step = 2 * kBM >> lg;          // tokens of an item
    // before[c]: a thread counts up to four neighbouring chunks, then a scan
    const int per = (a.num_chunks + kThreads - 1) / kThreads;
    int counts[4], sum = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int c = (int)threadIdx.x * per + j;
        counts[j] = sum;
        if (j < per && c < a.num_chunks) sum += (chunk_rows(a, c, blockIdx.x == 0) + step - 1) / step;
    }
    int upto = sum;  // of the warp's lanes up to this one
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int s = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += s;
    }
    if (lane == 31) scratch[warp] = upto;
    if (threadIdx.x == 0) {
        for (int x = 0; x < 2; ++x) {
            mbar_init(&B.q_full[x], 1);
            mbar_init(&B.q_empty[x], 1);
            mbar_init(&B.q_f16[x], 128);
            mbar_init(&B.s_full[x], 1);
            mbar_init(&B.p_full[x], 256);
            mbar_init(&B.o_done[x], 1);
            mbar_init(&B.o_free[x], 128);
            mbar_init(&B.l_full[x], 256);
        }
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&B.k_full[s], 1);
            mbar_init(&B.k_empty[s], 1);
            mbar_init(&B.v_full[s], 1);
            mbar_init(&B.v_empty[s], 1);
            mbar_init(&B.v_raw[s], 1);
        }
        mbar_init(&B.drain, 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 1) tmem_alloc(&B.tmem, 512);
    __syncthreads();
    int n_pairs = 0, base = upto - sum;
#pragma unroll
    for (int i = 0; i < kThreads / 32; ++i) {
        if (i == warp) base += n_pairs;
        n_pairs += scratch[i];
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int c = (int)threadIdx.x * per + j;
        if (j < per && c < a.num_chunks) before[c] = base + counts[j];
    }
    __syncthreads();
    const bool sorted = n_pairs <= kMaxPairs;
    static_assert(kMaxPairs == kThreads, "a thread ranks one pair");
    if (sorted) {
        // rank = pairs with more tiles, or as many and a smaller index: with larger keys
        Pair mine{0, 0, 0, 0};
        int key = -1;
        if ((int)threadIdx.x < n_pairs) {
            mine = make_pair(a, before, step, threadIdx.x);
            key = min(pages_of(a, mine).tiles, 1 << 20) * kMaxPairs + (kMaxPairs - 1 - (int)threadIdx.x);
        }
        scratch[threadIdx.x] = key;
        __syncthreads();
        if ((int)threadIdx.x < n_pairs) {
            int rank = 0;
#pragma unroll 4
            for (int q = 0; q < (n_pairs + 3) / 4; ++q) {
                const int4 o = reinterpret_cast<const int4*>(scratch)[q];
                rank += (o.x > key) + (o.y > key) + (o.z > key) + (o.w > key);
            }
            sorted_pairs[rank] = mine;
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = B.tmem;  // S_A at +0, S_B at +128, O_A at +256, O_B at +384
    const int n_items = n_pairs * a.hkv;
    // Walks this CTA's items.
    struct Walk {
        int round = 0;
        int h;
        Pair p;
        Pages g;
    };
    auto next_item = [&](Walk& w) -> bool {
        const int i = w.round * (int)gridDim.x + ((w.round & 1) ? (int)gridDim.x - 1 - (int)blockIdx.x : (int)blockIdx.x);
        if (i >= n_items) return false;
        const int pr = div.hkv.quot(i);
        w.h = i - pr * a.hkv;
        w.p = sorted ? sorted_pairs[pr] : make_pair(a, before, step, pr);
        w.g = pages_of(a, w.p);
        ++w.round;
        return true;
    };

    if (warp < 4) {
        setmaxnreg_dec<kRegsIssue>();
        if (warp == 0 || warp == 2) {
            // ====================== TMA producers: K and Q, V ======================
            // Warp 0 copies K tiles and Q, warp 2 V tiles: neither waits behind the
            // other's buffers.
            const uint64_t pol_q = l2_evict_first_policy();
            const uint64_t pol_kv = l2_evict_normal_policy();
            const bool is_k = warp == 0;
            if (lane == 0) {
                if (is_k) tma_prefetch_map(&maps.q);
                tma_prefetch_map(is_k ? &maps.k : &maps.v);
            }
            bool go = true;
            // lane 0 waits for `empty` (unless the buffer is new) and arms `full`
            auto arm = [&](uint64_t* full, uint64_t* empty, bool fresh, uint32_t parity, uint32_t bytes) -> bool {
                if (lane == 0) {
                    go = fresh ? !*abort_flag : wait_or_abort(empty, parity, abort_flag, a.status);
                    if (go) mbar_arrive_expect_tx(full, bytes);
                }
                return go = __shfl_sync(0xffffffffu, go, 0);
            };
            // Lane p < 8 copies page p of a tile.  Its block's id, from the table a
            // tile ahead: nothing of the load's result is looked at until then (lanes
            // without a page read their row's first entry).
            auto has_page = [&](const Pages& pg, int t) -> bool {
                return lane < kBN / kPage && t * (kBN / kPage) + lane < pg.n;
            };
            auto page = [&](const Pages& pg, int t) -> int {
                const int p = t * (kBN / kPage) + lane;
                return p >= pg.sink ? p + pg.gap : p;
            };
            auto block_id = [&](const Walk& w, int t) -> int32_t {
                const int col = has_page(w.g, t) ? div.block_pages.quot(page(w.g, t)) : 0;
                return a.block_table[(int64_t)w.p.c * a.max_blocks + col];
            };
            // The pool row of this lane's page, or -1.
            auto page_row = [&](const Walk& w, int t, int32_t blk) -> int {
                if (!has_page(w.g, t)) return -1;
                if (blk < 0 || blk >= a.num_blocks) {
                    if (is_k) record_error(a.status, KVATTN_ERR_BAD_INDEX);
                    return -1;
                }
                const int pg = page(w.g, t), in = pg * kPage - div.block_pages.quot(pg) * a.block_size;
                return (int)(((int64_t)blk * a.hkv + w.h) * a.block_size) + in;
            };
            auto copy = [&](const CUtensorMap* m, unsigned char* tile, int row, uint64_t* full) {
                if (row < 0) return;
                if constexpr (kHD == 128)
                    tma_load_4d(tile + lane * kPageBytes, m, 0, 0, 0, row >> 3, full, pol_kv);
                else
                    tma_load_2d(tile + lane * kPageBytes, m, 0, row, full, pol_kv);
            };
            int g = 0, ii = 0;     // tiles and items started so far (this CTA)
            int kg = 0, qg = 0;    // K and Q tiles (A then B, item by item) armed
            // bit s of stage s's V: armed; its last copies complete on v_raw (else on
            // v_full), in a phase of this parity; parity of its tiles that did so far
            uint32_t v_armed = 0, v_raw = 0, v_parity = 0, fixes = 0;
            Walk w, ahead;  // this item and the next
            bool more = next_item(ahead);
            int32_t blk_next = more ? block_id(ahead, 0) : 0;
            while (go && more) {
                w = ahead;
                for (int t = 0; t < w.g.tiles; ++t, ++g) {
                    const int row = page_row(w, t, blk_next);
                    const uint32_t bytes = (uint32_t)__popc(__ballot_sync(0xffffffffu, row >= 0)) * (uint32_t)kPageBytes;
                    const int s = g % kStages;
                    const uint32_t parity = ((g / kStages) - 1) & 1;
                    if (is_k) {
                        // K stage: free once S_A and S_B of tile g - kStages are done
                        if (!arm(&B.k_full[s], &B.k_empty[s], g < kStages, parity, bytes)) break;
                        copy(&maps.k, smem + kOffK + s * kTileBytes, row, &B.k_full[s]);
                        kg = g + 1;
                    }
                    if (t == 0) more = next_item(ahead);
                    const bool last = t + 1 == w.g.tiles;
                    blk_next = block_id(last ? ahead : w, last ? 0 : t + 1);
                    if (is_k) {
                        if (t > 0) continue;
                        // Q_x: free once every S_x MMA of the previous item is done (its
                        // K stage is free sooner, so K goes first)
                        for (int x = 0; x < 2; ++x) {
                            if (!arm(&B.q_full[x], &B.q_empty[x], ii == 0, (ii - 1) & 1, kTileBytes)) break;
                            if (lane < GE::kPanels)
                                tma_load_3d(smem + kOffQ + x * kTileBytes + lane * kPanel, &maps.q, 64 * lane, w.h << lg,
                                            w.p.row0 + x * (kBM >> lg), &B.q_full[x], pol_q);
                            ++qg;
                        }
                        if (!go) break;
                        ++ii;
                    } else {
                        // V stage: free once PV_A and PV_B of tile g - kStages are done
                        const bool fix = has_unseen(a, unseen_of(a, w.p, w.g), t);
                        uint64_t* full = fix ? &B.v_raw[s] : &B.v_full[s];
                        if (!arm(full, &B.v_empty[s], g < kStages, parity, bytes)) break;
                        copy(&maps.v, smem + kOffV + s * kTileBytes, row, full);
                        const uint32_t phase = fix ? fixes >> s & 1u : (g / kStages) & 1u;
                        const uint32_t bit = 1u << s;
                        v_armed |= bit;
                        v_raw = fix ? v_raw | bit : v_raw & ~bit;
                        v_parity = phase ? v_parity | bit : v_parity & ~bit;
                        if (fix) fixes ^= bit;
                    }
                }
            }
            // After an abort, let every armed copy land before the CTA can exit.
            __syncwarp();
            if (lane == 0 && *abort_flag) {
                for (int t = max(0, kg - kStages); t < kg; ++t)
                    mbar_wait(&B.k_full[t % kStages], (t / kStages) & 1, a.status);
                for (int s = 0; s < kStages; ++s)
                    if (v_armed >> s & 1u)
                        mbar_wait(v_raw >> s & 1u ? &B.v_raw[s] : &B.v_full[s], v_parity >> s & 1u, a.status);
                for (int q = max(0, qg - 2); q < qg; ++q) mbar_wait(&B.q_full[q & 1], (q >> 1) & 1, a.status);
            }
        } else if (warp == 1) {
            // ============================== MMA issuer ==============================
            // The whole warp runs the schedule (waits agreed by the warp) and one
            // elected lane issues.  Operand descriptors are built once: a stage or
            // k-step only adds (byte offset >> 4) to the start-address field, which
            // cannot carry out of it (shared-memory offsets stay below 256 KB).
            constexpr uint32_t idesc_s = kF16 ? idesc_f16_f32(kBM, kBN, false) : idesc_bf16_f32(kBM, kBN, false);
            constexpr uint32_t idesc_o = kF16 ? idesc_f16_f32(kBM, kHD, true) : idesc_bf16_f32(kBM, kHD, true);
            const uint32_t sbase = smem_addr(smem);
            const uint64_t dQ = umma_desc_sw128(sbase + kOffQ, 16, 1024);      // Q_x: + x * kTileBytes
            const uint64_t dK = umma_desc_sw128(sbase + kOffK, 16, kGroup);    // K stage s: + s * kTileBytes
            const uint64_t dV = umma_desc_sw128(sbase + kOffV, 1024, kGroup);  // V stage s: + s * kTileBytes
            constexpr uint64_t kTileStep = kTileBytes >> 4;
            auto issue_s = [&](int x, int g) {  // S_x = Q_x K_g^T
                if (elect_one()) {
                    const uint64_t q = dQ + x * kTileStep, kd = dK + (g % kStages) * kTileStep;
                    const uint32_t d = tmem + x * 128;
#pragma unroll
                    for (int k = 0; k < kHD / 16; ++k)  // k-step: 16 columns, 32 B inside the 128-byte atom
                        tc_mma_f16(d, q + (uint64_t)(((k >> 2) * kPanel + (k & 3) * 32) >> 4),
                                   kd + (uint64_t)(((k >> 2) * 1024 + (k & 3) * 32) >> 4), idesc_s, k > 0);
                    tc_commit(&B.s_full[x]);
                }
                __syncwarp();
            };
            // O_x += P_x V_g, P_x in S_x's first 64 columns; the first tile of an
            // item overwrites O_x (o_free: the previous item's has been read)
            auto issue_pv = [&](int x, int g, bool first, bool last) {
                if (elect_one()) {
                    const uint64_t vd = dV + (g % kStages) * kTileStep;
                    const uint32_t d = tmem + 256 + x * 128, pa = tmem + x * 128;
#pragma unroll
                    for (int k = 0; k < kBN / 16; ++k)  // k-step: 16 keys = two 8-key groups
                        tc_mma_f16_ts(d, pa + k * 8, vd + (uint64_t)((k * 2 * kGroup) >> 4), idesc_o, (!first || k > 0));
                    if (x == 1) tc_commit(&B.v_empty[g % kStages]);
                    if (last) tc_commit(&B.o_done[x]);
                }
                __syncwarp();
            };
            auto commit = [&](uint64_t* b) {
                if (elect_one()) tc_commit(b);
                __syncwarp();
            };
            auto wait = [&](uint64_t* b, uint32_t parity) {
                if (__all_sync(0xffffffffu, mbar_try_wait(b, parity))) return true;
                return warp_wait(b, parity, abort_flag, a.status);
            };
            // Order per tile t: PV_A(t) S_A(t+1) PV_B(t) S_B(t+1); S_x(t+1)
            // overwrites S_x's columns after PV_x(t) has read P_x(t) from them
            // (tensor operations of one thread run in issue order).
            Walk w;
            int n_kv = next_item(w) ? w.g.tiles : 0;
            int g = 0, item = 0;
            bool ok = n_kv > 0;
            uint64_t* q_ready = kF16 ? B.q_f16 : B.q_full;
            if (ok && (ok = wait(&q_ready[0], 0) && wait(&B.k_full[0], 0))) {
                tc_fence_after();
                issue_s(0, 0);
                if (n_kv == 1) commit(&B.q_empty[0]);
                if ((ok = wait(&q_ready[1], 0))) {
                    tc_fence_after();
                    issue_s(1, 0);
                    commit(&B.k_empty[0]);
                    if (n_kv == 1) commit(&B.q_empty[1]);
                }
            }
            while (ok && n_kv > 0) {
                const uint32_t op = (item - 1) & 1;
                for (int t = 0; t + 1 < n_kv; ++t, ++g) {
                    const int g1 = g + 1;
                    if (!(ok = wait(&B.v_full[g % kStages], (g / kStages) & 1) && wait(&B.p_full[0], g & 1))) break;
                    if (t == 0 && item > 0 && !(ok = wait(&B.o_free[0], op))) break;
                    tc_fence_after();
                    issue_pv(0, g, t == 0, false);
                    if (!(ok = wait(&B.k_full[g1 % kStages], (g1 / kStages) & 1))) break;
                    tc_fence_after();
                    issue_s(0, g1);
                    if (t + 2 == n_kv) commit(&B.q_empty[0]);
                    if (!(ok = wait(&B.p_full[1], g & 1))) break;
                    if (t == 0 && item > 0 && !(ok = wait(&B.o_free[1], op))) break;
                    tc_fence_after();
                    issue_pv(1, g, t == 0, false);
                    issue_s(1, g1);
                    commit(&B.k_empty[g1 % kStages]);
                    if (t + 2 == n_kv) commit(&B.q_empty[1]);
                }
                if (!ok) break;
                // the item's last tile, and the next item's first S
                const int n_next = next_item(w) ? w.g.tiles : 0;
                const int g1 = g + 1;
                if (!(ok = wait(&B.v_full[g % kStages], (g / kStages) & 1) && wait(&B.p_full[0], g & 1))) break;
                if (n_kv == 1 && item > 0 && !(ok = wait(&B.o_free[0], op))) break;
                tc_fence_after();
                issue_pv(0, g, n_kv == 1, true);
                if (n_next > 0) {
                    if (!(ok = wait(&q_ready[0], (item + 1) & 1) && wait(&B.k_full[g1 % kStages], (g1 / kStages) & 1)))
                        break;
                    tc_fence_after();
                    issue_s(0, g1);
                    if (n_next == 1) commit(&B.q_empty[0]);
                }
                if (!(ok = wait(&B.p_full[1], g & 1))) break;
                if (n_kv == 1 && item > 0 && !(ok = wait(&B.o_free[1], op))) break;
                tc_fence_after();
                issue_pv(1, g, n_kv == 1, true);
                if (n_next > 0) {
                    if (!(ok = wait(&q_ready[1], (item + 1) & 1))) break;
                    tc_fence_after();
                    issue_s(1, g1);
                    commit(&B.k_empty[g1 % kStages]);
                    if (n_next == 1) commit(&B.q_empty[1]);
                }
                ++g;
                ++item;
                n_kv = n_next;
            }
            // every MMA this warp issued has completed once `drain` flips
            commit(&B.drain);
            mbar_wait(&B.drain, 0, a.status);
        } else {
            // ============================ stale V rows =============================
            // V rows that no row of the item sees must be zero for the MMA: they
            // may hold anything, and 0 * NaN is NaN.
            // The copies of such a tile complete on v_raw, and this warp completes
            // v_full.
            int g = 0, since = 0;  // tiles; tiles since the last wait
            uint32_t fixes = 0;    // bit s: parity of stage s's tiles seen here so far
            bool ok = true;
            Walk w;
            while (ok && next_item(w)) {
                const Unseen un = unseen_of(a, w.p, w.g);
                for (int t = 0; t < w.g.tiles; ++t, ++g) {
                    ++since;
                    if (!has_unseen(a, un, t)) continue;
                    const int s = g % kStages;
                    if (!(ok = long_wait(&B.v_raw[s], fixes >> s & 1u, since, abort_flag, a.status))) break;
                    since = 0;
                    fixes ^= 1u << s;
                    unsigned char* tile = smem + kOffV + s * kTileBytes;
                    constexpr int kChunks = kHD / 8;  // 16-byte chunks of a row: a warp's stores are of whole rows
                    auto zero = [&](int r0, int r1) {
                        for (int i = r0 * kChunks + lane; i < r1 * kChunks; i += 32) {
                            const int r = i / kChunks, ch = i % kChunks;
                            *reinterpret_cast<uint4*>(tile + (r >> 3) * kGroup + (r & 7) * 128 + (ch >> 3) * 1024 +
                                                      (ch & 7) * 16) = make_uint4(0, 0, 0, 0);
                        }
                    };
                    zero(min(max(a.sinks - t * kBN, 0), kBN), min(max(un.low + 1 - t * kBN, 0), kBN));
                    zero(min(max(un.end - t * kBN, 0), kBN), kBN);
                    fence_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&B.v_full[s]);
                }
            }
        }
    } else if (warp < 12) {
        setmaxnreg_inc<kRegsSoftmax>();
        // ================================= softmax ==================================
        // All eight warps work on whichever tile's S is due (A(t), B(t), A(t+1),
        // ...): thread (quarter, lane) owns row r = 32 quarter + lane of the
        // tile, warps 4-7 its columns 0..63 (half hf = 0) and warps 8-11 its
        // columns 64..127 (hf = 1).  The halves of a row (warps w and w + 4: the
        // same TMEM lane quarter) agree on the row max through shared memory, with
        // a named barrier of that pair per tile.
        // These warps never stop early: after an abort their waits return at once
        // and they run on, over whatever TMEM holds, to the end of their items
        // (nothing of it is reported good).  What a tile costs is its instructions'
        // way to the warps as much as their number: each branch that is not here
        // saves about 100 cycles of 1200 (16 chunks, window 4096: 315 us with the
        // wait's result looked at and the maximum's three cases in branches, 307),
        // and one body for A and B, whose states change places after each, stays in
        // the instruction cache where two do not (windows of 128 and 1024: 41.9 and
        // 103 us, two bodies 47.7 and 107).
        const int hf = (warp - 4) >> 2;
        const int quarter = warp & 3;        // TMEM lanes 32*quarter .. +31
        const int r = quarter * 32 + lane;   // row of the tile
        const uint32_t lane_base = (uint32_t)(quarter * 32) << 16;
        float* xchg = reinterpret_cast<float*>(smem + GE::kOffX);  // [2 tile phases][2 halves][128 rows]
        int g = 0, ii = 0;
        Walk w;
        while (next_item(w)) {
            // (f16: q was divided by 16)
            const float sl2 = kF16 ? a.kv_scale[(int64_t)w.p.c * a.hkv + w.h].x * 16.f * a.scale_log2 : a.scale_log2;
            const int col0 = w.g.gap * kPage;
            const int tok = w.p.pos0 - col0;                    // column of the item's first token
            float m_now = -INFINITY, l_now = 0.f, m_other = -INFINITY, l_other = 0.f;  // of A and B in turn
            auto swap = [&] {
                const float m = m_now, l = l_now;
                m_now = m_other;
                l_now = l_other;
                m_other = m;
                l_other = l;
            };
#pragma unroll 1
            for (int st = 0; st < 2 * w.g.tiles; ++st) {
                const int t = st >> 1, x = st & 1;
                const uint32_t tS = tmem + lane_base + x * 128 + hf * 64;
                const uint32_t tO = tmem + lane_base + 256 + x * 128 + hf * (kHD / 2);
                const int p0 = tok + ((x * kBM + quarter * 32) >> lg);  // column of the warp's first row
                const int p1 = p0 + ((32 >> lg) - 1);                   // ... of its last
                const int pr = p0 + (lane >> lg);                       // ... of this thread's
                const int c = t * kBN + hf * 64;                        // first column of this half
                const bool some = c + 63 > p0 || (c <= p1 - a.window && c + 63 >= a.sinks);
                wait_or_abort(&B.s_full[x], g & 1, abort_flag, a.status);
                __syncwarp();
                if (x == 1 && w.p.rows <= step / 2) {  // B has no rows: P_B may be anything
                    mbar_arrive(&B.p_full[1]);
                    ++g;
                    swap();
                    continue;
                }
                uint32_t sv[64];
                tc_fence_after();
                tmem_ld32(tS, *reinterpret_cast<uint32_t(*)[32]>(&sv[0]));
                tmem_ld32(tS + 32, *reinterpret_cast<uint32_t(*)[32]>(&sv[32]));
                tmem_ld_wait();
                if (some) {  // bit e: column c + e is seen
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        const int cq = c + 32 * q;
                        const uint32_t m = low_bits(pr - cq + 1) & (~low_bits(pr - a.window - cq + 1) | low_bits(a.sinks - cq));
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            if (!(m & (1u << e))) sv[32 * q + e] = __float_as_uint(-INFINITY);
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
                const bool none = m_now == -INFINITY;  // no seen key so far
                const bool rescale = !none && m_tile > m_now + 8.f;
                const float m_new = none || rescale ? m_tile : m_now;
                const float alpha = none ? 1.f : fast_exp2(m_now - m_new);
                m_now = m_new;
                // P = 2^(s*scale*log2e - m), in the type of V that the MMA takes it
                // with, into columns 32hf..32hf+31 of S_x (both halves have read
                // their S before the barrier); a row with no seen key yet subtracts
                // +inf so every p is 0.  The row sum adds the fp32 p, whose rounding
                // to bf16 (f16) is off by at most 2^-8 (2^-11) relative, at random.
                uint32_t pw[32];
                const float msub = m_now == -INFINITY ? INFINITY : m_now;
                const uint64_t scale2 = pk(sl2, sl2), msub2 = pk(-msub, -msub);
                uint64_t sum2[2] = {0, 0};
#pragma unroll
                for (int e = 0; e < 32; ++e) {
                    const uint64_t xx =
                        ffma2(pk(__uint_as_float(sv[2 * e]), __uint_as_float(sv[2 * e + 1])), scale2, msub2);
                    const uint64_t pp = pk(fast_exp2(pk_lo(xx)), fast_exp2(pk_hi(xx)));
                    pw[e] = kF16 ? pack_f16_rn(pk_lo(pp), pk_hi(pp)) : pack_bf16_rn(pk_lo(pp), pk_hi(pp));
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
                mbar_arrive(&B.p_full[x]);
                g += x;
                swap();
            }
            // this item's row sums to the output warps (two items' worth: the sums
            // of item ii - 2 were read before S_x of this item was issued)
            float* lx = xchg + 512 + (ii & 1) * 512;  // [2 halves][2 tiles][128 rows]
            lx[(hf * 2 + 0) * 128 + r] = l_now;
            lx[(hf * 2 + 1) * 128 + r] = l_other;
            mbar_arrive(&B.l_full[ii & 1]);
            ++ii;
        }
    } else {
        setmaxnreg_dec<kRegsOutput>();
        // ================================== output ==================================
        // Thread (quarter, lane) owns row r of both tiles.
        const int quarter = warp & 3;
        const int r = quarter * 32 + lane;
        const uint32_t lane_base = (uint32_t)(quarter * 32) << 16;
        const float* xchg = reinterpret_cast<const float*>(smem + GE::kOffX);
        // Rows go out of registers, in whole 32-byte sectors where out is aligned to
        // them: O_x is free sooner than by way of shared memory and bulk stores,
        // which the first P.V of the next item waits for (16 chunks of 512 queries,
        // window 128 and 1024: 47.0 and 106.4 us, bulk stores 49.5 and 108.4).
        const bool wide = (reinterpret_cast<uintptr_t>(a.out) & 31) == 0;
        int ii = 0;
        bool ok = true;
        auto convert_q = [&](uint32_t parity, int tiles) {
#pragma unroll 1
            for (int x = 0; ok && x < 2; ++x) {
                if (!(ok = long_wait(&B.q_full[x], parity, tiles, abort_flag, a.status))) break;
                uint4* q = reinterpret_cast<uint4*>(smem + kOffQ + x * kTileBytes);
#pragma unroll 4
                for (int i = r; i < kTileBytes / 16; i += 128) {
                    const uint4 v = q[i];
                    auto half2 = [](uint32_t u) { return pack_f16_rn(bf16lo(u) * 0.0625f, bf16hi(u) * 0.0625f); };
                    q[i] = make_uint4(half2(v.x), half2(v.y), half2(v.z), half2(v.w));
                }
                fence_async_smem();
                mbar_arrive(&B.q_f16[x]);
            }
        };
        Walk w, ahead;
        bool more = next_item(ahead);
        if (kF16 && more) convert_q(0, 0);
        while (ok && more) {
            w = ahead;
            more = next_item(ahead);
            // (the next item's Q comes once this one's scores are done, before its
            // sums and outputs are)
            if (kF16 && more) convert_q((ii + 1) & 1, w.g.tiles);
            if (!ok || !long_wait(&B.l_full[ii & 1], (ii >> 1) & 1, w.g.tiles, abort_flag, a.status)) break;
            const float* lx = xchg + 512 + (ii & 1) * 512;
            const float l[2] = {lx[r] + lx[256 + r], lx[128 + r] + lx[384 + r]};
            const float vmul = kF16 ? a.kv_scale[(int64_t)w.p.c * a.hkv + w.h].y : 1.f;
#pragma unroll 1
            for (int x = 0; x < 2; ++x) {
                if (!(ok = warp_wait(&B.o_done[x], ii & 1, abort_flag, a.status))) break;
                tc_fence_after();
                const float lr = x ? l[1] : l[0];
                const float inv = (lr > 0.f ? 1.f / lr : 0.f) * vmul;
                const int row = (x * kBM + r) >> lg;  // token of the item
                const uint32_t tO = tmem + lane_base + 256 + x * 128;
                __nv_bfloat16* orow =
                    reinterpret_cast<__nv_bfloat16*>(a.out) +
                    ((int64_t)(w.p.row0 + row) * a.hq + (w.h << lg) + (r & ((1 << lg) - 1))) * kHD;
#pragma unroll 1
                for (int q = 0; q < kHD / 32; ++q) {
                    uint32_t v[32];
                    tmem_ld32(tO + q * 32, v);
                    tmem_ld_wait();
                    if (q + 1 == kHD / 32) {
                        tc_fence_before();
                        mbar_arrive(&B.o_free[x]);
                    }
                    uint32_t o[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        o[e] = pack_bf16_rn(__uint_as_float(v[2 * e]) * inv, __uint_as_float(v[2 * e + 1]) * inv);
                    if (row < w.p.rows) {
                        if (wide) {
                            store_256(orow + q * 32, o);
                            store_256(orow + q * 32 + 16, o + 8);
                        } else {
#pragma unroll
                            for (int ch = 0; ch < 4; ++ch)
                                *reinterpret_cast<uint4*>(orow + q * 32 + 8 * ch) =
                                    make_uint4(o[4 * ch], o[4 * ch + 1], o[4 * ch + 2], o[4 * ch + 3]);
                        }
                    }
                }
            }
            ++ii;
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// ---- host: tensor maps --------------------------------------------------------

template <int kHD>
bool make_maps(const PrefillArgs& a, Maps& m)
{
    std::memset(&m, 0, sizeof(m));
    const cuuint32_t G = a.hq / a.hkv;
    const cuuint64_t dims[3] = {(cuuint64_t)kHD, (cuuint64_t)a.hq, (cuuint64_t)a.total_q};
    const cuuint64_t strides[2] = {(cuuint64_t)kHD * 2, (cuuint64_t)a.hq * kHD * 2};
    const cuuint32_t qbox[3] = {64, G, (cuuint32_t)kBM / G};
    if (!encode(&m.q, a.q, 3, dims, strides, qbox)) return false;
    const int64_t rows = (int64_t)a.num_blocks * a.hkv * a.block_size;
    if constexpr (kHD == 128) return pool_maps(a.k_pool, a.v_pool, rows, false, &m.k, &m.v);
    // (64 columns, rows): a box of (64, 16) is one 16-row page, [16 rows][128 B]
    const cuuint64_t pdims[2] = {64, (cuuint64_t)rows};
    const cuuint64_t pstrides[1] = {64 * 2};
    const cuuint32_t pbox[2] = {64, 16};
    return encode(&m.k, a.k_pool, 2, pdims, pstrides, pbox) &&
           encode(&m.v, a.v_pool, 2, pdims, pstrides, pbox);
}

template <int kHD, bool kF16>
kvattn_status launch(const PrefillArgs& a, cudaStream_t s)
{
    if ((int64_t)a.num_blocks * a.hkv * a.block_size >= ((int64_t)1 << 31)) return KVATTN_ERR_UNSUPPORTED;
    const int64_t step = 2 * kBM / (a.hq / a.hkv);
    if (!window_items_ok(a)) return KVATTN_ERR_UNSUPPORTED;
    const int64_t items = a.num_chunks * ((a.max_q_len + step - 1) / step) * a.hkv;  // at most
    Maps maps;
    if (!make_maps<kHD>(a, maps)) return KVATTN_ERR_CUDA;
    constexpr int kSmem = Geo<kHD>::kSmemBytes;
    static_assert(kSmem <= 232448, "shared memory of a block");
    static SmemLimit limit;
    if (limit.ensure(reinterpret_cast<const void*>(prefill_window_kernel<kHD, kF16>), kSmem) != cudaSuccess)
        return KVATTN_ERR_CUDA;
    const int64_t grid = std::min<int64_t>(items, num_sms());  // persistent: one CTA per SM
    const Divisors div{Divisor(a.hkv), Divisor(a.block_size / kPage)};
    for (int c = 0; c < a.num_chunks; c += kMaxChunks) {
        PrefillArgs b = a;
        b.num_chunks = std::min(a.num_chunks - c, kMaxChunks);
        b.cu_q_lens += c;
        b.prefix_lens += c;
        b.block_table += (int64_t)c * a.max_blocks;
        if (b.kv_scale) b.kv_scale += (int64_t)c * a.hkv;
        const kvattn_status st = cuda_status(launch_pdl(prefill_window_kernel<kHD, kF16>, dim3((unsigned)grid),
                                                        dim3(kThreads), kSmem, s, b, maps, div));
        if (st != KVATTN_OK) return st;
    }
    return KVATTN_OK;
}

}  // namespace

kvattn_status launch_prefill_window(const PrefillArgs& a, cudaStream_t s)
{
    if (a.kv_scale) return a.d == 128 ? launch<128, true>(a, s) : KVATTN_ERR_UNSUPPORTED;
    return a.d == 128 ? launch<128, false>(a, s) : a.d == 64 ? launch<64, false>(a, s) : KVATTN_ERR_UNSUPPORTED;
}

}  // namespace kvattn
