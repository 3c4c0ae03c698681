// Windowed decode attention in one launch, for calls whose keys are few: a
// thread-block cluster per (sequence, KV head).
//
// What it computes: kvattn_decode_window's out[b][j], an online softmax over
// the seen 16-token tiles of each (sequence, KV head), as decode_kernel.cuh.
//
// How: with a window the keys of a segment are bounded, so the segments of a
// call are of much the same length and need neither a balanced stream nor a
// second kernel that merges its pieces.  What such a call waits for is
// latency: every step below is one that a short chain of dependent loads asks
// for.  The warps of a cluster take the segment's tiles in turn.  A warp loads
// its tile straight from global memory into MMA fragments (no shared memory,
// no barrier; fp8 pages, which take longer to convert than to arrive, by way of
// two buffers of the warp's own): the dims of a dot product may be taken in any
// order, so a lane loads whole 16-byte chunks and the query's fragments follow
// the same order, and the dims of the output are named so that each lane's chunks
// of V hold the rows it owns.  S^T = K Q^T and O^T += V^T P^T have the 16 tokens and the
// dims on the M axis and up to 8 query heads on N; P goes from the C fragment
// of one to the B fragment of the other by movmatrix.  A warp keeps its own
// running maximum and sum; the warps of a CTA merge through shared memory and
// the CTAs of a cluster through distributed shared memory.
#include <mutex>
#include <type_traits>

#include <cooperative_groups.h>

#include "decode_kernel.cuh"

namespace kvattn {
namespace {

namespace cg = cooperative_groups;

enum DirectKind { kBf16Cache, kFp8Cache, kF32Cache };

// One warp's share of a segment over a bf16 cache: its running maxima and sums
// (log2 units) of query heads 2 q4 and 2 q4 + 1, and how they weigh a tile's
// scores (fp8 pages: Fp8Softmax).
struct Softmax {
    float m[2], l[2];
    __device__ __forceinline__ void init()
    {
        m[0] = m[1] = -INFINITY;
        l[0] = l[1] = 0.f;
    }
    // Probabilities of this lane's tokens r0, r1 (scores x: (r0, head 0),
    // (r0, 1), (r1, 0), (r1, 1)).  The maxima are raised, and o rescaled, when a
    // score exceeds them by more than 2^8; the warp agrees on them only then.
    template <int kN>
    __device__ __forceinline__ void step(const float (&x)[4], float (&o)[kN][4], float (&p)[4])
    {
        float l0 = fmaxf(x[0], x[2]), l1 = fmaxf(x[1], x[3]);
        if (__any_sync(0xffffffffu, l0 > m[0] + 8.f || l1 > m[1] + 8.f)) {
#pragma unroll
            for (int s = 4; s < 32; s <<= 1) {
                l0 = fmaxf(l0, __shfl_xor_sync(0xffffffffu, l0, s));
                l1 = fmaxf(l1, __shfl_xor_sync(0xffffffffu, l1, s));
            }
            float f0 = 1.f, f1 = 1.f;
            if (l0 > m[0] + 8.f) {
                f0 = m[0] == -INFINITY ? 0.f : fast_exp2(m[0] - l0);
                l[0] *= f0;
                m[0] = l0;
            }
            if (l1 > m[1] + 8.f) {
                f1 = m[1] == -INFINITY ? 0.f : fast_exp2(m[1] - l1);
                l[1] *= f1;
                m[1] = l1;
            }
#pragma unroll
            for (int e = 0; e < kN; ++e) {
                o[e][0] *= f0;
                o[e][1] *= f1;
                o[e][2] *= f0;
                o[e][3] *= f1;
            }
        }
        // a head whose scores are all -inf so far has no weight yet
        const float m0 = m[0] == -INFINITY ? 0.f : m[0], m1 = m[1] == -INFINITY ? 0.f : m[1];
        p[0] = fast_exp2(x[0] - m0);
        p[1] = fast_exp2(x[1] - m1);
        p[2] = fast_exp2(x[2] - m0);
        p[3] = fast_exp2(x[3] - m1);
        l[0] += p[0] + p[2];
        l[1] += p[1] + p[3];
    }
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ uint4 ldg16(const void* p) { return __ldg(reinterpret_cast<const uint4*>(p)); }

// ---- bf16 cache.  K: lane (g4, q4) holds rows (tokens) g4 and g4 + 8, 16-byte
// chunks q4 + 4i of each; chunk i is the lane's share of MMA k-steps 2i and
// 2i + 1.  V: rows 2 q4, 2 q4 + 1, 2 q4 + 8, 2 q4 + 9, chunks g4 (+ 8 at D =
// 128); two rows' words interleave into pairs of tokens of one dim.
template <int kD>
struct Bf16Tile {
    static constexpr int kC = kD / 32;   // K chunks per row and lane
    static constexpr int kVC = kD / 64;  // V chunks per row and lane
    uint4 k[2][kC];
    __device__ __forceinline__ void load_k(const char* kp, uint32_t seen, int g4, int q4)
    {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const bool in = seen >> (g4 + 8 * r) & 1u;
#pragma unroll
            for (int i = 0; i < kC; ++i)
                k[r][i] = in ? ldg16(kp + (g4 + 8 * r) * (kD * 2) + (q4 + 4 * i) * 16) : make_uint4(0, 0, 0, 0);
        }
    }
    static __device__ __forceinline__ void load_v(uint4 (&v)[4][kVC], const char* vp, uint32_t seen, int g4, int q4)
    {
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int row = 2 * q4 + (r & 1) + 8 * (r >> 1);
            const bool in = seen >> row & 1u;
#pragma unroll
            for (int i = 0; i < kVC; ++i)
                v[r][i] = in ? ldg16(vp + row * (kD * 2) + (g4 + 8 * i) * 16) : make_uint4(0, 0, 0, 0);
        }
    }
    __device__ __forceinline__ void scores(float (&s)[4], const uint32_t (&q)[kD / 16][2]) const
    {
        float u[4] = {0.f, 0.f, 0.f, 0.f};  // two chains of dependent MMAs
#pragma unroll
        for (int i = 0; i < kC; ++i) {
            mma_bf16_16816(s, k[0][i].x, k[1][i].x, k[0][i].y, k[1][i].y, q[2 * i][0], q[2 * i][1]);
            mma_bf16_16816(u, k[0][i].z, k[1][i].z, k[0][i].w, k[1][i].w, q[2 * i + 1][0], q[2 * i + 1][1]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) s[i] += u[i];
    }
    // O^T rows g4 and g4 + 8 of fragment e are dims dim_of(e, 0) and dim_of(e, 1)
    static __device__ __forceinline__ int dim_of(int e, int half, int g4)
    {
        return kD == 128 ? 64 * half + 8 * g4 + e : 8 * g4 + 4 * half + e;
    }
    static __device__ __forceinline__ void add(const uint4 (&v)[4][kVC], float (&o)[kD / 16][4], uint32_t b0, uint32_t b1)
    {
        uint32_t w[4][kVC * 4];
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int i = 0; i < kVC; ++i) {
                w[r][4 * i] = v[r][i].x;
                w[r][4 * i + 1] = v[r][i].y;
                w[r][4 * i + 2] = v[r][i].z;
                w[r][4 * i + 3] = v[r][i].w;
            }
        // pair of dim d (0 .. 8 kVC - 1 of this lane) of rows r, r + 1
        auto pair = [&](int r, int d) { return __byte_perm(w[r][d / 2], w[r + 1][d / 2], d & 1 ? 0x7632 : 0x5410); };
#pragma unroll
        for (int e = 0; e < kD / 16; ++e) {
            const int d0 = e, d1 = kD == 128 ? e + 8 : e + 4;
            mma_bf16_16816(o[e], pair(0, d0), pair(0, d1), pair(2, d0), pair(2, d1), b0, b1);
        }
    }
};

// ---- fp8 pages (layout: kF8Page), f16 operands.  K: rows rk0, rk1 = rk0 + 2,
// chunks q4 and q4 + 4, each the lane's share of four k-steps.  V is stored
// transposed: one word is tokens 4 q4 .. 4 q4 + 3 of a dim, whose order the
// rows rk0, rk1 follow.
struct Fp8Tile {
    uint4 k[2][2];
    uint32_t v[16];
    float ks[2], vs[2];
    __device__ __forceinline__ void load(const unsigned char* pg, int rk0, int g4, int q4)
    {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const int row = rk0 + 2 * r;
#pragma unroll
            for (int i = 0; i < 2; ++i)
                k[r][i] = *reinterpret_cast<const uint4*>(pg + row * 128 + (((q4 + 4 * i) ^ f8_swz(row)) << 4));
            ks[r] = *reinterpret_cast<const float*>(pg + kF8KsOff + 4 * row);
            vs[r] = *reinterpret_cast<const float*>(pg + kF8VsOff + 4 * row);
        }
#pragma unroll
        for (int m = 0; m < 16; ++m)
            v[m] = *reinterpret_cast<const uint32_t*>(pg + kF8VOff + 16 * (8 * m + g4) + 4 * q4);
    }
    __device__ __forceinline__ void scores(float (&s)[4], const uint32_t (&q)[8][2]) const
    {
        float u[4] = {0.f, 0.f, 0.f, 0.f};  // two chains of dependent MMAs
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint32_t a[4] = {k[0][i].x, k[0][i].y, k[0][i].z, k[0][i].w};
            const uint32_t b[4] = {k[1][i].x, k[1][i].y, k[1][i].z, k[1][i].w};
#pragma unroll
            for (int j = 0; j < 4; ++j)
                mma_f16_16816(i ? u : s, e4m3x2_to_f16x2(a[j]), e4m3x2_to_f16x2(b[j]), e4m3x2_to_f16x2(a[j] >> 16),
                              e4m3x2_to_f16x2(b[j] >> 16), q[4 * i + j][0], q[4 * i + j][1]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) s[i] += u[i];
    }
    static __device__ __forceinline__ int dim_of(int e, int half, int g4) { return 16 * e + 8 * half + g4; }
    __device__ __forceinline__ void add(float (&o)[8][4], uint32_t b0, uint32_t b1, uint32_t vmask) const
    {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const uint32_t x = v[2 * e] & vmask, y = v[2 * e + 1] & vmask;
            mma_f16_16816(o[e], e4m3x2_to_f16x2(x), e4m3x2_to_f16x2(y), e4m3x2_to_f16x2(x >> 16),
                          e4m3x2_to_f16x2(y >> 16), b0, b1);
        }
    }
};

// Resident warps per SM that the registers leave room for.  Measured: a
// bf16 tile at D = 128, with the next one on its way, wants 200 registers (32 / 8
// heads, 32 sequences, window 4096: 88.5 us with 8 warps, 91.9 with 12, 100.7
// with 16, which spill); an fp8 page that is converted while the warp's next two
// are under way 128 (64 / 8 heads, 64 sequences, window 1024: 29.4 us with 16
// warps, 29.6 with 20, 36 with 24, which spill; straight from global memory into
// registers 33.1, two pages ahead so 33.9, with three more 36.5; the scores of the
// next page before this one's P.V 30.6).
constexpr int warps_per_sm(int kind, int d, int g)
{
    return kind == kF32Cache ? (d * g > 64 ? 8 : 16) : kind == kFp8Cache || d == 64 ? 16 : 8;
}

constexpr int kRing = 2;  // fp8: pages of a warp in shared memory
// Floats of a warp's output of each head (fp8: they take the place of its pages).
__host__ __device__ constexpr int warp_floats(int kind, int heads, int d)
{
    return kind == kFp8Cache ? kRing * kF8Page / 4 : heads * d;
}
// Shared floats of a CTA: every warp's output, the CTA's merge of them (read by
// the other CTAs of the cluster), and the (max, sum) of each of these heads.
__host__ __device__ constexpr int direct_floats(int kind, int warps, int heads, int d)
{
    return warps * warp_floats(kind, heads, d) + heads * d + (warps + 1) * heads * 2;
}
static_assert(warp_floats(kFp8Cache, 8, 128) >= 8 * 128, "a warp's outputs fit where its pages were");

template <int kKind, int kD, int kG>
__global__ void __launch_bounds__(warps_per_sm(kKind, kD, kG) * 32, 1)
    decode_direct_kernel(const __grid_constant__ DecodeArgs a, const int cluster)
{
    pdl_wait();
    extern __shared__ __align__(128) float part[];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, warps = blockDim.x >> 5;
    const int g4 = lane >> 2, q4 = lane & 3;
    const int rank = blockIdx.x % cluster, seg = blockIdx.x / cluster;
    const int b = seg / a.hkv, h = seg - b * a.hkv;
    const int G = a.hq / a.hkv;
    const int64_t q0 = ((int64_t)b * a.hq + h * G) * kD;  // first element of the group's queries and outputs
    const int32_t* trow = a.block_table + (int64_t)b * a.max_blocks;
    const bool contiguous = a.max_blocks == 1;  // its only block is looked up beside the length
    const int32_t block0 = contiguous ? trow[0] : -1;
    const int L = a.seq_lens[b];

    // per-head rows of the warps' (and, last, the CTA's) outputs and (max, sum)
    const int wf = warp_floats(kKind, G, kD);
    auto row_of = [&](int w, int g) { return part + w * wf + g * kD; };
    float* ml = part + warps * wf + G * kD;
    auto ml_of = [&](int w, int g) { return ml + 2 * (w * G + g); };

    Piece pc;
    pc.len = 0;
    Window win{0, 0, 0, 0};
    if (len_ok(L, a)) {
        win = window_of(L, a);
        pc.len = L;
        pc.sink_tiles = win.sink_tiles;
        pc.gap = win.gap;
        pc.low = win.low;
    } else if (rank == 0 && h == 0 && tid == 0) {
        record_error(a.status, KVATTN_ERR_BAD_INDEX);
    }
    auto first_token = [&](int t) { return (t >= pc.sink_tiles ? t + pc.gap : t) * kTile; };
    const int n = cluster * warps, first = rank * warps + warp;  // this warp: tiles first, first + n, ...
    const int mine = first < win.tiles ? (win.tiles - 1 - first) / n + 1 : 0;
    // row in the pool of this lane's tile of a batch of 32 (-1: none)
    auto lookup = [&](int base) -> int64_t {
        if (base + lane >= mine) return -1;
        const int tok = first_token(first + (base + lane) * n);
        const int32_t id = contiguous ? block0 : trow[tok / a.block_size];
        if (id < 0 || id >= a.num_blocks) {
            record_error(a.status, KVATTN_ERR_BAD_INDEX);
            return -1;
        }
        return ((int64_t)id * a.hkv + h) * a.block_size + tok % a.block_size;
    };
    // keys of the j-th tile of this warp that are seen (0 when its block id is bad)
    auto seen_of = [&](int j, int64_t row) -> uint32_t {
        return row < 0 ? 0u : seen_bits(first_token(first + j * n), pc, a);
    };
    int64_t rows = lookup(0);

    if constexpr (kKind != kF32Cache) {
        // the group's queries as B fragments: head g4, the dims in the order of K's chunks
        uint32_t q[kD / 16][2];
#pragma unroll
        for (int i = 0; i < kD / 16; ++i) q[i][0] = q[i][1] = 0u;
        if (g4 < G) {
            const __nv_bfloat16* qh = reinterpret_cast<const __nv_bfloat16*>(a.q) + q0 + g4 * kD;
            if constexpr (kKind == kBf16Cache) {
#pragma unroll
                for (int i = 0; i < kD / 32; ++i) {
                    const uint4 w = ldg16(qh + 8 * (q4 + 4 * i));
                    q[2 * i][0] = w.x;
                    q[2 * i][1] = w.y;
                    q[2 * i + 1][0] = w.z;
                    q[2 * i + 1][1] = w.w;
                }
            } else {  // scaled by 2^-4 into f16's range (the scores are scaled back)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint4 w = ldg16(qh + 16 * (q4 + 4 * (i >> 1)) + 8 * (i & 1));
                    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        q[2 * i + (j >> 1)][j & 1] = pack_f16_rn(bf16lo(u[j]) * 0.0625f, bf16hi(u[j]) * 0.0625f);
                }
            }
        }
        std::conditional_t<kKind == kFp8Cache, Fp8Softmax, Softmax> st;
        st.init();
        float o[kD / 16][4];  // unnormalised output
#pragma unroll
        for (int e = 0; e < kD / 16; ++e) o[e][0] = o[e][1] = o[e][2] = o[e][3] = 0.f;
        const float sl2 = a.scale_log2 * (kKind == kFp8Cache ? 16.f : 1.f);
        if constexpr (kKind == kBf16Cache) {
            Bf16Tile<kD> t;
            const char *kp = (const char*)a.k_pool, *vp = (const char*)a.v_pool;
            uint4 v[2][4][kD / 64];
            int64_t row = __shfl_sync(0xffffffffu, rows, 0);
            uint32_t seen = mine ? seen_of(0, row) : 0u;
            if (mine) {
                t.load_k(kp + row * (kD * 2), seen, g4, q4);
                t.load_v(v[0], vp + row * (kD * 2), seen, g4, q4);
            }
            auto step = [&](int j, const uint4 (&vnow)[4][kD / 64], uint4 (&vnext)[4][kD / 64]) {
                float s[4] = {0.f, 0.f, 0.f, 0.f};
                t.scores(s, q);
                // the next tile flies during this tile's softmax and P.V
                const uint32_t now = seen;
                if (j + 1 < mine) {
                    if (((j + 1) & 31) == 0) rows = lookup(j + 1);
                    row = __shfl_sync(0xffffffffu, rows, (j + 1) & 31);
                    seen = seen_of(j + 1, row);
                    t.load_k(kp + row * (kD * 2), seen, g4, q4);
                    t.load_v(vnext, vp + row * (kD * 2), seen, g4, q4);
                }
                const float x[4] = {now >> g4 & 1u ? s[0] * sl2 : -INFINITY, now >> g4 & 1u ? s[1] * sl2 : -INFINITY,
                                    now >> (g4 + 8) & 1u ? s[2] * sl2 : -INFINITY,
                                    now >> (g4 + 8) & 1u ? s[3] * sl2 : -INFINITY};
                float p[4];
                st.step(x, o, p);
                // P in bf16, the type of V that the MMA takes it with: off by at most
                // 2^-8 relative, at random; the sum adds the fp32 p
                t.add(vnow, o, movmatrix_trans(pack_bf16_rn(p[0], p[1])), movmatrix_trans(pack_bf16_rn(p[2], p[3])));
            };
            for (int j = 0; j < mine; j += 2) {
                step(j, v[0], v[1]);
                if (j + 1 < mine) step(j + 1, v[1], v[0]);
            }
        } else {
            const int rk0 = (g4 >> 1) * 4 + (g4 & 1), rk1 = rk0 + 2;
            const unsigned char* pool = (const unsigned char*)a.k_pool;
            unsigned char* ring = reinterpret_cast<unsigned char*>(row_of(warp, 0));
            uint32_t seen[kRing];  // of the pages under way, the next one first
            // page j on its way to its slot (one group of copies, empty past the last page)
            auto fetch = [&](int j) -> uint32_t {
                uint32_t bits = 0;
                if (j < mine) {
                    if (j > 0 && (j & 31) == 0) rows = lookup(j);
                    const int64_t row = __shfl_sync(0xffffffffu, rows, j & 31);
                    bits = seen_of(j, row);
                    // (of a bad block nothing is seen)
                    const unsigned char* src = pool + (row < 0 ? 0 : row) / kTile * kF8Page + 16 * lane;
                    const uint32_t dst = smem_addr(ring + j % kRing * kF8Page + 16 * lane);
#pragma unroll
                    for (int c = 0; c < kF8Page / 512; ++c) cp_async16(dst + 512 * c, src + 512 * c);
                    if (lane < kF8Page % 512 / 16) cp_async16(dst + kF8Page / 512 * 512, src + kF8Page / 512 * 512);
                }
                asm volatile("cp.async.commit_group;" ::: "memory");
                return bits;
            };
#pragma unroll
            for (int i = 0; i < kRing; ++i) seen[i] = fetch(i);
            for (int j = 0; j < mine; ++j) {
                asm volatile("cp.async.wait_group %0;" ::"n"(kRing - 1) : "memory");
                __syncwarp();  // every lane's copies of page j are there
                Fp8Tile t;
                t.load(ring + j % kRing * kF8Page, rk0, g4, q4);
                const uint32_t now = seen[0];
#pragma unroll
                for (int i = 0; i + 1 < kRing; ++i) seen[i] = seen[i + 1];
                __syncwarp();  // and every lane has read it
                seen[kRing - 1] = fetch(j + kRing);
                float s[4] = {0.f, 0.f, 0.f, 0.f};
                t.scores(s, q);
                const float k0 = t.ks[0] * sl2, k1 = t.ks[1] * sl2;
                const bool in0 = now >> rk0 & 1u, in1 = now >> rk1 & 1u;
                const float x[4] = {in0 ? s[0] * k0 : -INFINITY, in0 ? s[1] * k0 : -INFINITY,
                                    in1 ? s[2] * k1 : -INFINITY, in1 ? s[3] * k1 : -INFINITY};
                const float sv0 = in0 ? t.vs[0] : 0.f, sv1 = in1 ? t.vs[1] : 0.f;
                uint32_t vmask = 0xffffffffu;  // the bytes of this lane's words whose tokens are seen
                if (now != (1u << kTile) - 1u) {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (!(now >> (4 * q4 + i) & 1u)) vmask &= ~(0xffu << (8 * i));
                }
                float w[4];
                st.step(x, sv0, sv1, lane, [&](int i) { return t.v[i] & vmask; }, o, w);
                t.add(o, movmatrix_trans(pack_f16_rn(w[0], w[1])), movmatrix_trans(pack_f16_rn(w[2], w[3])), vmask);
            }
            asm volatile("cp.async.wait_group 0;" ::: "memory");
            __syncwarp();  // the outputs take the pages' place
        }
#pragma unroll
        for (int s = 4; s < 32; s <<= 1) {
            st.l[0] += __shfl_xor_sync(0xffffffffu, st.l[0], s);
            st.l[1] += __shfl_xor_sync(0xffffffffu, st.l[1], s);
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int g = 2 * q4 + e;
            if (g < G) {
                float* r = row_of(warp, g);
#pragma unroll
                for (int i = 0; i < kD / 16; ++i)
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        int d;
                        if constexpr (kKind == kBf16Cache) d = Bf16Tile<kD>::dim_of(i, half, g4);
                        else d = Fp8Tile::dim_of(i, half, g4);
                        if constexpr (kKind == kFp8Cache) r[d] = o[i][2 * half + e] * st.ref[e];
                        else r[d] = o[i][2 * half + e];
                    }
                if (g4 == 0) {
                    ml_of(warp, g)[0] = st.m[e];
                    ml_of(warp, g)[1] = st.l[e];
                }
            }
        }
    } else {
        // ---- fp32 cache, CUDA cores.  Scores: lane (g4, q4) holds tokens g4 and
        // g4 + 8, 16-byte chunks q4 + 4i; a quad's partial sums meet by shuffle.
        // P.V: a lane owns 4 dims of every (D = 128) or every other (D = 64)
        // token; the probabilities go through the warp's slot of shared memory.
        constexpr int kC = kD / 16;        // chunks per row and lane
        constexpr int kRep = 128 / kD;     // lanes that share a dim slice
        constexpr int kVR = kTile / kRep;  // tokens per lane
        const int dl = lane % (kD / 4), tr = lane / (kD / 4);
        const float* qs = reinterpret_cast<const float*>(a.q) + q0;
        float* pb = row_of(warp, 0);  // [token][kG], before the warp's output takes its place
        float o[kG][4], m[kG], l[kG];
#pragma unroll
        for (int g = 0; g < kG; ++g) {
            o[g][0] = o[g][1] = o[g][2] = o[g][3] = 0.f;
            m[g] = -INFINITY;
            l[g] = 0.f;
        }
        const uint4 none = make_uint4(0, 0, 0, 0);
        for (int j = 0; j < mine; ++j) {
            if (j > 0 && (j & 31) == 0) rows = lookup(j);
            const int64_t row = __shfl_sync(0xffffffffu, rows, j & 31);
            const uint32_t seen = seen_of(j, row);
            const char* kp = (const char*)a.k_pool + row * (kD * 4);
            const char* vp = (const char*)a.v_pool + row * (kD * 4);
            uint4 k[2][kC], v[kVR];
#pragma unroll
            for (int r = 0; r < 2; ++r)
#pragma unroll
                for (int i = 0; i < kC; ++i)
                    k[r][i] = seen >> (g4 + 8 * r) & 1u ? ldg16(kp + (g4 + 8 * r) * (kD * 4) + (q4 + 4 * i) * 16) : none;
#pragma unroll
            for (int t = 0; t < kVR; ++t)
                v[t] = seen >> (t * kRep + tr) & 1u ? ldg16(vp + (t * kRep + tr) * (kD * 4) + dl * 16) : none;
            float x[2][kG];
#pragma unroll
            for (int g = 0; g < kG; ++g) {
                float s0 = 0.f, s1 = 0.f;
#pragma unroll
                for (int i = 0; i < kC; ++i) {
                    const float4 w = __ldg(reinterpret_cast<const float4*>(qs + g * kD) + q4 + 4 * i);
                    const float* k0 = reinterpret_cast<const float*>(&k[0][i]);
                    const float* k1 = reinterpret_cast<const float*>(&k[1][i]);
                    s0 = fmaf(w.x, k0[0], fmaf(w.y, k0[1], fmaf(w.z, k0[2], fmaf(w.w, k0[3], s0))));
                    s1 = fmaf(w.x, k1[0], fmaf(w.y, k1[1], fmaf(w.z, k1[2], fmaf(w.w, k1[3], s1))));
                }
                s0 += __shfl_xor_sync(0xffffffffu, s0, 1);
                s1 += __shfl_xor_sync(0xffffffffu, s1, 1);
                s0 += __shfl_xor_sync(0xffffffffu, s0, 2);
                s1 += __shfl_xor_sync(0xffffffffu, s1, 2);
                x[0][g] = seen >> g4 & 1u ? s0 * a.scale_log2 : -INFINITY;
                x[1][g] = seen >> (g4 + 8) & 1u ? s1 * a.scale_log2 : -INFINITY;
            }
#pragma unroll
            for (int g = 0; g < kG; ++g) {
                float t = fmaxf(x[0][g], x[1][g]);
#pragma unroll
                for (int s = 4; s < 32; s <<= 1) t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, s));
                t = fmaxf(t, m[g]);
                const float f = m[g] == -INFINITY ? 0.f : exp2f(m[g] - t);
                m[g] = t;
                const float base = t == -INFINITY ? 0.f : t;
                x[0][g] = exp2f(x[0][g] - base);
                x[1][g] = exp2f(x[1][g] - base);
                l[g] = l[g] * f + (x[0][g] + x[1][g]);
                o[g][0] *= f;
                o[g][1] *= f;
                o[g][2] *= f;
                o[g][3] *= f;
                if (q4 == 0) {
                    pb[g4 * kG + g] = x[0][g];
                    pb[(g4 + 8) * kG + g] = x[1][g];
                }
            }
            __syncwarp();
#pragma unroll
            for (int t = 0; t < kVR; ++t) {
                const float* vv = reinterpret_cast<const float*>(&v[t]);
#pragma unroll
                for (int g = 0; g < kG; ++g) {
                    const float p = pb[(t * kRep + tr) * kG + g];
                    o[g][0] = fmaf(p, vv[0], o[g][0]);
                    o[g][1] = fmaf(p, vv[1], o[g][1]);
                    o[g][2] = fmaf(p, vv[2], o[g][2]);
                    o[g][3] = fmaf(p, vv[3], o[g][3]);
                }
            }
            __syncwarp();
        }
#pragma unroll
        for (int g = 0; g < kG; ++g) {
#pragma unroll
            for (int s = 4; s < 32; s <<= 1) l[g] += __shfl_xor_sync(0xffffffffu, l[g], s);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (kRep == 2) o[g][i] += __shfl_xor_sync(0xffffffffu, o[g][i], 16);
            if (tr == 0) *reinterpret_cast<float4*>(row_of(warp, g) + 4 * dl) = make_float4(o[g][0], o[g][1], o[g][2], o[g][3]);
            if (lane == 0) {
                ml_of(warp, g)[0] = m[g];
                ml_of(warp, g)[1] = l[g];
            }
        }
    }
    __syncthreads();

    // ---- the warps' states, then the CTAs', kV dims a thread: four, or one where
    // that leaves most threads idle (12 heads of 64 without groups, fp32, 8
    // sequences, window 256: 4.3 us, with four 4.45)
    constexpr int kV = kKind == kF32Cache && kG * kD <= 128 ? 1 : 4;
    struct Dims {
        float v[kV];
    };
    auto read = [](const float* p) {
        Dims o;
        if constexpr (kV == 4) {
            const float4 x = *reinterpret_cast<const float4*>(p);
            o.v[0] = x.x;
            o.v[1] = x.y;
            o.v[2] = x.z;
            o.v[3] = x.w;
        } else {
            o.v[0] = *p;
        }
        return o;
    };
    auto write = [](float* p, const Dims& o) {
        if constexpr (kV == 4) *reinterpret_cast<float4*>(p) = make_float4(o.v[0], o.v[1], o.v[2], o.v[3]);
        else *p = o.v[0];
    };
    auto store = [&](int e, Dims num, float den) {
        const float inv = den == 0.f ? 0.f : 1.f / den;
#pragma unroll
        for (int i = 0; i < kV; ++i) num.v[i] *= inv;
        if constexpr (kKind == kF32Cache)
            write(reinterpret_cast<float*>(a.out) + q0 + e, num);
        else
            *reinterpret_cast<uint2*>(reinterpret_cast<__nv_bfloat16*>(a.out) + q0 + e) =
                make_uint2(pack_bf16_rn(num.v[0], num.v[1]), pack_bf16_rn(num.v[2], num.v[3]));
    };
    // The merge of `n` states (at most 8, their loads under way together): outputs
    // at row(i), (max, sum) at stat(i).
    auto merge = [&](int n, auto row, auto stat, Dims& num, float& M, float& den) {
        float2 s[8];
        Dims o[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            s[i] = make_float2(-INFINITY, 0.f);
            if (i < n) {
                s[i] = *reinterpret_cast<const float2*>(stat(i));
                o[i] = read(row(i));
            }
        }
        M = -INFINITY;
#pragma unroll
        for (int i = 0; i < 8; ++i) M = fmaxf(M, s[i].x);
#pragma unroll
        for (int k = 0; k < kV; ++k) num.v[k] = 0.f;
        den = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (i < n && s[i].y != 0.f) {  // a state without a key has no weight (one whose scores are NaN has a sum of NaN)
                const float f = exp2f(s[i].x - M);
#pragma unroll
                for (int k = 0; k < kV; ++k) num.v[k] += f * o[i].v[k];
                den += f * s[i].y;
            }
        }
    };
    for (int e = kV * tid; e < G * kD; e += kV * blockDim.x) {
        const int g = e / kD, d = e - g * kD;
        Dims num;
        float M, den;
        merge(warps, [&](int w) { return row_of(w, g) + d; }, [&](int w) { return ml_of(w, g); }, num, M, den);
        if (cluster == 1) {
            store(e, num, den);
        } else {
            write(row_of(warps, g) + d, num);
            if (d == 0) *reinterpret_cast<float2*>(ml_of(warps, g)) = make_float2(M, den);
        }
    }
    if (cluster > 1) {
        cg::cluster_group cl = cg::this_cluster();
        cl.sync();
        for (int e = kV * (rank * blockDim.x + tid); e < G * kD; e += kV * n * 32) {
            const int g = e / kD, d = e - g * kD;
            Dims num;
            float M, den;
            merge(cluster, [&](int r) { return cl.map_shared_rank(row_of(warps, g) + d, r); },
                  [&](int r) { return cl.map_shared_rank(ml_of(warps, g), r); }, num, M, den);
            store(e, num, den);
        }
        cl.sync();  // the others' shared memory stays until it has been read
    }
}

// How many clusters of a size are resident at once, per device (a pure function of
// the kernel, its block, which is of 8 warps wherever clusters are, and its shared
// memory; asking the runtime takes longer than a launch).  Clusters do not cross the
// GPU's groups of SMs, so these are fewer than the SMs' CTAs over the size: of 8 CTAs
// at one per SM 15, where 152 / 8 is 19.
class ClusterResidency {
public:
    template <typename Kernel>
    int query(Kernel kern, const cudaLaunchConfig_t& cfg, int log2_size)
    {
        int dev = 0;
        if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
        std::lock_guard<std::mutex> g(mu_);
        Entry& e = kept_[dev][log2_size];
        if (e.bytes != (int)cfg.dynamicSmemBytes) {
            int n = 0;
            if (cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess) {
                (void)cudaGetLastError();
                return 0;
            }
            e.bytes = (int)cfg.dynamicSmemBytes;
            e.clusters = n;
        }
        return e.clusters;
    }

private:
    struct Entry {
        int bytes, clusters;
    };
    std::mutex mu_;
    Entry kept_[64][4] = {};
};

// False, with nothing launched, where the balanced stream is the faster one.
template <int kKind, int kD, int kG>
bool run_direct(const DecodeArgs& a, int max_tiles, int warps, int cluster, cudaStream_t s, kvattn_status* st)
{
    auto kern = decode_direct_kernel<kKind, kD, kG>;
    const int G = a.hq / a.hkv, bytes = direct_floats(kKind, warps, G, kD) * 4;
    static SmemLimit limit;
    if (limit.ensure(reinterpret_cast<const void*>(kern), bytes) != cudaSuccess) {
        *st = KVATTN_ERR_CUDA;
        return true;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(warps * 32);
    cfg.dynamicSmemBytes = bytes;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    // half the CTAs per segment rather than a second wave of clusters (bf16 D = 128,
    // 16 segments of 32768 keys: in clusters of 8 98.9 us, of 4 88.7)
    static ClusterResidency resident;
    for (; cluster > 1; cluster /= 2) {
        attr[1].val.clusterDim.x = cluster;
        cfg.gridDim = dim3((unsigned)(a.batch * a.hkv * cluster));
        cfg.numAttrs = 2;
        if (resident.query(kern, cfg, cluster == 8 ? 3 : cluster == 4 ? 2 : 1) >= a.batch * a.hkv) break;
    }
    // Clusters that leave warps' places empty, with many bytes a warp: the stream,
    // which cuts segments anywhere, fills them once there are 16 segments (at most
    // 16 pieces each).  Measured (us, this and the stream): bf16 D = 128 without
    // groups, 38 segments of 16384 keys 88.7 / 68.3, groups of 4, 16 of 32768 88.7 /
    // 78.5; fp32 groups of 4, 16 of 16384 84.6 / 68.3, 38 of 4096 53.9 / 45.7.  With
    // fewer segments it loses (bf16, 8 of 32768 51.8 / 78.5, 15 62.1 / 78.5), with
    // half the bf16 keys it gains little or loses (groups of 4, 16 of 16384 51.8 /
    // 49.8, repeated calls 41.1 / 46.6), and it always does with fp8 pages and bf16 D
    // = 64 (16 of 32768 66.2 / 86.7 and 47.7 / 72.3).
    if constexpr (kKind == kF32Cache || (kKind == kBf16Cache && kD == 128)) {
        const int64_t segs = (int64_t)a.batch * a.hkv, places = (int64_t)num_sms() * warps_per_sm(kKind, kD, G);
        const int64_t per_warp = (int64_t)max_tiles * 2 * kTile * kD * (kKind == kF32Cache ? 4 : 2) / (cluster * warps);
        const int64_t many = (kKind == kF32Cache ? 256 : 512) << 10;
        if (segs >= 16 && segs * cluster * warps * 10 < places * 7 && per_warp >= many) return false;
    }
    cfg.gridDim = dim3((unsigned)(a.batch * a.hkv * cluster));
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    *st = cuda_status(cudaLaunchKernelEx(&cfg, kern, a, cluster));
    return true;
}

bool direct_dispatch(const DecodeArgs& a, int max_tiles, int warps, int cluster, cudaStream_t s, kvattn_status* st)
{
    if (a.fp8) return run_direct<kFp8Cache, 128, 8>(a, max_tiles, warps, cluster, s, st);
    if (a.dtype == KVATTN_BF16)
        return a.d == 128 ? run_direct<kBf16Cache, 128, 8>(a, max_tiles, warps, cluster, s, st)
                          : run_direct<kBf16Cache, 64, 8>(a, max_tiles, warps, cluster, s, st);
    switch (a.hq / a.hkv) {
#define KVATTN_DIRECT_F32(GG)                                                                   \
    case GG:                                                                                    \
        return a.d == 128 ? run_direct<kF32Cache, 128, GG>(a, max_tiles, warps, cluster, s, st) \
                          : run_direct<kF32Cache, 64, GG>(a, max_tiles, warps, cluster, s, st);
        KVATTN_DIRECT_F32(1)
        KVATTN_DIRECT_F32(2)
        KVATTN_DIRECT_F32(4)
        KVATTN_DIRECT_F32(8)
#undef KVATTN_DIRECT_F32
    }
    return false;
}

}  // namespace

bool launch_decode_direct(const DecodeArgs& a, int32_t max_tiles, cudaStream_t s, kvattn_status* st)
{
    const int kind = a.fp8 ? kFp8Cache : a.dtype == KVATTN_BF16 ? kBf16Cache : kF32Cache;
    const int G = a.hq / a.hkv;
    const int64_t segs = (int64_t)a.batch * a.hkv, tiles = segs * max_tiles;
    // Where the balanced stream of decode_kernel.cuh is faster: long calls of
    // many keys.  Measured (us, this and the stream; thousands of tiles): bf16
    // D = 128 17 27 / 32, 66 88 / 90, 264 343 / 324; fp32 groups of 4 4.2 13.4 /
    // 20.6, 16 49 / 48, 66 171 / 160; bf16 D = 64 264 165 / 307 and fp32 without
    // groups 264 574 / 608, so these come here at any length (run_direct refuses the
    // rest).  fp8 pages stream as fast from here (17 13.9 / 26.0, 66 47 / 59, 264 172
    // / 195, 526 330 / 364) and lose only where a long sequence among short ones keeps
    // its few warps busy (64 sequences of 1 to 32768 tokens, windows of 8192 and
    // 16384: 162 / 179 and 304 / 286).
    int64_t most = INT64_MAX;
    if (kind == kF32Cache) most = G == 1 ? most : 16384;
    else if (kind == kFp8Cache) most = max_tiles <= 512 + 2 ? most : 65536;  // (a window of 8192 and a few sinks)
    else if (a.d == 128) most = 65536;
    if (tiles > most || segs * 8 > INT32_MAX) return false;
    // One wave of warps: the most warps per CTA that let every segment be
    // resident (a quarter of the SM's when not even that does), at most 8;
    // then CTAs per segment, a cluster as large as lets them be resident (run_direct
    // has the last word); but no warp without a tile, and no second CTA for
    // fewer than 4 tiles per warp, which cost less than the cluster's launch and
    // merge (18 tiles: 8 sequences of 12 fp32 heads of 64 4.4 us in one CTA and
    // 5.25 in two, 1 of 32 / 8 fp8 heads 5.1 and 5.3, of bf16 4.9 and 4.95).
    const int cap = warps_per_sm(kind, a.d, G);
    const int64_t sms = num_sms();
    int warps = 8;
    while (warps > cap / 4 && sms * (cap / warps) < segs) --warps;
    int cluster = 1;
    while (max_tiles >= 32 && cluster < 8 && warps == 8 && sms * (cap / 8) >= 2 * cluster * segs && 16 * cluster <= max_tiles) cluster *= 2;
    warps = std::min(warps, max_tiles);
    return direct_dispatch(a, max_tiles, warps, cluster, s, st);
}

}  // namespace kvattn
