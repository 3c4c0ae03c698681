// One warp's work on 16 tokens of a bf16 cache with mma.sync, straight from global
// memory, and its softmax state.
#pragma once

#include "fast_exp2.cuh"
#include "kvattn_tc.cuh"

namespace kvattn {
namespace {

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

}  // namespace
}  // namespace kvattn
