// One warp's work on an fp8 page with mma.sync: operands, and the softmax state whose
// reference follows weight times V scale.
#pragma once

#include "fast_exp2.cuh"
#include "kvattn_tc.cuh"

namespace kvattn {
namespace {

// In the place of a token's V scale: its page is not there, and the token not seen.  A NaN of a payload that no
// arithmetic gives.  It is met where scales are looked at, so it costs nothing elsewhere (a flag per page of the
// balanced stream, loaded besides: 1.5 % of 64 sequences of up to 32768 tokens, a compare per token 2.7 %).
constexpr uint32_t kNoPage = 0x7fc0deadu;

// max(a, b), NaN if either is.
__device__ __forceinline__ float max_nan(float a, float b)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// Softmax state of a warp over fp8 pages, windowed form: of query heads 2 q4 and
// 2 q4 + 1 the running maximum (log2 units), the sum, and the reference that the
// output o is in units of.  P goes into the MMA in f16 as weight * V scale /
// reference.  The reference follows that product, not the scale, so that a token
// of large V and no weight leaves the others their bits, and a row of zeros, which
// is stored with the scale 1, does not count.  f16 rounds each product within
// 2^-11 relative, or 2^-25 of the head's largest.
struct Fp8Softmax {
    static constexpr float kLeast = 0x1p-100f;  // of a reference: its inverse is finite
    float m[2], l[2], ref[2], rinv[2];
    float scale16;  // 16 times the smaller reference
    __device__ __forceinline__ void init()
    {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            m[e] = -INFINITY;
            l[e] = ref[e] = rinv[e] = 0.f;
        }
        scale16 = 0.f;
    }
    // One tile: scores x of this lane's tokens rk0 and rk1 ((rk0, head 0), (rk0,
    // 1), (rk1, 0), (rk1, 1)), their V scales sv0 and sv1 (0: not seen), word(i)
    // the lane's i-th word of V codes (tokens 4 q4 .. 4 q4 + 3).  Gives the
    // products w for P.V and rescales o.  The maximum is raised when a score
    // exceeds it by more than 2^8.  A V scale over 16 times a reference has the
    // products looked at, and the reference raised to one that is; so w stays
    // within 2^12.  The warp agrees on these only then, and (kMissing) only then finds tokens
    // of kNoPage, whose x it sets; V's codes of those are finite.
    template <bool kMissing = false, int kN, typename Word>
    __device__ __forceinline__ void step(float (&x)[4], float sv0, float sv1, int lane, Word word, float (&o)[kN][4],
                                         float (&w)[4])
    {
        float l0 = fmaxf(x[0], x[2]), l1 = fmaxf(x[1], x[3]);
        const bool raise = l0 > m[0] + 8.f || l1 > m[1] + 8.f ||
                           (kMissing ? !(max_nan(sv0, sv1) <= scale16) : fmaxf(sv0, sv1) > scale16);
        float p[4];
        auto weigh = [&] {
            // a head whose scores are all -inf so far has no weight yet
            const float m0 = m[0] == -INFINITY ? 0.f : m[0], m1 = m[1] == -INFINITY ? 0.f : m[1];
            p[0] = fast_exp2(x[0] - m0);
            p[1] = fast_exp2(x[1] - m1);
            p[2] = fast_exp2(x[2] - m0);
            p[3] = fast_exp2(x[3] - m1);
        };
        if (__any_sync(0xffffffffu, raise)) {
            if constexpr (kMissing) {
                if (__float_as_uint(sv0) == kNoPage) {
                    x[0] = x[1] = -INFINITY;
                    sv0 = 0.f;
                }
                if (__float_as_uint(sv1) == kNoPage) {
                    x[2] = x[3] = -INFINITY;
                    sv1 = 0.f;
                }
                l0 = fmaxf(x[0], x[2]);
                l1 = fmaxf(x[1], x[3]);
            }
            if (__any_sync(0xffffffffu, sv0 == 1.f || sv1 == 1.f)) {  // rows of zeros?
                uint32_t any = 0;
#pragma unroll
                for (int i = 0; i < 16; ++i) any |= word(i) & 0x7f7f7f7fu;
#pragma unroll
                for (int s = 4; s < 32; s <<= 1) any |= __shfl_xor_sync(0xffffffffu, any, s);
                const int g4 = lane >> 2;  // rk0 = 4 (g4 / 2) + g4 % 2, rk1 = rk0 + 2
                any = __shfl_sync(0xffffffffu, any, g4 >> 1) >> (8 * (g4 & 1));
                if (sv0 == 1.f && (any & 0xffu) == 0u) sv0 = 0.f;
                if (sv1 == 1.f && (any & 0xff0000u) == 0u) sv1 = 0.f;
            }
#pragma unroll
            for (int s = 4; s < 32; s <<= 1) {
                l0 = fmaxf(l0, __shfl_xor_sync(0xffffffffu, l0, s));
                l1 = fmaxf(l1, __shfl_xor_sync(0xffffffffu, l1, s));
            }
            const float top[2] = {l0, l1};
#pragma unroll
            for (int e = 0; e < 2; ++e)
                if (top[e] > m[e] + 8.f) {  // (-inf: nothing before)
                    const float f = m[e] == -INFINITY ? 0.f : fast_exp2(m[e] - top[e]);
                    l[e] *= f;
                    ref[e] *= f;
                    m[e] = top[e];
                }
            weigh();
            float most[2] = {fmaxf(p[0] * sv0, p[2] * sv1), fmaxf(p[1] * sv0, p[3] * sv1)};
            float f[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
#pragma unroll
                for (int s = 4; s < 32; s <<= 1) most[e] = fmaxf(most[e], __shfl_xor_sync(0xffffffffu, most[e], s));
                const float r = fmaxf(most[e] > ref[e] * 16.f ? most[e] : ref[e], kLeast);
                f[e] = ref[e] / r;
                ref[e] = r;
                rinv[e] = 1.f / r;
            }
            scale16 = 16.f * fminf(ref[0], ref[1]);
#pragma unroll
            for (int i = 0; i < kN; ++i) {
                o[i][0] *= f[0];
                o[i][1] *= f[1];
                o[i][2] *= f[0];
                o[i][3] *= f[1];
            }
        } else {
            weigh();
        }
        l[0] += p[0] + p[2];
        l[1] += p[1] + p[3];
        w[0] = p[0] * sv0 * rinv[0];
        w[1] = p[1] * sv0 * rinv[1];
        w[2] = p[2] * sv1 * rinv[0];
        w[3] = p[3] * sv1 * rinv[1];
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

}  // namespace
}  // namespace kvattn
