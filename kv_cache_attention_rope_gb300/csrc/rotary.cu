// Rotary position embedding in the forms rope_append does not have (pairs of
// the two halves, part of the head, speeds scaled for long contexts), fused
// with the KV-cache append.
//
// What it computes: with R rotated dims, n = R / 2 pairs and pair i turning by
// f_i radians per position (kvattn_rotary_append in kvattn.h states f_i), the
// pair (x0, x1) of a token at position m becomes
//     y0 = a (x0 cos(m f_i) - x1 sin(m f_i)),  y1 = a (x0 sin(m f_i) + x1 cos(m f_i))
// where (x0, x1) = (x[i], x[i + n]) (half layout) or (x[2i], x[2i+1])
// (adjacent); dims R .. D-1 are copied.  "Tokenizer, KV Cache and RoPE" page,
// section 4 (the rotation); "From-scratch AI inference engine" page, section
// 3.2 (k and v go to the cache index equal to the position).
//
// How: the op moves 2 (Hq + 2 Hkv) D elements per token and computes little,
// so it is bound by HBM.  A unit is two 16-byte vectors of one head whose
// elements pair up with each other (half) or inside themselves (adjacent):
// units u < R / (2 kEPV) turn with pairs kEPV u .. kEPV u + kEPV - 1 in either
// layout, the others are copied.  A thread keeps one unit index and walks the
// heads, so it reads its kEPV twiddles once per token.
//
// Rounding.  The speed of a pair is a 64-bit fixed-point count of turns per
// position, so position * speed mod 2^64 is the angle's fraction of a turn
// whatever the position; the nearest quarter turn comes off exactly and the
// rest (at most 1/8 turn, rounded to fp32: 2^-25 relative) goes through
// sincospif.  Products and sums are fp32, each stored value rounded once:
// within half an ulp of the stored type plus 2^-21 a (|x0| + |x1|) of exact.
#include <algorithm>

#include "kvattn_internal.cuh"

namespace kvattn {
namespace {

constexpr int kThreads = 128;
constexpr int kFlight = 3;  // units a thread loads before it waits for its twiddles

// (cos, sin) of u * 2^-64 turns.
__device__ __forceinline__ float2 twiddle(uint64_t u)
{
    const uint32_t quad = (uint32_t)((u + (1ull << 61)) >> 62);
    const int64_t r = (int64_t)(u - ((uint64_t)quad << 62));  // [-2^61, 2^61): at most 1/8 turn
    float s, c;
    sincospif((float)r * 0x1p-63f, &s, &c);
    switch (quad & 3u) {
        case 0: return make_float2(c, s);
        case 1: return make_float2(-s, c);
        case 2: return make_float2(-c, -s);
        default: return make_float2(s, -c);
    }
}

// Two vectors of a rotated unit in place: c2[i], s2[i] hold the twiddles of
// pairs 2i and 2i + 1 of the unit, packed.
template <bool kBF16, bool kHalf>
__device__ __forceinline__ void turn(uint4& va, uint4& vb, const uint64_t* c2, const uint64_t* s2)
{
    uint32_t* a = reinterpret_cast<uint32_t*>(&va);
    uint32_t* b = reinterpret_cast<uint32_t*>(&vb);
    const uint64_t neg = 0x8000000080000000ull;
    if constexpr (kBF16) {
        if constexpr (kHalf) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint64_t x0 = pk(bf16lo(a[i]), bf16hi(a[i])), x1 = pk(bf16lo(b[i]), bf16hi(b[i]));
                const uint64_t y0 = ffma2(x1, s2[i] ^ neg, fmul2(x0, c2[i]));
                const uint64_t y1 = ffma2(x1, c2[i], fmul2(x0, s2[i]));
                a[i] = pack_bf16_rn(pk_lo(y0), pk_hi(y0));
                b[i] = pack_bf16_rn(pk_lo(y1), pk_hi(y1));
            }
        } else {
            // words 2i, 2i + 1 of the unit are its pairs 2i, 2i + 1
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                uint32_t& w0 = i < 2 ? a[2 * i] : b[2 * i - 4];
                uint32_t& w1 = i < 2 ? a[2 * i + 1] : b[2 * i - 3];
                const uint64_t x0 = pk(bf16lo(w0), bf16lo(w1)), x1 = pk(bf16hi(w0), bf16hi(w1));
                const uint64_t y0 = ffma2(x1, s2[i] ^ neg, fmul2(x0, c2[i]));
                const uint64_t y1 = ffma2(x1, c2[i], fmul2(x0, s2[i]));
                w0 = pack_bf16_rn(pk_lo(y0), pk_lo(y1));
                w1 = pack_bf16_rn(pk_hi(y0), pk_hi(y1));
            }
        }
    } else {
        float* fa = reinterpret_cast<float*>(&va);
        float* fb = reinterpret_cast<float*>(&vb);
#pragma unroll
        for (int i = 0; i < 2; ++i) {  // pairs 2i, 2i + 1 of the unit
            float& p0 = kHalf ? fa[2 * i] : (i ? fb[0] : fa[0]);
            float& p1 = kHalf ? fb[2 * i] : (i ? fb[1] : fa[1]);
            float& q0 = kHalf ? fa[2 * i + 1] : (i ? fb[2] : fa[2]);
            float& q1 = kHalf ? fb[2 * i + 1] : (i ? fb[3] : fa[3]);
            const uint64_t x0 = pk(p0, q0), x1 = pk(p1, q1);
            const uint64_t y0 = ffma2(x1, s2[i] ^ neg, fmul2(x0, c2[i]));
            const uint64_t y1 = ffma2(x1, c2[i], fmul2(x0, s2[i]));
            p0 = pk_lo(y0);
            q0 = pk_hi(y0);
            p1 = pk_lo(y1);
            q1 = pk_hi(y1);
        }
    }
}

// Largest magnitude of the 8 bf16 values of v.
__device__ __forceinline__ float amax8(const uint4& v)
{
    const uint32_t* w = reinterpret_cast<const uint32_t*>(&v);
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) m = fmaxf(m, fmaxf(fabsf(bf16lo(w[i])), fabsf(bf16hi(w[i]))));
    return m;
}

// e4m3 codes of the 8 bf16 values of v times inv (fp32, RN), RN, saturating.
__device__ __forceinline__ uint2 codes8(const uint4& v, float inv)
{
    const uint32_t* w = reinterpret_cast<const uint32_t*>(&v);
    uint32_t c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        c[i] = __nv_cvt_float2_to_fp8x2(make_float2(__fmul_rn(bf16lo(w[i]), inv), __fmul_rn(bf16hi(w[i]), inv)),
                                        __NV_SATFINITE, __NV_E4M3);
    return make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
}

// One token per CTA.
template <bool kBF16, int kD, bool kHalf, bool kFP8>
__global__ void __launch_bounds__(kThreads) rotary_append_kernel(const __grid_constant__ RotaryArgs a)
{
    pdl_wait();
    constexpr int kE = kBF16 ? 2 : 4;
    constexpr int kEPV = 16 / kE;              // elements per 16-byte vector
    constexpr int kU = kD / (2 * kEPV);        // units per head
    constexpr int kGroups = kThreads / kU;     // heads in flight
    constexpr int kVPH = kD / kEPV;            // vectors per head
    static_assert(!kFP8 || (kBF16 && kD == 128), "fp8 pages hold D = 128 rows quantised from bf16");
    __shared__ __align__(16) float2 tw[kD / 2];

    const int t = blockIdx.x, tid = threadIdx.x;
    const int u = tid % kU, hg = tid / kU;
    const bool rot = u < a.rot / (2 * kEPV);
    // element offsets of the unit's two vectors in a head
    const int ea = kHalf && rot ? u * kEPV : 2 * u * kEPV;
    const int eb = kHalf && rot ? a.rot / 2 + u * kEPV : 2 * u * kEPV + kEPV;
    const int heads = a.hq + a.hkv;            // q heads, then k heads
    const char* qrow = (const char*)a.q + t * a.q_stride;
    const char* krow = (const char*)a.k + t * a.k_stride;
    const char* vrow = (const char*)a.v + t * a.v_stride;
    const int nvec = kFP8 ? 0 : a.hkv * kVPH;  // v vectors of the token (an fp8 cache's V has its own kernel)

    auto load = [&](int hh, uint4& x, uint4& y) {
        const char* row = hh < a.hq ? qrow + hh * (kD * kE) : krow + (hh - a.hq) * (kD * kE);
        x = *reinterpret_cast<const uint4*>(row + ea * kE);
        y = *reinterpret_cast<const uint4*>(row + eb * kE);
    };
    uint4 xa[kFlight], xb[kFlight], xv = make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int i = 0; i < kFlight; ++i)
        if (hg + i * kGroups < heads) load(hg + i * kGroups, xa[i], xb[i]);
    if (tid < nvec) xv = *reinterpret_cast<const uint4*>(vrow + tid * 16);

    const int pos = a.positions[t], seq = a.seq_ids[t];
    bool ok = pos >= 0 && seq >= 0 && seq < a.num_seqs && pos / a.block_size < a.max_blocks;
    int64_t blk = -1;
    if (ok) {
        blk = a.block_table[(int64_t)seq * a.max_blocks + pos / a.block_size];
        ok = blk >= 0 && blk < a.num_blocks;
    }
    if (!ok) {  // the same for every thread
        if (tid == 0) record_error(a.status, KVATTN_ERR_BAD_INDEX);
        return;
    }
    const int off = pos % a.block_size;
    if (tid < a.rot / 2) {
        const float2 w = twiddle((uint64_t)(uint32_t)pos * a.turns[tid]);
        tw[tid] = make_float2(w.x * a.amplitude, w.y * a.amplitude);
    }
    __syncthreads();
    uint64_t c2[kEPV / 2], s2[kEPV / 2];
#pragma unroll
    for (int i = 0; i < kEPV / 2; ++i) {
        if (rot) {
            const float4 w = *reinterpret_cast<const float4*>(&tw[u * kEPV + 2 * i]);
            c2[i] = pk(w.x, w.z);
            s2[i] = pk(w.y, w.w);
        }
    }

    auto finish = [&](int hh, uint4 x, uint4 y) {
        if (rot) turn<kBF16, kHalf>(x, y, c2, s2);
        if (hh < a.hq) {
            char* row = (char*)a.q_out + t * a.q_out_stride + hh * (kD * kE);
            *reinterpret_cast<uint4*>(row + ea * kE) = x;
            *reinterpret_cast<uint4*>(row + eb * kE) = y;
        } else if constexpr (kFP8) {
            // scale = amax / 448 over the head row; its kU lanes are neighbours
            const unsigned mask = ((1u << kU) - 1u) << (threadIdx.x & 31u & ~(unsigned)(kU - 1));
            float m = fmaxf(amax8(x), amax8(y));
#pragma unroll
            for (int o = 1; o < kU; o <<= 1) m = fmaxf(m, __shfl_xor_sync(mask, m, o));
            const float inv = m > 0.f ? __fdiv_rn(448.f, m) : 1.f;
            const int pages = a.block_size / 16, r = off & 15;
            unsigned char* pg = (unsigned char*)a.k_pool +
                                ((blk * a.hkv + (hh - a.hq)) * pages + off / 16) * (int64_t)kF8Page;
            // dims 8 dv .. 8 dv + 7: half a 16-byte chunk (layout: kF8Page)
            auto put = [&](int dv, const uint4& v) {
                *reinterpret_cast<uint2*>(pg + r * 128 + (((dv >> 1) ^ f8_swz(r)) << 4) + (dv & 1) * 8) = codes8(v, inv);
            };
            put(ea / 8, x);
            put(eb / 8, y);
            if (u == 0) reinterpret_cast<float*>(pg + kF8KsOff)[r] = m > 0.f ? __fdiv_rn(m, 448.f) : 1.f;
        } else {
            char* row = (char*)a.k_pool + ((blk * a.hkv + (hh - a.hq)) * a.block_size + off) * (int64_t)(kD * kE);
            *reinterpret_cast<uint4*>(row + ea * kE) = x;
            *reinterpret_cast<uint4*>(row + eb * kE) = y;
        }
    };
    auto put_v = [&](int j, const uint4& x) {
        char* row = (char*)a.v_pool + ((blk * a.hkv + j / kVPH) * a.block_size + off) * (int64_t)(kD * kE);
        *reinterpret_cast<uint4*>(row + (j % kVPH) * 16) = x;
    };
    for (int h0 = hg; h0 < heads; h0 += kFlight * kGroups) {
        if (h0 != hg) {
#pragma unroll
            for (int i = 0; i < kFlight; ++i)
                if (h0 + i * kGroups < heads) load(h0 + i * kGroups, xa[i], xb[i]);
        }
#pragma unroll
        for (int i = 0; i < kFlight; ++i)
            if (h0 + i * kGroups < heads) finish(h0 + i * kGroups, xa[i], xb[i]);
    }
    if (tid < nvec) put_v(tid, xv);
    for (int j = tid + kThreads; j < nvec; j += kThreads) put_v(j, *reinterpret_cast<const uint4*>(vrow + j * 16));
}

template <bool kBF16, int kD, bool kFP8>
kvattn_status launch(const RotaryArgs& a, cudaStream_t s)
{
    const cudaError_t e = a.half ? launch_pdl(rotary_append_kernel<kBF16, kD, true, kFP8>, dim3(a.num_tokens),
                                              dim3(kThreads), 0, s, a)
                                 : launch_pdl(rotary_append_kernel<kBF16, kD, false, kFP8>, dim3(a.num_tokens),
                                              dim3(kThreads), 0, s, a);
    return cuda_status(e);
}

}  // namespace

kvattn_status launch_rotary_append(const RotaryArgs& a, cudaStream_t s)
{
    if (a.fp8) {
        if (a.dtype != KVATTN_BF16 || a.d != 128) return KVATTN_ERR_UNSUPPORTED;
        return launch<true, 128, true>(a, s);
    }
    const bool bf16 = a.dtype == KVATTN_BF16;
    if (a.d == 128) return bf16 ? launch<true, 128, false>(a, s) : launch<false, 128, false>(a, s);
    if (a.d == 64) return bf16 ? launch<true, 64, false>(a, s) : launch<false, 64, false>(a, s);
    return KVATTN_ERR_UNSUPPORTED;
}

}  // namespace kvattn
