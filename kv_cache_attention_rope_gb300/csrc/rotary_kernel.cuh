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
// elements pair up with each other (half layout), or two vectors that hold their
// pairs (adjacent); vectors past R are copied.  A thread keeps one unit index and
// walks the heads, so it reads its twiddles once per token.
//
// Rounding.  The speed of a pair is a 64-bit fixed-point count of turns per
// position, so position * speed mod 2^64 is the angle's fraction of a turn
// whatever the position; the nearest quarter turn comes off exactly and the
// rest (at most 1/8 turn, rounded to fp32: 2^-25 relative) goes through
// sincospif.  Products and sums are fp32, each stored value rounded once:
// within half an ulp of the stored type plus 2^-21 a (|x0| + |x1|) of exact.
//
// With several axes (kAxes): the pair turns by the position on its axis, and k
// and v go to a slot of their own.
#pragma once

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

// Packed twiddles: c[i], s[i] are the cosines and sines of pairs 2i and 2i + 1.
template <int kN>
struct Twiddles {
    uint64_t c[kN / 2], s[kN / 2];
    __device__ __forceinline__ void load(const float2* tw)  // kN pairs
    {
#pragma unroll
        for (int i = 0; i < kN / 2; ++i) {
            const float4 w = *reinterpret_cast<const float4*>(tw + 2 * i);
            c[i] = pk(w.x, w.z);
            s[i] = pk(w.y, w.w);
        }
    }
};
__device__ __forceinline__ void turn2(uint64_t x0, uint64_t x1, uint64_t c, uint64_t s, uint64_t& y0, uint64_t& y1)
{
    y0 = ffma2(x1, s ^ 0x8000000080000000ull, fmul2(x0, c));
    y1 = ffma2(x1, c, fmul2(x0, s));
}

// Half layout: element e of va pairs with element e of vb.
template <bool kBF16>
__device__ __forceinline__ void turn_half(uint4& va, uint4& vb, const uint64_t* c, const uint64_t* s)
{
    uint32_t* a = reinterpret_cast<uint32_t*>(&va);
    uint32_t* b = reinterpret_cast<uint32_t*>(&vb);
    uint64_t y0, y1;
    if constexpr (kBF16) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            turn2(pk(bf16lo(a[i]), bf16hi(a[i])), pk(bf16lo(b[i]), bf16hi(b[i])), c[i], s[i], y0, y1);
            a[i] = pack_bf16_rn(pk_lo(y0), pk_hi(y0));
            b[i] = pack_bf16_rn(pk_lo(y1), pk_hi(y1));
        }
    } else {
        uint64_t* a2 = reinterpret_cast<uint64_t*>(&va);
        uint64_t* b2 = reinterpret_cast<uint64_t*>(&vb);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            turn2(a2[i], b2[i], c[i], s[i], y0, y1);
            a2[i] = y0;
            b2[i] = y1;
        }
    }
}

// Adjacent layout: the pairs of one vector.
template <bool kBF16>
__device__ __forceinline__ void turn_adjacent(uint4& v, const uint64_t* c, const uint64_t* s)
{
    uint32_t* w = reinterpret_cast<uint32_t*>(&v);
    uint64_t y0, y1;
    if constexpr (kBF16) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            turn2(pk(bf16lo(w[2 * i]), bf16lo(w[2 * i + 1])), pk(bf16hi(w[2 * i]), bf16hi(w[2 * i + 1])), c[i], s[i], y0, y1);
            w[2 * i] = pack_bf16_rn(pk_lo(y0), pk_lo(y1));
            w[2 * i + 1] = pack_bf16_rn(pk_hi(y0), pk_hi(y1));
        }
    } else {
        float* f = reinterpret_cast<float*>(&v);
        turn2(pk(f[0], f[2]), pk(f[1], f[3]), c[0], s[0], y0, y1);
        v = make_uint4(__float_as_uint(pk_lo(y0)), __float_as_uint(pk_lo(y1)), __float_as_uint(pk_hi(y0)),
                       __float_as_uint(pk_hi(y1)));
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

// kTPT threads per token (kSplit: and 2^parts_log2 CTAs, each with a share of its
// heads).  Residency: 8 CTAs per SM (7 where the half layout
// keeps twice the twiddles) at a few spilled bytes beat 5 without: 8320 tokens of
// 32 / 8 heads at D = 128, half 34.8 against 42.9 us, adjacent 32.8 against 37.5.
template <bool kBF16, int kD, bool kHalf, bool kFP8, bool kAxes, int kTPT, bool kSplit>
__global__ void __launch_bounds__(kThreads, (kHalf ? 7 : 8)) rotary_append_kernel(const __grid_constant__ RotaryArgs a, const int parts_log2)
{
    pdl_wait();
    constexpr int kE = kBF16 ? 2 : 4;
    constexpr int kEPV = 16 / kE;              // elements per 16-byte vector
    constexpr int kU = kD / (2 * kEPV);        // units per head
    constexpr int kGroups = kTPT / kU;         // heads in flight
    constexpr int kVPH = kD / kEPV;            // vectors per head
    static_assert(!kFP8 || (kBF16 && kD == 128), "fp8 pages hold D = 128 rows quantised from bf16");
    constexpr int kFlightV = kTPT == kThreads ? 1 : 2;
    static_assert(kGroups >= 1, "a token's threads hold whole heads");
    __shared__ __align__(16) float2 tws[kThreads / kTPT][kD / 2];

    static_assert(kTPT == 32 || kTPT == kThreads, "a token's threads are a warp or the CTA");
    const int tid = kTPT == kThreads ? (int)threadIdx.x : (int)threadIdx.x % kTPT;  // thread of the token
    static_assert(!kSplit || kTPT == kThreads, "parts are CTAs");
    const int lp = kSplit ? parts_log2 : 0, part = kSplit ? blockIdx.x & ((1 << lp) - 1) : 0;
    const int t = kTPT == kThreads ? blockIdx.x >> lp : blockIdx.x * (kThreads / kTPT) + threadIdx.x / kTPT;
    if (kTPT != kThreads && t >= a.num_tokens) return;
    float2* tw = tws[kTPT == kThreads ? 0 : threadIdx.x / kTPT];
    const int u = tid % kU, hg = tid / kU + part * kGroups;  // unit, first head
    const int hs = kGroups << lp;                            // heads between a thread's
    const int vg = tid + part * kTPT, vs = kTPT << lp;       // V vectors: first, step
    // element offsets of the unit's two vectors in a head, and whether they turn:
    // neighbouring units hold neighbouring vectors, so a warp's accesses are whole lines
    const int nu = a.rot / (2 * kEPV);  // units that turn (half layout)
    const bool rot_a = kHalf ? u < nu : u * kEPV < a.rot;
    const bool rot_b = kHalf ? u < nu : (u + kU) * kEPV < a.rot;
    const int ea = kHalf && !rot_a ? a.rot + (u - nu) * kEPV : u * kEPV;
    const int eb = !kHalf ? (u + kU) * kEPV : rot_a ? a.rot / 2 + u * kEPV : a.rot + (u - nu + kU - nu) * kEPV;
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
    uint4 xa[kFlight], xb[kFlight], xv[kFlightV];
#pragma unroll
    for (int i = 0; i < kFlightV; ++i) xv[i] = make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int i = 0; i < kFlight; ++i)
        if (hg + i * hs < heads) load(hg + i * hs, xa[i], xb[i]);
#pragma unroll
    for (int i = 0; i < kFlightV; ++i)
        if (vg + i * vs < nvec) xv[i] = *reinterpret_cast<const uint4*>(vrow + (vg + i * vs) * 16);

    const int slot = kAxes ? a.slots[t] : a.positions[t], seq = a.seq_ids[t];
    // positions of this thread's pairs.  kAxes: each on its pair's axis; all of the token's are
    // looked at below, by a vote.  (Every thread loading all axes: 10,200 tokens of 32 / 8 heads
    // 52.4 us instead of 43.5; one axis, rotary_append, 42.9.)
    constexpr int kPairs = (kD / 2 + kTPT - 1) / kTPT;
    int at[kAxes ? kPairs : 1] = {slot};
    bool good = true;
    if constexpr (kAxes) {
        auto on = [&](int x) { return a.positions[(int64_t)x * a.num_tokens + t]; };
#pragma unroll
        for (int j = 0; j < kPairs; ++j) {
            const int i = j * kTPT + tid;
            at[j] = i < a.rot / 2 ? on((int)((i < 32 ? a.axis[0] : a.axis[1]) >> (2 * (i & 31))) & 3) : 0;
        }
        if (tid < a.num_axes) good = on(tid) >= 0;
    }
    bool ok = slot >= 0 && seq >= 0 && seq < a.num_seqs && slot / a.block_size < a.max_blocks;
    int64_t blk = -1;
    if (ok) {
        blk = a.block_table[(int64_t)seq * a.max_blocks + slot / a.block_size];
        ok = blk >= 0 && blk < a.num_blocks;
    }
    if (!ok) {  // the same for every thread
        if (tid == 0) record_error(a.status, KVATTN_ERR_BAD_INDEX);
        return;
    }
    const int off = slot % a.block_size;
#pragma unroll
    for (int i0 = 0; i0 < kD / 2; i0 += kTPT) {
        const int i = i0 + tid;
        if (i < a.rot / 2) {
            const int pos = at[kAxes ? i0 / kTPT : 0];
            const float2 w = twiddle((uint64_t)(uint32_t)pos * a.turns[i]);
            tw[i] = make_float2(w.x * a.amplitude, w.y * a.amplitude);
        }
    }
    if constexpr (kAxes) {
        if constexpr (kTPT == 32) good = __all_sync(0xffffffffu, good);
        else good = __syncthreads_and(good);
        if (!good) {
            if (tid == 0) record_error(a.status, KVATTN_ERR_BAD_INDEX);
            return;
        }
    }
    if constexpr (kTPT == 32) __syncwarp();
    else if constexpr (!kAxes) __syncthreads();
    Twiddles<kHalf ? kEPV : kEPV / 2> ta, tb;  // (half: tb unused)
    if (rot_a) ta.load(&tw[kHalf ? u * kEPV : u * kEPV / 2]);
    if (!kHalf && rot_b) tb.load(&tw[(u + kU) * kEPV / 2]);

    auto finish = [&](int hh, uint4 x, uint4 y) {
        if constexpr (kHalf) {
            if (rot_a) turn_half<kBF16>(x, y, ta.c, ta.s);
        } else {
            if (rot_a) turn_adjacent<kBF16>(x, ta.c, ta.s);
            if (rot_b) turn_adjacent<kBF16>(y, tb.c, tb.s);
        }
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
    for (int h0 = hg; h0 < heads; h0 += kFlight * hs) {
        if (h0 != hg) {
#pragma unroll
            for (int i = 0; i < kFlight; ++i)
                if (h0 + i * hs < heads) load(h0 + i * hs, xa[i], xb[i]);
        }
#pragma unroll
        for (int i = 0; i < kFlight; ++i)
            if (h0 + i * hs < heads) finish(h0 + i * hs, xa[i], xb[i]);
    }
#pragma unroll
    for (int i = 0; i < kFlightV; ++i)
        if (vg + i * vs < nvec) put_v(vg + i * vs, xv[i]);
    for (int j = vg + kFlightV * vs; j < nvec; j += vs)
        put_v(j, *reinterpret_cast<const uint4*>(vrow + j * 16));
}

template <bool kBF16, int kD, bool kHalf, bool kFP8, bool kAxes>
kvattn_status launch(const RotaryArgs& a, cudaStream_t s)
{
    auto run = [&](auto kern, int tpt, int parts_log2) {
        const int per = kThreads / tpt;
        return cuda_status(launch_pdl(kern, dim3(((a.num_tokens + per - 1) / per) << parts_log2), dim3(kThreads), 0, s, a,
                                      parts_log2));
    };
    // A CTA per token, or a warp when the token is small and there are enough of
    // them for every SM's warps (8320 tokens, CTA and warp: 32 / 8 heads of 128
    // 34.8 and 40.1 us; 16 / 8 of 128 32.1 and 27.8; 12 / 12 of 64 17.4 and 12.1;
    // 64 tokens of those 2.4 and 3.0).
    const int units = (a.hq + a.hkv) * (kD / (kBF16 ? 16 : 8));
    if (units <= 192 && a.num_tokens >= 2048) return run(rotary_append_kernel<kBF16, kD, kHalf, kFP8, kAxes, 32, false>, 32, 0);
    // Two or four CTAs for a large token: as many as one wave of CTAs has room for
    // (fp32, 32 / 32 heads of 128, 8 and 300 tokens: 5.2 -> 2.5 and 5.9 -> 4.8 us),
    // or two beyond a wave, for a fuller last one (1319 and 4300: 28 -> 24.4 and 75
    // -> 70).  With 600 tokens, half a wave, two cost 9.0 against 7.8; smaller tokens
    // lose to the second look-up and twiddles (bf16, 32 / 8, 300: 3.0 -> 3.4).
    const int64_t wave = (int64_t)num_sms() * (kHalf ? 7 : 8);
    int parts = 0;
    while (parts < 2 && units >> (parts + 1) >= 256 && ((int64_t)a.num_tokens << (parts + 1)) <= wave) ++parts;
    if (units >= 1024 && a.num_tokens > wave && a.num_tokens <= INT32_MAX / 2) parts = 1;
    return parts ? run(rotary_append_kernel<kBF16, kD, kHalf, kFP8, kAxes, 128, true>, 128, parts)
                 : run(rotary_append_kernel<kBF16, kD, kHalf, kFP8, kAxes, 128, false>, 128, 0);
}

template <bool kBF16, int kD, bool kFP8, bool kAxes>
kvattn_status launch_layout(const RotaryArgs& a, cudaStream_t s)
{
    return a.half ? launch<kBF16, kD, true, kFP8, kAxes>(a, s) : launch<kBF16, kD, false, kFP8, kAxes>(a, s);
}

template <bool kAxes>
kvattn_status dispatch(const RotaryArgs& a, cudaStream_t s)
{
    if (a.fp8) {
        if (a.dtype != KVATTN_BF16 || a.d != 128) return KVATTN_ERR_UNSUPPORTED;
        return launch_layout<true, 128, true, kAxes>(a, s);
    }
    const bool bf16 = a.dtype == KVATTN_BF16;
    if (a.d == 128) return bf16 ? launch_layout<true, 128, false, kAxes>(a, s) : launch_layout<false, 128, false, kAxes>(a, s);
    if (a.d == 64) return bf16 ? launch_layout<true, 64, false, kAxes>(a, s) : launch_layout<false, 64, false, kAxes>(a, s);
    return KVATTN_ERR_UNSUPPORTED;
}

}  // namespace
}  // namespace kvattn
