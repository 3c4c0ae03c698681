// What the warp-specialised attention kernels on the tcgen05 tensor cores have in
// common: bounded waits that end when any role gives up, small device helpers,
// and the encoding of tensor maps.
#pragma once

#include <mutex>

#include "fast_exp2.cuh"
#include "kvattn_tc.cuh"

namespace kvattn {
namespace {

// The flag is looked at only where the wait does not succeed at once: a role
// that finds its barriers complete runs on after an abort (a try in vain comes
// back within a microsecond on this GPU).
__device__ __forceinline__ bool wait_or_abort(uint64_t* bar, uint32_t parity, volatile int* abort_flag, int* status)
{
    if (__builtin_expect(mbar_try_wait(bar, parity), 1)) return true;
    if (*abort_flag) return false;
    if (mbar_wait(bar, parity, status)) return true;
    *abort_flag = 1;
    return false;
}

// Whole-warp wait of the roles that do not take part in every tile: for as long as
// the `tiles` that go by meanwhile may take besides (1.3 to 3.5 us each), and not
// past an abort.
constexpr uint64_t kTileLimitNs = 8000;
__device__ __forceinline__ bool long_wait(uint64_t* bar, uint32_t parity, int tiles, volatile int* abort_flag, int* status)
{
    const uint64_t limit = kWaitLimitNs + (uint64_t)tiles * kTileLimitNs, t0 = global_timer_ns();
    bool ok = false;
    while (!(ok = mbar_try_wait(bar, parity)) && !*abort_flag) {
        if (global_timer_ns() - t0 > limit) {
            record_error(status, KVATTN_ERR_TIMEOUT);
            *abort_flag = 1;
        }
    }
    return __all_sync(0xffffffffu, ok);
}

// Whole-warp wait: every lane waits, the warp agrees.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag, int* status)
{
    const bool ok = wait_or_abort(bar, parity, abort_flag, status);
    return __all_sync(0xffffffffu, ok);
}

__device__ __forceinline__ float max3(float a, float b, float c)
{
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// Named barrier `id` over `nthreads` threads.
__device__ __forceinline__ void bar_sync(int id, int nthreads)
{
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(nthreads) : "memory");
}

// 32 bytes (a sector) to p, aligned to 32.
__device__ __forceinline__ void store_256(void* p, const uint32_t* v)
{
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]),
                 "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}

// One lane of the (converged) warp is elected.
__device__ __forceinline__ bool elect_one()
{
    uint32_t pred = 0;
    asm volatile("{\n\t.reg .pred P;\n\telect.sync _|P, 0xffffffff;\n\tselp.u32 %0, 1, 0, P;\n\t}" : "=r"(pred));
    return pred != 0;
}

// Bits 0 .. n-1 of a word (all for n >= 32, none for n <= 0).
__device__ __forceinline__ uint32_t low_bits(int n)
{
    uint32_t m;
    asm("bmsk.clamp.b32 %0, 0, %1;" : "=r"(m) : "r"(max(n, 0)));
    return m;
}

// i / d for 0 <= i < 2^30: with 2^s >= d, m = ceil(2^(30+s) / d) is above
// 2^(30+s) / d by less than 2^s / d, so i m / 2^(30+s) is above i / d by less
// than 1 / d.
struct Divisor {
    uint32_t m, shift;
    explicit Divisor(int d)
    {
        int s = 0;
        while ((1 << s) < d) ++s;
        m = (uint32_t)((((uint64_t)1 << (30 + s)) + d - 1) / d);
        shift = 30 + s;
    }
    __device__ __forceinline__ int quot(int i) const { return (int)(((uint64_t)(uint32_t)i * m) >> shift); }
};
// ---- host: tensor maps --------------------------------------------------------

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                 const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encoder()
{
    static EncodeTiled fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiled>(p);
    });
    return fn;
}

bool encode(CUtensorMap* m, const void* base, int rank, const cuuint64_t* dims, const cuuint64_t* strides,
            const cuuint32_t* box)
{
    const cuuint32_t estr[3] = {1, 1, 1};
    EncodeTiled enc = encoder();
    return enc && enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, const_cast<void*>(base), dims, strides, box, estr,
                      CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                      CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace
}  // namespace kvattn
