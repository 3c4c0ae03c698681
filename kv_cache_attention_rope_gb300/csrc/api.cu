// C ABI of kvattn: argument validation, per-device set-up, dispatch to the
// kernels.  Every check the host can make is made here, before any launch.
#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <limits>
#include <mutex>

#include "kvattn_internal.cuh"

namespace kvattn {

// Module-scope device status word: first device-side error since the last
// kvattn_get_device_status().  One instance per device that loads the module.
__device__ int g_device_status = 0;

namespace {

constexpr int kMaxDevices = 64;
std::mutex g_mu;
int* g_status_ptr[kMaxDevices] = {};
int g_sms[kMaxDevices] = {};

int current_device()
{
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return -1;
    return dev;
}

}  // namespace

int* device_status_ptr()
{
    const int dev = current_device();
    if (dev < 0) return nullptr;
    std::lock_guard<std::mutex> g(g_mu);
    if (!g_status_ptr[dev]) {
        void* p = nullptr;
        if (cudaGetSymbolAddress(&p, g_device_status) != cudaSuccess) return nullptr;
        g_status_ptr[dev] = static_cast<int*>(p);
    }
    return g_status_ptr[dev];
}

int num_sms()
{
    const int dev = current_device();
    if (dev < 0) return 1;
    std::lock_guard<std::mutex> g(g_mu);
    if (!g_sms[dev]) {
        int n = 0;
        if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) n = 1;
        g_sms[dev] = n;
    }
    return g_sms[dev];
}

bool device_smem(DeviceSmem* out)
{
    static DeviceSmem cache[kMaxDevices] = {};
    const int dev = current_device();
    if (dev < 0) return false;
    std::lock_guard<std::mutex> g(g_mu);
    DeviceSmem& c = cache[dev];
    if (!c.per_sm) {
        int per_sm = 0, reserved = 0;
        if (cudaDeviceGetAttribute(&per_sm, cudaDevAttrMaxSharedMemoryPerMultiprocessor, dev) != cudaSuccess ||
            per_sm <= 0)
            return false;
        if (cudaDeviceGetAttribute(&reserved, cudaDevAttrReservedSharedMemoryPerBlock, dev) != cudaSuccess)
            reserved = 1024;
        c.reserved = reserved;
        c.per_sm = per_sm;
    }
    *out = c;
    return true;
}

cudaError_t SmemLimit::ensure(const void* func, int bytes)
{
    const int dev = current_device();
    if (dev < 0) return cudaErrorInvalidDevice;
    std::lock_guard<std::mutex> g(mu_);
    if (set_[dev] >= bytes) return cudaSuccess;
    const cudaError_t e = cudaFuncSetAttribute(func, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) set_[dev] = bytes;
    return e;
}

cudaError_t Residency::query(const void* func, int threads, int bytes, int* per_sm)
{
    const int dev = current_device();
    if (dev < 0) return cudaErrorInvalidDevice;
    cudaError_t e = limit_.ensure(func, bytes);
    if (e != cudaSuccess) return e;
    std::lock_guard<std::mutex> g(mu_);
    if (per_sm_[dev] == 0 || threads_[dev] != threads || bytes_[dev] != bytes) {
        int n = 0;
        e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, func, threads, bytes);
        if (e != cudaSuccess) return e;
        threads_[dev] = threads;
        bytes_[dev] = bytes;
        per_sm_[dev] = std::max(1, n);
    }
    *per_sm = per_sm_[dev];
    return cudaSuccess;
}

namespace {

bool config_ok(const kvattn_config* c)
{
    return c && c->num_q_heads > 0 && c->num_kv_heads > 0 && c->head_dim > 0 &&
           (c->dtype == KVATTN_F32 || c->dtype == KVATTN_BF16) && std::isfinite(c->rope_base) &&
           c->rope_base > 0.f && std::isfinite(c->scale) && c->scale >= 0.f;
}

kvattn_status config_supported(const kvattn_config* c)
{
    if (c->num_q_heads % c->num_kv_heads != 0) return KVATTN_ERR_UNSUPPORTED;
    const int g = c->num_q_heads / c->num_kv_heads;
    if (g != 1 && g != 2 && g != 4 && g != 8) return KVATTN_ERR_UNSUPPORTED;
    if (c->head_dim != 64 && c->head_dim != 128) return KVATTN_ERR_UNSUPPORTED;
    return KVATTN_OK;
}

bool cache_ok(const kvattn_cache* k, int32_t max_blocks_per_seq)
{
    if (!k || !k->k_pool || !k->v_pool || k->num_blocks <= 0 || k->num_blocks > INT32_MAX || k->block_size <= 0)
        return false;
    if (max_blocks_per_seq <= 0) return false;
    // a 16-token tile must not cross a block boundary
    if (max_blocks_per_seq > 1 && k->block_size % 16 != 0) return false;
    // 16-byte alignment of the pools (bulk copies)
    if ((reinterpret_cast<uintptr_t>(k->k_pool) | reinterpret_cast<uintptr_t>(k->v_pool)) & 15u) return false;
    return true;
}

float scale_of(const kvattn_config* c)
{
    return c->scale > 0.f ? c->scale : 1.0f / std::sqrt((float)c->head_dim);
}

// Host tables of the rotary embedding for (base, D): per-pair speed in 2^-64
// turns per position, and the float-float cos/sin of k*pi/16, k = 0..4, from
// their nested-radical closed forms (exactly rounded square roots, so the
// values do not depend on the host's libm).
void rope_tables(double base, int d, RopeArgs& a)
{
    static thread_local double cached_base = -1.0;
    static thread_local int cached_d = -1;
    static thread_local uint64_t turns[64];
    if (cached_base != base || cached_d != d) {
        const double two_pi = 6.283185307179586476925286766559;
        for (int i = 0; i < d / 2; ++i) {
            const double f = std::pow(base, -2.0 * (double)i / (double)d) / two_pi;  // turns per position
            turns[i] = (uint64_t)std::llrint(std::ldexp(f, 64));  // f < 1/(2 pi): fits in int64
        }
        cached_base = base;
        cached_d = d;
    }
    std::memcpy(a.turns, turns, sizeof(turns));
    const double r2 = std::sqrt(2.0);
    const double c[5] = {1.0, 0.5 * std::sqrt(2.0 + std::sqrt(2.0 + r2)), 0.5 * std::sqrt(2.0 + r2),
                         0.5 * std::sqrt(2.0 + std::sqrt(2.0 - r2)), 0.5 * r2};
    const double s[5] = {0.0, 0.5 * std::sqrt(2.0 - std::sqrt(2.0 + r2)), 0.5 * std::sqrt(2.0 - r2),
                         0.5 * std::sqrt(2.0 - std::sqrt(2.0 - r2)), 0.5 * r2};
    for (int k = 0; k < 5; ++k) {
        const float ch = (float)c[k], sh = (float)s[k];
        a.sector[k] = make_float4(ch, (float)(c[k] - (double)ch), sh, (float)(s[k] - (double)sh));
    }
}

bool rotary_ok(const kvattn_config* c, const kvattn_rotary* r)
{
    if (!r || (r->layout != KVATTN_ROPE_ADJACENT && r->layout != KVATTN_ROPE_HALF) || r->rotary_dim < 0 ||
        !std::isfinite(r->amplitude) || r->amplitude < 0.f || c->rope_base < 1.f)
        return false;
    switch (r->scaling) {
        case KVATTN_ROPE_UNSCALED: return true;
        case KVATTN_ROPE_LINEAR:
        case KVATTN_ROPE_BASE: return std::isfinite(r->factor) && r->factor >= 1.f;
        case KVATTN_ROPE_PARTS:
            return std::isfinite(r->factor) && r->factor >= 1.f && std::isfinite(r->original_len) &&
                   r->original_len > 0.f && std::isfinite(r->low) && std::isfinite(r->high) && r->low >= 0.f &&
                   r->high > r->low;
    }
    return false;
}

// Speed of pair i < rot / 2 in 2^-64 turns per position (kvattn_rotary_append
// in kvattn.h states the formulas; with base and factor at least 1 it is below
// 1 / (2 pi) turns).  At position 2^31 an error of 2^-53 in a speed near 1 would be
// 2^-22 radians, hence the wider type, which takes longer (128 bits in software on
// Arm).  The layers of a model share one form or a few: the last ones computed by
// this host thread are kept.
void rotary_turns(const kvattn_config* c, const kvattn_rotary* r, int rot, uint64_t* turns)
{
    using real = long double;
    static_assert(std::numeric_limits<real>::digits >= 64, "the host's long double holds a speed to 2^-64");
    struct Form {
        kvattn_rotary r;
        float base;
        int rot;  // 0: none
        uint64_t turns[64];
    };
    constexpr int kForms = 4;
    static thread_local Form kept[kForms];
    static thread_local int oldest = 0;
    for (const Form& k : kept)
        if (k.rot == rot && k.base == c->rope_base && std::memcmp(&k.r, r, sizeof(k.r)) == 0) {
            std::memcpy(turns, k.turns, sizeof(k.turns));
            return;
        }
    Form& k = kept[oldest];
    oldest = (oldest + 1) % kForms;
    const real two_pi = 6.28318530717958647692528676655900577L, s = r->factor;
    real base = c->rope_base;
    if (r->scaling == KVATTN_ROPE_BASE) base *= std::pow(s, (real)rot / (real)(rot - 2));
    for (int i = 0; i < rot / 2; ++i) {
        real f = std::pow(base, (real)(-2 * i) / (real)rot) / two_pi;
        if (r->scaling == KVATTN_ROPE_LINEAR) {
            f /= s;
        } else if (r->scaling == KVATTN_ROPE_PARTS) {
            const real g = ((real)r->original_len * f - r->low) / ((real)r->high - r->low);
            const real share = std::min<real>(1, std::max<real>(0, g));
            f = f * (share + (1 - share) / s);
        }
        k.turns[i] = (uint64_t)std::llrint(std::ldexp(f, 64));
    }
    k.r = *r;
    k.base = c->rope_base;
    k.rot = rot;
    std::memcpy(turns, k.turns, sizeof(k.turns));
}

// One CTA waits on an mbarrier that nothing will complete, through the same
// bounded wait every kernel uses; the wait runs out and records
// KVATTN_ERR_TIMEOUT.
__global__ void selftest_timeout_kernel(int* status, uint64_t limit_ns)
{
    __shared__ uint64_t bar;
    if (threadIdx.x == 0) {
        mbar_init(&bar, 1);
        fence_mbar_init();
    }
    __syncthreads();
    mbar_wait(&bar, 0, status, limit_ns);
}

}  // namespace

kvattn_status decode_check(const kvattn_config* cfg, const kvattn_cache* cache, bool fp8, const void* q,
                           const int32_t* block_table, int32_t max_blocks_per_seq, const int32_t* seq_lens,
                           int32_t batch, int32_t max_seq_len, int32_t num_splits, const void* out)
{
    if (!config_ok(cfg) || batch < 0 || max_seq_len < 0 || num_splits < 0) return KVATTN_ERR_INVALID_ARG;
    kvattn_status st = config_supported(cfg);
    if (st != KVATTN_OK) return st;
    if (!cache_ok(cache, max_blocks_per_seq)) return KVATTN_ERR_INVALID_ARG;
    if (fp8) {
        if (cache->block_size % 16 != 0) return KVATTN_ERR_INVALID_ARG;
        const int g = cfg->num_q_heads / cfg->num_kv_heads;
        if (cfg->dtype != KVATTN_BF16 || cfg->head_dim != 128 || (g != 4 && g != 8)) return KVATTN_ERR_UNSUPPORTED;
    }
    if (batch == 0) return KVATTN_OK;
    if (batch > kMaxDecodeBatch) return KVATTN_ERR_UNSUPPORTED;
    if (!q || !block_table || !seq_lens || !out) return KVATTN_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(out)) & 15u) return KVATTN_ERR_INVALID_ARG;
    return KVATTN_OK;
}

}  // namespace kvattn

using namespace kvattn;

extern "C" {

int32_t kvattn_version(void) { return KVATTN_VERSION; }

const char* kvattn_status_string(kvattn_status s)
{
    switch (s) {
        case KVATTN_OK: return "ok";
        case KVATTN_ERR_INVALID_ARG: return "invalid argument";
        case KVATTN_ERR_UNSUPPORTED: return "unsupported configuration";
        case KVATTN_ERR_OUT_OF_BLOCKS: return "out of KV blocks";
        case KVATTN_ERR_WORKSPACE_TOO_SMALL: return "workspace too small";
        case KVATTN_ERR_CUDA: return "CUDA error";
        case KVATTN_ERR_TIMEOUT: return "device wait timed out";
        case KVATTN_ERR_BAD_INDEX: return "block id or position out of range";
    }
    return "unknown status";
}

kvattn_status kvattn_rope_append(const kvattn_config* cfg, const kvattn_cache* cache, void* q, const void* k,
                                 const void* v, const int32_t* positions, const int32_t* seq_ids,
                                 const int32_t* block_table, int32_t num_seqs, int32_t max_blocks_per_seq,
                                 int32_t num_tokens, void* stream)
{
    if (!config_ok(cfg)) return KVATTN_ERR_INVALID_ARG;
    const int64_t qrow = (int64_t)cfg->num_q_heads * cfg->head_dim;
    const int64_t kvrow = (int64_t)cfg->num_kv_heads * cfg->head_dim;
    return kvattn_rope_append_strided(cfg, cache, q, qrow, k, kvrow, v, kvrow, nullptr, positions, seq_ids,
                                      block_table, num_seqs, max_blocks_per_seq, num_tokens, stream);
}

kvattn_status kvattn_rope_append_strided(const kvattn_config* cfg, const kvattn_cache* cache, void* q,
                                         int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                                         int64_t v_stride, void* q_out, const int32_t* positions,
                                         const int32_t* seq_ids, const int32_t* block_table, int32_t num_seqs,
                                         int32_t max_blocks_per_seq, int32_t num_tokens, void* stream)
{
    if (!config_ok(cfg) || num_tokens < 0 || num_seqs <= 0) return KVATTN_ERR_INVALID_ARG;
    kvattn_status st = config_supported(cfg);
    if (st != KVATTN_OK) return st;
    if (!cache_ok(cache, max_blocks_per_seq)) return KVATTN_ERR_INVALID_ARG;
    // a row never overlaps the next one, and every row starts on a 16-byte boundary
    const int64_t e = cfg->dtype == KVATTN_BF16 ? 2 : 4;
    const int64_t qrow = (int64_t)cfg->num_q_heads * cfg->head_dim;
    const int64_t kvrow = (int64_t)cfg->num_kv_heads * cfg->head_dim;
    const int64_t max_stride = INT64_MAX / 4 / std::max<int64_t>(1, num_tokens);
    if (q_stride < qrow || k_stride < kvrow || v_stride < kvrow) return KVATTN_ERR_INVALID_ARG;
    if (q_stride > max_stride || k_stride > max_stride || v_stride > max_stride) return KVATTN_ERR_INVALID_ARG;
    if (((q_stride | k_stride | v_stride) * e) & 15) return KVATTN_ERR_INVALID_ARG;
    if (num_tokens == 0) return KVATTN_OK;
    if (!q || !k || !v || !positions || !seq_ids || !block_table) return KVATTN_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(v) |
         reinterpret_cast<uintptr_t>(q_out)) & 15u)
        return KVATTN_ERR_INVALID_ARG;
    RopeArgs a;
    std::memset(&a, 0, sizeof(a));
    a.q = q;
    a.k = k;
    a.v = v;
    a.q_stride = q_stride * e;
    a.k_stride = k_stride * e;
    a.v_stride = v_stride * e;
    a.q_out = q_out ? q_out : q;
    a.q_out_stride = q_out ? qrow * e : a.q_stride;
    a.k_pool = cache->k_pool;
    a.v_pool = cache->v_pool;
    a.positions = positions;
    a.seq_ids = seq_ids;
    a.block_table = block_table;
    a.num_blocks = cache->num_blocks;
    a.block_size = cache->block_size;
    a.num_seqs = num_seqs;
    a.max_blocks = max_blocks_per_seq;
    a.num_tokens = num_tokens;
    a.hq = cfg->num_q_heads;
    a.hkv = cfg->num_kv_heads;
    a.d = cfg->head_dim;
    a.dtype = cfg->dtype;
    a.status = device_status_ptr();
    if (!a.status) return KVATTN_ERR_CUDA;
    rope_tables((double)cfg->rope_base, cfg->head_dim, a);
    return launch_rope_append(a, static_cast<cudaStream_t>(stream));
}

namespace {

constexpr int32_t kMaxRotaryHeads = 1 << 20;  // the kernel counts a token's bytes in 32 bits
constexpr int32_t kMaxFp8KvHeads = 65535;     // the kernel of an fp8 cache's V has them in its grid's second dimension

// The axis of each of `pairs` pairs; false for axes that kvattn.h does not allow.
bool axes_of_pairs(const kvattn_rope_axes* x, int pairs, uint8_t* axis)
{
    if (x->num_axes < 1 || x->num_axes > kMaxAxes) return false;
    if (x->order != KVATTN_AXES_SECTIONS && x->order != KVATTN_AXES_CYCLIC) return false;
    int64_t all = 0;
    for (int a = 0; a < x->num_axes; ++a) {
        if (x->sections[a] < 0 || x->sections[a] > pairs) return false;
        all += x->sections[a];
    }
    if (all != pairs) return false;
    int n = 0;
    if (x->order == KVATTN_AXES_SECTIONS) {
        for (int a = 0; a < x->num_axes; ++a)
            for (int j = 0; j < x->sections[a]; ++j) axis[n++] = (uint8_t)a;
        return true;
    }
    for (int a = 1; a < x->num_axes; ++a)  // its last pair is there
        if (x->sections[a] > 0 && a + (x->sections[a] - 1) * x->num_axes >= pairs) return false;
    for (; n < pairs; ++n) {
        const int a = n % x->num_axes;
        axis[n] = (uint8_t)(n / x->num_axes < x->sections[a] ? a : 0);
    }
    return true;
}

// axes null: `positions` are the slots too.
kvattn_status rotary_append_any(const kvattn_config* cfg, const kvattn_rotary* rotary, const kvattn_rope_axes* axes,
                                const int32_t* slots, const kvattn_cache* cache, bool fp8, void* q, int64_t q_stride,
                                const void* k, int64_t k_stride, const void* v,
                                int64_t v_stride, void* q_out, const int32_t* positions, const int32_t* seq_ids,
                                const int32_t* block_table, int32_t num_seqs, int32_t max_blocks_per_seq,
                                int32_t num_tokens, void* stream)
{
    if (!config_ok(cfg) || !rotary_ok(cfg, rotary) || num_tokens < 0 || num_seqs <= 0) return KVATTN_ERR_INVALID_ARG;
    const kvattn_status st = config_supported(cfg);
    if (st != KVATTN_OK) return st;
    if (fp8 && (cfg->dtype != KVATTN_BF16 || cfg->head_dim != 128)) return KVATTN_ERR_UNSUPPORTED;
    const int rot = rotary->rotary_dim ? rotary->rotary_dim : cfg->head_dim;
    if (rot > cfg->head_dim || rot % 16 != 0) return KVATTN_ERR_UNSUPPORTED;
    uint8_t axis[64] = {};
    if (axes && !axes_of_pairs(axes, rot / 2, axis)) return KVATTN_ERR_INVALID_ARG;
    if (cfg->num_q_heads > kMaxRotaryHeads || (fp8 && cfg->num_kv_heads > kMaxFp8KvHeads)) return KVATTN_ERR_UNSUPPORTED;
    if (!cache_ok(cache, max_blocks_per_seq) || (fp8 && cache->block_size % 16 != 0)) return KVATTN_ERR_INVALID_ARG;
    const int64_t e = cfg->dtype == KVATTN_BF16 ? 2 : 4;
    const int64_t qrow = (int64_t)cfg->num_q_heads * cfg->head_dim;
    const int64_t kvrow = (int64_t)cfg->num_kv_heads * cfg->head_dim;
    const int64_t max_stride = INT64_MAX / 4 / std::max<int64_t>(1, num_tokens);
    if (q_stride < qrow || k_stride < kvrow || v_stride < kvrow) return KVATTN_ERR_INVALID_ARG;
    if (q_stride > max_stride / e || k_stride > max_stride / e || v_stride > max_stride / e)
        return KVATTN_ERR_INVALID_ARG;
    if (((q_stride | k_stride | v_stride) * e) & 15) return KVATTN_ERR_INVALID_ARG;
    if (num_tokens == 0) return KVATTN_OK;
    if (!q || !k || !v || !positions || !seq_ids || !block_table || (axes && !slots)) return KVATTN_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(v) |
         reinterpret_cast<uintptr_t>(q_out)) & 15u)
        return KVATTN_ERR_INVALID_ARG;
    RotaryArgs a;
    std::memset(&a, 0, sizeof(a));
    a.q = q;
    a.k = k;
    a.v = v;
    a.q_stride = q_stride * e;
    a.k_stride = k_stride * e;
    a.v_stride = v_stride * e;
    a.q_out = q_out ? q_out : q;
    a.q_out_stride = q_out ? qrow * e : a.q_stride;
    a.fp8 = fp8 ? 1 : 0;
    a.k_pool = cache->k_pool;
    a.v_pool = cache->v_pool;
    a.positions = positions;
    a.seq_ids = seq_ids;
    a.block_table = block_table;
    a.num_blocks = cache->num_blocks;
    a.block_size = cache->block_size;
    a.num_seqs = num_seqs;
    a.max_blocks = max_blocks_per_seq;
    a.num_tokens = num_tokens;
    a.hq = cfg->num_q_heads;
    a.hkv = cfg->num_kv_heads;
    a.d = cfg->head_dim;
    a.dtype = cfg->dtype;
    a.half = rotary->layout == KVATTN_ROPE_HALF ? 1 : 0;
    a.rot = rot;
    a.amplitude = rotary->amplitude > 0.f ? rotary->amplitude : 1.f;
    a.status = device_status_ptr();
    if (!a.status) return KVATTN_ERR_CUDA;
    rotary_turns(cfg, rotary, rot, a.turns);
    if (axes) {
        a.slots = slots;
        a.num_axes = axes->num_axes;
        for (int i = 0; i < 64; ++i) a.axis[i / 32] |= (uint64_t)axis[i] << (2 * (i % 32));
    }
    const kvattn_status kst = axes ? launch_rotary_append_axes(a, static_cast<cudaStream_t>(stream))
                                   : launch_rotary_append(a, static_cast<cudaStream_t>(stream));
    if (kst != KVATTN_OK || !fp8) return kst;
    RopeArgs r;  // the V pages
    std::memset(&r, 0, sizeof(r));
    r.v = v;
    r.v_stride = a.v_stride;
    r.k_pool = cache->k_pool;
    r.fp8 = 1;
    r.positions = axes ? slots : positions;
    r.axes = axes ? positions : nullptr;
    r.num_axes = axes ? axes->num_axes : 0;
    r.seq_ids = seq_ids;
    r.block_table = block_table;
    r.num_blocks = cache->num_blocks;
    r.block_size = cache->block_size;
    r.num_seqs = num_seqs;
    r.max_blocks = max_blocks_per_seq;
    r.num_tokens = num_tokens;
    r.hkv = cfg->num_kv_heads;
    return launch_append_v_fp8(r, static_cast<cudaStream_t>(stream));
}

}  // namespace

kvattn_status kvattn_rotary_append(const kvattn_config* cfg, const kvattn_rotary* rotary, const kvattn_cache* cache,
                                   void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                                   int64_t v_stride, void* q_out, const int32_t* positions, const int32_t* seq_ids,
                                   const int32_t* block_table, int32_t num_seqs, int32_t max_blocks_per_seq,
                                   int32_t num_tokens, void* stream)
{
    return rotary_append_any(cfg, rotary, nullptr, nullptr, cache, false, q, q_stride, k, k_stride, v, v_stride, q_out, positions,
                             seq_ids, block_table, num_seqs, max_blocks_per_seq, num_tokens, stream);
}

kvattn_status kvattn_rotary_append_fp8(const kvattn_config* cfg, const kvattn_rotary* rotary,
                                       const kvattn_cache_fp8* cache, void* q, int64_t q_stride, const void* k,
                                       int64_t k_stride, const void* v, int64_t v_stride, void* q_out,
                                       const int32_t* positions, const int32_t* seq_ids, const int32_t* block_table,
                                       int32_t num_seqs, int32_t max_blocks_per_seq, int32_t num_tokens, void* stream)
{
    if (!cache) return KVATTN_ERR_INVALID_ARG;
    const kvattn_cache c{cache->pool, cache->pool, cache->num_blocks, cache->block_size};
    return rotary_append_any(cfg, rotary, nullptr, nullptr, &c, true, q, q_stride, k, k_stride, v, v_stride, q_out, positions, seq_ids,
                             block_table, num_seqs, max_blocks_per_seq, num_tokens, stream);
}

kvattn_status kvattn_rotary_append_axes(const kvattn_config* cfg, const kvattn_rotary* rotary,
                                        const kvattn_rope_axes* axes, const kvattn_cache* cache, void* q,
                                        int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                                        int64_t v_stride, void* q_out, const int32_t* positions, const int32_t* slots,
                                        const int32_t* seq_ids, const int32_t* block_table, int32_t num_seqs,
                                        int32_t max_blocks_per_seq, int32_t num_tokens, void* stream)
{
    if (!axes) return KVATTN_ERR_INVALID_ARG;
    return rotary_append_any(cfg, rotary, axes, slots, cache, false, q, q_stride, k, k_stride, v, v_stride, q_out,
                             positions, seq_ids, block_table, num_seqs, max_blocks_per_seq, num_tokens, stream);
}

kvattn_status kvattn_rotary_append_axes_fp8(const kvattn_config* cfg, const kvattn_rotary* rotary,
                                            const kvattn_rope_axes* axes, const kvattn_cache_fp8* cache, void* q,
                                            int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                                            int64_t v_stride, void* q_out, const int32_t* positions,
                                            const int32_t* slots, const int32_t* seq_ids, const int32_t* block_table,
                                            int32_t num_seqs, int32_t max_blocks_per_seq, int32_t num_tokens,
                                            void* stream)
{
    if (!axes || !cache) return KVATTN_ERR_INVALID_ARG;
    const kvattn_cache c{cache->pool, cache->pool, cache->num_blocks, cache->block_size};
    return rotary_append_any(cfg, rotary, axes, slots, &c, true, q, q_stride, k, k_stride, v, v_stride, q_out, positions,
                             seq_ids, block_table, num_seqs, max_blocks_per_seq, num_tokens, stream);
}

namespace {

// bytes of one layer's K (or V) region, 0 if invalid or too large
int64_t layer_region_bytes(const kvattn_config* cfg, int32_t num_layers, int64_t num_blocks, int32_t block_size)
{
    if (!config_ok(cfg) || num_layers <= 0 || num_blocks <= 0 || block_size <= 0) return 0;
    const int64_t e = cfg->dtype == KVATTN_BF16 ? 2 : 4;
    const int64_t per_block = (int64_t)cfg->num_kv_heads * block_size * cfg->head_dim * e;
    if (per_block <= 0 || num_blocks > INT64_MAX / 4 / per_block / (2 * (int64_t)num_layers)) return 0;
    return num_blocks * per_block;
}

}  // namespace

size_t kvattn_layered_cache_bytes(const kvattn_config* cfg, int32_t num_layers, int64_t num_blocks,
                                  int32_t block_size)
{
    const int64_t region = layer_region_bytes(cfg, num_layers, num_blocks, block_size);
    return region ? (size_t)(region * 2 * num_layers) : 0;
}

kvattn_status kvattn_layer_cache(const kvattn_config* cfg, void* base, int32_t num_layers, int64_t num_blocks,
                                 int32_t block_size, int32_t layer, kvattn_cache* out)
{
    if (!out || !base || layer < 0 || layer >= num_layers) return KVATTN_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(base) & 15u) != 0) return KVATTN_ERR_INVALID_ARG;
    const int64_t region = layer_region_bytes(cfg, num_layers, num_blocks, block_size);
    if (!region) return KVATTN_ERR_INVALID_ARG;
    const kvattn_status st = config_supported(cfg);
    if (st != KVATTN_OK) return st;
    char* b = static_cast<char*>(base);
    out->k_pool = b + (2 * (int64_t)layer) * region;
    out->v_pool = b + (2 * (int64_t)layer + 1) * region;
    out->num_blocks = num_blocks;
    out->block_size = block_size;
    return KVATTN_OK;
}

namespace {

// block_bytes: of a region (kvattn_cache: of K or V; kvattn_cache_fp8: its pages)
int64_t region_block_bytes(const kvattn_config* cfg, bool fp8, int32_t block_size)
{
    if (fp8) return (int64_t)cfg->num_kv_heads * (block_size / 16) * kF8Page;
    return (int64_t)cfg->num_kv_heads * block_size * cfg->head_dim * (cfg->dtype == KVATTN_BF16 ? 2 : 4);
}

kvattn_status copy_blocks(char* k_base, char* v_base, int64_t layer_stride, int32_t regions, int64_t block_bytes,
                          int64_t num_blocks, const int32_t* src_ids, const int32_t* dst_ids, int32_t n, void* stream)
{
    if (n < 0) return KVATTN_ERR_INVALID_ARG;
    if (n == 0) return KVATTN_OK;
    if (!src_ids || !dst_ids) return KVATTN_ERR_INVALID_ARG;
    CopyArgs a;
    std::memset(&a, 0, sizeof(a));
    a.k_base = k_base;
    a.v_base = v_base;
    a.layer_stride = layer_stride;
    a.regions = regions;
    a.block_bytes = block_bytes;
    a.num_blocks = num_blocks;
    a.src = src_ids;
    a.dst = dst_ids;
    a.n = n;
    a.status = device_status_ptr();
    if (!a.status) return KVATTN_ERR_CUDA;
    return launch_copy_blocks(a, static_cast<cudaStream_t>(stream));
}

// A kvattn_cache_fp8 and the config that it needs.
kvattn_status fp8_cache_check(const kvattn_config* cfg, const kvattn_cache* c, int32_t max_blocks_per_seq)
{
    if (!config_ok(cfg) || !cache_ok(c, max_blocks_per_seq) || c->block_size % 16 != 0) return KVATTN_ERR_INVALID_ARG;
    const kvattn_status st = config_supported(cfg);
    if (st != KVATTN_OK) return st;
    return cfg->dtype != KVATTN_BF16 || cfg->head_dim != 128 ? KVATTN_ERR_UNSUPPORTED : KVATTN_OK;
}

kvattn_status compact_tokens(const kvattn_config* cfg, char* k_base, char* v_base, int64_t layer_stride, int32_t layers,
                             bool fp8, int64_t num_blocks, int32_t block_size, const int32_t* starts,
                             const int32_t* cu_keep, const int32_t* keep, int32_t total_keep,
                             const int32_t* block_table, int32_t num_seqs, int32_t max_blocks_per_seq, void* stream)
{
    if (num_seqs < 0 || total_keep < 0) return KVATTN_ERR_INVALID_ARG;
    if (num_seqs == 0 || total_keep == 0) return KVATTN_OK;
    if (!starts || !cu_keep || !keep || !block_table) return KVATTN_ERR_INVALID_ARG;
    CompactArgs a;
    std::memset(&a, 0, sizeof(a));
    a.k_base = k_base;
    a.v_base = v_base;
    a.layer_stride = layer_stride;
    a.layers = layers;
    a.fp8 = fp8 ? 1 : 0;
    a.hkv = cfg->num_kv_heads;
    a.row_bytes = cfg->head_dim * (cfg->dtype == KVATTN_BF16 ? 2 : 4);
    a.num_blocks = num_blocks;
    a.block_size = block_size;
    a.max_blocks = max_blocks_per_seq;
    a.num_seqs = num_seqs;
    a.total_keep = total_keep;
    a.starts = starts;
    a.cu = cu_keep;
    a.keep = keep;
    a.block_table = block_table;
    a.status = device_status_ptr();
    if (!a.status) return KVATTN_ERR_CUDA;
    return launch_compact(a, static_cast<cudaStream_t>(stream));
}

}  // namespace

kvattn_status kvattn_copy_blocks(const kvattn_config* cfg, const kvattn_cache* cache, const int32_t* src_ids,
                                 const int32_t* dst_ids, int32_t n, void* stream)
{
    if (!config_ok(cfg) || !cache_ok(cache, 1)) return KVATTN_ERR_INVALID_ARG;
    const kvattn_status st = config_supported(cfg);
    if (st != KVATTN_OK) return st;
    return copy_blocks(static_cast<char*>(cache->k_pool), static_cast<char*>(cache->v_pool), 0, 2,
                       region_block_bytes(cfg, false, cache->block_size), cache->num_blocks, src_ids, dst_ids, n, stream);
}

kvattn_status kvattn_copy_blocks_fp8(const kvattn_config* cfg, const kvattn_cache_fp8* cache, const int32_t* src_ids,
                                     const int32_t* dst_ids, int32_t n, void* stream)
{
    if (!cache) return KVATTN_ERR_INVALID_ARG;
    const kvattn_cache c{cache->pool, cache->pool, cache->num_blocks, cache->block_size};
    const kvattn_status st = fp8_cache_check(cfg, &c, 1);
    if (st != KVATTN_OK) return st;
    char* pool = static_cast<char*>(cache->pool);
    return copy_blocks(pool, pool, 0, 1, region_block_bytes(cfg, true, cache->block_size), cache->num_blocks, src_ids,
                       dst_ids, n, stream);
}

kvattn_status kvattn_copy_blocks_layered(const kvattn_config* cfg, void* base, int32_t num_layers,
                                         int64_t num_blocks, int32_t block_size, const int32_t* src_ids,
                                         const int32_t* dst_ids, int32_t n, void* stream)
{
    kvattn_cache first;
    const kvattn_status st = kvattn_layer_cache(cfg, base, num_layers, num_blocks, block_size, 0, &first);
    if (st != KVATTN_OK) return st;
    if (num_blocks > INT32_MAX) return KVATTN_ERR_INVALID_ARG;
    const int64_t region = static_cast<char*>(first.v_pool) - static_cast<char*>(first.k_pool);
    if (num_layers > INT32_MAX / 2) return KVATTN_ERR_UNSUPPORTED;
    return copy_blocks(static_cast<char*>(first.k_pool), static_cast<char*>(first.v_pool), 2 * region, 2 * num_layers,
                       region_block_bytes(cfg, false, block_size), num_blocks, src_ids, dst_ids, n, stream);
}

kvattn_status kvattn_compact_tokens(const kvattn_config* cfg, const kvattn_cache* cache, const int32_t* starts,
                                    const int32_t* cu_keep, const int32_t* keep, int32_t total_keep,
                                    const int32_t* block_table, int32_t num_seqs, int32_t max_blocks_per_seq,
                                    void* stream)
{
    if (!config_ok(cfg) || !cache_ok(cache, max_blocks_per_seq)) return KVATTN_ERR_INVALID_ARG;
    const kvattn_status st = config_supported(cfg);
    if (st != KVATTN_OK) return st;
    return compact_tokens(cfg, static_cast<char*>(cache->k_pool), static_cast<char*>(cache->v_pool), 0, 1, false,
                          cache->num_blocks, cache->block_size, starts, cu_keep, keep, total_keep, block_table, num_seqs,
                          max_blocks_per_seq, stream);
}

kvattn_status kvattn_compact_tokens_layered(const kvattn_config* cfg, void* base, int32_t num_layers,
                                            int64_t num_blocks, int32_t block_size, const int32_t* starts,
                                            const int32_t* cu_keep, const int32_t* keep, int32_t total_keep,
                                            const int32_t* block_table, int32_t num_seqs, int32_t max_blocks_per_seq,
                                            void* stream)
{
    kvattn_cache first;
    kvattn_status st = kvattn_layer_cache(cfg, base, num_layers, num_blocks, block_size, 0, &first);
    if (st != KVATTN_OK) return st;
    if (!cache_ok(&first, max_blocks_per_seq)) return KVATTN_ERR_INVALID_ARG;
    if (num_layers > INT32_MAX / 2) return KVATTN_ERR_UNSUPPORTED;
    char* k = static_cast<char*>(first.k_pool);
    char* v = static_cast<char*>(first.v_pool);
    return compact_tokens(cfg, k, v, 2 * (v - k), num_layers, false, num_blocks, block_size, starts, cu_keep, keep,
                          total_keep, block_table, num_seqs, max_blocks_per_seq, stream);
}

kvattn_status kvattn_compact_tokens_fp8(const kvattn_config* cfg, const kvattn_cache_fp8* cache, const int32_t* starts,
                                        const int32_t* cu_keep, const int32_t* keep, int32_t total_keep,
                                        const int32_t* block_table, int32_t num_seqs, int32_t max_blocks_per_seq,
                                        void* stream)
{
    if (!cache) return KVATTN_ERR_INVALID_ARG;
    const kvattn_cache c{cache->pool, cache->pool, cache->num_blocks, cache->block_size};
    const kvattn_status st = fp8_cache_check(cfg, &c, max_blocks_per_seq);
    if (st != KVATTN_OK) return st;
    char* pool = static_cast<char*>(cache->pool);
    return compact_tokens(cfg, pool, pool, 0, 1, true, cache->num_blocks, cache->block_size, starts, cu_keep, keep,
                          total_keep, block_table, num_seqs, max_blocks_per_seq, stream);
}

int32_t kvattn_decode_num_splits(const kvattn_config* cfg, int32_t batch, int32_t max_seq_len, int32_t num_splits)
{
    if (!config_ok(cfg) || config_supported(cfg) != KVATTN_OK || batch < 0 || max_seq_len < 0 || num_splits < 0)
        return 0;
    return decode_plan(batch, cfg->num_kv_heads, cfg->num_q_heads / cfg->num_kv_heads, max_seq_len, num_splits)
        .slots;
}

namespace {
// Workspace: [batch][segments] int32 piece counts | [batch][hq][slots][D] f32
// partial outputs | [batch][hq][slots][2] f32 (max, sum); each 256-byte aligned.
struct WorkspaceLayout {
    size_t nslots_off, o_off, ml_off, bytes;
};
WorkspaceLayout workspace_layout(const kvattn_config* cfg, int32_t batch, int32_t slots)
{
    auto up = [](size_t x) { return (x + 255) / 256 * 256; };
    WorkspaceLayout w;
    const size_t rows = (size_t)batch * cfg->num_q_heads * slots;
    w.nslots_off = 0;
    w.o_off = up((size_t)batch * decode_segments(cfg->num_q_heads, cfg->num_kv_heads) * 4);
    w.ml_off = w.o_off + up(rows * cfg->head_dim * 4);
    w.bytes = std::max<size_t>(256, w.ml_off + up(rows * 2 * 4));
    return w;
}
}  // namespace

size_t kvattn_decode_workspace_size(const kvattn_config* cfg, int32_t batch, int32_t max_seq_len,
                                    int32_t num_splits)
{
    const int32_t slots = kvattn_decode_num_splits(cfg, batch, max_seq_len, num_splits);
    if (slots <= 0) return 0;
    return workspace_layout(cfg, batch, slots).bytes;
}

namespace {

// The window of a call; window == 0: the whole cache.
struct DecodeWindow {
    int32_t window, sinks;
};

// Most keys that one query sees, rounded up to whole 16-token tiles.
int32_t window_span(int32_t max_seq_len, DecodeWindow w)
{
    if (w.window == 0) return max_seq_len;
    const int64_t tiles = ((int64_t)w.sinks + 15) / 16 + ((int64_t)w.window + 14) / 16 + 1;
    return (int32_t)std::min<int64_t>(max_seq_len, tiles * 16);
}

void decode_args(const kvattn_config* cfg, const kvattn_cache* cache, bool fp8, const void* q, const int32_t* block_table,
                 int32_t max_blocks_per_seq, const int32_t* seq_lens, int32_t batch, int32_t max_seq_len, int32_t slots,
                 void* out, void* workspace, DecodeArgs& a)
{
    std::memset(&a, 0, sizeof(a));
    a.q = q;
    a.k_pool = cache->k_pool;
    a.v_pool = cache->v_pool;
    a.block_table = block_table;
    a.seq_lens = seq_lens;
    a.out = out;
    if (slots > 1) {
        const WorkspaceLayout wl = workspace_layout(cfg, batch, slots);
        char* w = static_cast<char*>(workspace);
        a.nslots = reinterpret_cast<int32_t*>(w + wl.nslots_off);
        a.part_o = reinterpret_cast<float*>(w + wl.o_off);
        a.part_ml = reinterpret_cast<float*>(w + wl.ml_off);
    }
    a.num_blocks = cache->num_blocks;
    a.block_size = cache->block_size;
    a.max_blocks = max_blocks_per_seq;
    a.batch = batch;
    a.max_seq_len = max_seq_len;
    a.splits = slots;
    a.hq = cfg->num_q_heads;
    a.hkv = cfg->num_kv_heads;
    a.d = cfg->head_dim;
    a.dtype = cfg->dtype;
    a.scale_log2 = scale_of(cfg) * 1.4426950408889634f;
    a.fp8 = fp8 ? 1 : 0;
}

kvattn_status decode_any(const kvattn_config* cfg, const kvattn_cache* cache, bool fp8, DecodeWindow win,
                         const void* q, const int32_t* block_table, int32_t max_blocks_per_seq,
                         const int32_t* seq_lens, int32_t batch, int32_t max_seq_len, int32_t num_splits, void* out,
                         void* workspace, size_t workspace_bytes, void* stream)
{
    const kvattn_status st = decode_check(cfg, cache, fp8, q, block_table, max_blocks_per_seq, seq_lens, batch,
                                          max_seq_len, num_splits, out);
    if (st != KVATTN_OK || batch == 0) return st;
    const DecodePlan p = decode_plan(batch, cfg->num_kv_heads, cfg->num_q_heads / cfg->num_kv_heads,
                                     window_span(max_seq_len, win), num_splits);
    const WorkspaceLayout wl = workspace_layout(cfg, batch, p.slots);
    if (p.slots > 1) {
        if (!workspace || workspace_bytes < wl.bytes) return KVATTN_ERR_WORKSPACE_TOO_SMALL;
        if (reinterpret_cast<uintptr_t>(workspace) & 255u) return KVATTN_ERR_INVALID_ARG;
    }
    DecodeArgs a;
    decode_args(cfg, cache, fp8, q, block_table, max_blocks_per_seq, seq_lens, batch, max_seq_len, p.slots, out, workspace,
                a);
    a.status = device_status_ptr();
    if (!a.status) return KVATTN_ERR_CUDA;
    a.window = win.window;
    a.sinks = win.sinks;
    const int32_t max_tiles = num_splits ? 0 : (int32_t)(((int64_t)window_span(max_seq_len, win) + 15) / 16);
    return win.window ? launch_decode_window(a, max_tiles, static_cast<cudaStream_t>(stream))
                      : launch_decode(a, static_cast<cudaStream_t>(stream));
}

}  // namespace

kvattn_status kvattn_decode(const kvattn_config* cfg, const kvattn_cache* cache, const void* q,
                            const int32_t* block_table, int32_t max_blocks_per_seq, const int32_t* seq_lens,
                            int32_t batch, int32_t max_seq_len, int32_t num_splits, void* out, void* workspace,
                            size_t workspace_bytes, void* stream)
{
    return decode_any(cfg, cache, false, {0, 0}, q, block_table, max_blocks_per_seq, seq_lens, batch, max_seq_len,
                      num_splits, out, workspace, workspace_bytes, stream);
}

kvattn_status kvattn_decode_fp8(const kvattn_config* cfg, const kvattn_cache_fp8* cache, const void* q,
                                const int32_t* block_table, int32_t max_blocks_per_seq, const int32_t* seq_lens,
                                int32_t batch, int32_t max_seq_len, int32_t num_splits, void* out, void* workspace,
                                size_t workspace_bytes, void* stream)
{
    if (!cache) return KVATTN_ERR_INVALID_ARG;
    const kvattn_cache c{cache->pool, cache->pool, cache->num_blocks, cache->block_size};
    return decode_any(cfg, &c, true, {0, 0}, q, block_table, max_blocks_per_seq, seq_lens, batch, max_seq_len,
                      num_splits, out, workspace, workspace_bytes, stream);
}

size_t kvattn_decode_window_workspace_size(const kvattn_config* cfg, int32_t batch, int32_t max_seq_len,
                                           int32_t window, int32_t num_sinks, int32_t num_splits)
{
    if (window < 1 || num_sinks < 0 || max_seq_len < 0) return 0;
    return kvattn_decode_workspace_size(cfg, batch, window_span(max_seq_len, {window, num_sinks}), num_splits);
}

kvattn_status kvattn_decode_window(const kvattn_config* cfg, const kvattn_cache* cache, const void* q,
                                   const int32_t* block_table, int32_t max_blocks_per_seq, const int32_t* seq_lens,
                                   int32_t batch, int32_t max_seq_len, int32_t window, int32_t num_sinks,
                                   int32_t num_splits, void* out, void* workspace, size_t workspace_bytes,
                                   void* stream)
{
    if (window < 1 || num_sinks < 0) return KVATTN_ERR_INVALID_ARG;
    return decode_any(cfg, cache, false, {window, num_sinks}, q, block_table, max_blocks_per_seq, seq_lens, batch,
                      max_seq_len, num_splits, out, workspace, workspace_bytes, stream);
}

kvattn_status kvattn_decode_window_fp8(const kvattn_config* cfg, const kvattn_cache_fp8* cache, const void* q,
                                       const int32_t* block_table, int32_t max_blocks_per_seq,
                                       const int32_t* seq_lens, int32_t batch, int32_t max_seq_len, int32_t window,
                                       int32_t num_sinks, int32_t num_splits, void* out, void* workspace,
                                       size_t workspace_bytes, void* stream)
{
    if (!cache || window < 1 || num_sinks < 0) return KVATTN_ERR_INVALID_ARG;
    const kvattn_cache c{cache->pool, cache->pool, cache->num_blocks, cache->block_size};
    return decode_any(cfg, &c, true, {window, num_sinks}, q, block_table, max_blocks_per_seq, seq_lens, batch,
                      max_seq_len, num_splits, out, workspace, workspace_bytes, stream);
}

namespace {

bool groups_ok(int32_t batch, int32_t num_groups, int32_t max_shared_len)
{
    return num_groups >= 0 && num_groups <= batch && max_shared_len >= 0;
}

// Whether prefixes are read once: if they save enough, by the call's bounds.  That form
// starts with a plan and ends with a merge, 12 us together at least; a prefix of a few rows costs
// it as much as one of 128; and beside the prefixes of several groups it reads own fp8 pages slower
// than decode_direct.cu does.
// Measured over batches of 2 to 64, prefixes of 128 to 8192 tokens and own parts of up
// to 32 to 2048 (us, once / each sequence by itself): bf16, saved MB 25 (2 x 8192, 12/12
// heads of 64): 16.8 / 12.6; 33 (64 x 128, 32/8 heads of 128): 13.7 / 8.0; 94 (16 x 2048,
// 12/12 heads): 19.9 / 30.4 with 2048 own tokens and 12.0 / 18.8 with 512; 528 (64 x 2048,
// 32/8): 32.1 / 93.8.
// Own keys do not count for bf16: the stream of own pages is no slower than the other form's, saved
// and own MB (bound) 41 and 1342 (80 x 128, 32/8 heads): 121 / 131; 65 and 1074 (32 x 512): 87 / 94; 50 and
// 805 (128 x 128, 12/12 heads of 64): 72 / 79; 66 and 1074 (64 x 256) with 8/8, 16/8 and 64/8 heads:
// 105 / 107, 106 / 110 and 109 / 123; and many sequences go better this way even where a bound of
// 128 lets nothing be shared (256 of 127 and up to 512 own tokens, 32/8 heads: 61 / 89).
// fp8, 138 shapes of 64/8, 32/8 and 8/2 heads, 4 to 128 sequences in 1 to 16 groups, 512 to 8192 shared
// and up to 64 to 4096 own tokens; saved and own MB.  One group: 52 and 9 (64/8) 23.0 / 17.5; 65 and 138 33.3 /
// 32.3; 68 and 554 85 / 83; 137 and 17 34.3 / 26.9 (32/8: 20.5 / 25.5); 272 and 138 (8/2) 35.4 / 76.2; 272
// and 554 84 / 110; 549 and 1107 132 / 176: own keys make no difference.  8 groups (64/8): 61 and 554
// 113 / 79; 242 and 138 64 / 60; 242 and 554 124 / 106; 969 and 554 186 / 255; 16 groups, 121 and 17
// 42 / 28; 484 and 277 101 / 102; 484 and 1107 218 / 178; 1938 and 1107 313 / 475.  The rule's choice
// takes 0.4 % more than the better one on the mean, 28 % at most.  Since max_seq_len may be far above the lengths (a
// step captured for what it may grow to), own keys count up to twice the saved bytes only, so that from
// 200 MB and 5 for each group and KV head on prefixes are shared at any bound: by the bound alone
// the choice takes 3 % more than the better one, 63 % at most.
bool prefixes_once(const kvattn_config* cfg, bool fp8, int32_t batch, int32_t max_seq_len, int32_t num_groups,
                   int32_t max_shared_len)
{
    const double token = (double)cfg->num_kv_heads * (fp8 ? kF8Page / 16 : 4 * cfg->head_dim);
    const double saved = token * (batch - num_groups) * max_shared_len;
    if (!fp8) return saved >= 40e6;
    const double own = num_groups > 1 ? token * batch * std::max(0, max_seq_len - max_shared_len) : 0.;
    return saved >= 80e6 + 2e6 * num_groups * cfg->num_kv_heads + 0.3 * std::min(own, 2. * saved);
}

// Workspace of the form that reads prefixes once (SharedArgs), each part 256-byte
// aligned.  bytes == 0: this call cannot take that form.
struct SharedLayout {
    size_t o_off, ml_off, own_o_off, own_ml_off, bytes;
};
SharedLayout shared_layout(const kvattn_config* cfg, int32_t batch, int32_t max_seq_len, int32_t num_groups,
                           int32_t max_shared_len)
{
    SharedLayout l{};
    if (cfg->dtype != KVATTN_BF16 || num_groups < 1 || num_groups > kMaxGroups || batch < 2 || batch > kMaxSharedBatch ||
        max_shared_len < 16)
        return l;
    const int32_t hkv = cfg->num_kv_heads, ctas = num_sms();
    const int64_t pieces = shared_pieces(cfg->num_q_heads, hkv, batch, num_groups, ctas);
    // (the streams' pages are counted in 32 bits)
    const int64_t pages = pieces * ((int64_t)max_shared_len / 16 + 1) + (int64_t)batch * hkv * ((int64_t)max_seq_len / 16 + 1);
    if (pages > (1 << 30)) return l;
    const size_t rows = (size_t)ctas * kSharedRows + (size_t)batch * cfg->num_q_heads;
    if (rows > INT32_MAX) return l;
    const size_t own_rows = (size_t)own_pieces(hkv, batch, ctas) * (cfg->num_q_heads / hkv);
    auto up = [](size_t x) { return (x + 255) / 256 * 256; };
    l.o_off = up((size_t)batch * sizeof(SharedOf));
    l.ml_off = l.o_off + up(rows * cfg->head_dim * 4);
    l.own_o_off = l.ml_off + up(rows * 2 * 4);
    l.own_ml_off = l.own_o_off + up(own_rows * cfg->head_dim * 4);
    l.bytes = l.own_ml_off + up(own_rows * 2 * 4);
    return l;
}

kvattn_status decode_shared_any(const kvattn_config* cfg, const kvattn_cache* cache, bool fp8, const void* q,
                                const int32_t* block_table, int32_t max_blocks_per_seq, const int32_t* seq_lens,
                                int32_t batch, int32_t max_seq_len, const int32_t* cu_groups,
                                const int32_t* shared_lens, int32_t num_groups, int32_t max_shared_len, void* out,
                                void* workspace, size_t workspace_bytes, void* stream)
{
    if (batch >= 0 && !groups_ok(batch, num_groups, max_shared_len)) return KVATTN_ERR_INVALID_ARG;
    if (num_groups > 0 && (!cu_groups || !shared_lens)) return KVATTN_ERR_INVALID_ARG;
    const kvattn_status st = decode_check(cfg, cache, fp8, q, block_table, max_blocks_per_seq, seq_lens, batch,
                                          max_seq_len, 0, out);
    if (st != KVATTN_OK || batch == 0) return st;
    const SharedLayout l = shared_layout(cfg, batch, max_seq_len, num_groups, max_shared_len);
    const bool once = l.bytes > 0 && prefixes_once(cfg, fp8, batch, max_seq_len, num_groups, max_shared_len) &&
                      cache->block_size % 16 == 0 &&
                      cache->num_blocks * cfg->num_kv_heads < ((int64_t)1 << 31) / cache->block_size;
    if (!once)  // every sequence by itself
        return decode_any(cfg, cache, fp8, {INT32_MAX, 0}, q, block_table, max_blocks_per_seq, seq_lens, batch,
                          max_seq_len, 0, out, workspace, workspace_bytes, stream);
    if (!workspace || workspace_bytes < l.bytes) return KVATTN_ERR_WORKSPACE_TOO_SMALL;
    if (reinterpret_cast<uintptr_t>(workspace) & 255u) return KVATTN_ERR_INVALID_ARG;
    SharedArgs a;
    std::memset(&a, 0, sizeof(a));
    decode_args(cfg, cache, fp8, q, block_table, max_blocks_per_seq, seq_lens, batch, max_seq_len, 1, out, nullptr, a.d);
    a.d.status = device_status_ptr();
    if (!a.d.status) return KVATTN_ERR_CUDA;
    char* w = static_cast<char*>(workspace);
    a.of = reinterpret_cast<SharedOf*>(w);
    a.o = reinterpret_cast<float*>(w + l.o_off);
    a.ml = reinterpret_cast<float*>(w + l.ml_off);
    a.own_o = reinterpret_cast<float*>(w + l.own_o_off);
    a.own_ml = reinterpret_cast<float*>(w + l.own_ml_off);
    a.cu_groups = cu_groups;
    a.shared_lens = shared_lens;
    a.num_groups = num_groups;
    a.max_shared = max_shared_len;
    return launch_decode_shared(a, static_cast<cudaStream_t>(stream));
}

}  // namespace

size_t kvattn_decode_shared_workspace_size(const kvattn_config* cfg, int32_t batch, int32_t max_seq_len,
                                           int32_t num_groups, int32_t max_shared_len)
{
    if (batch < 0 || max_seq_len < 0 || !groups_ok(batch, num_groups, max_shared_len)) return 0;
    const size_t alone = kvattn_decode_window_workspace_size(cfg, batch, max_seq_len, INT32_MAX, 0, 0);
    if (alone == 0) return 0;
    auto once = [&](bool fp8) { return prefixes_once(cfg, fp8, batch, max_seq_len, num_groups, max_shared_len); };
    if (!once(false) && !(cfg->head_dim == 128 && once(true))) return alone;
    return std::max(alone, shared_layout(cfg, batch, max_seq_len, num_groups, max_shared_len).bytes);
}

kvattn_status kvattn_decode_shared(const kvattn_config* cfg, const kvattn_cache* cache, const void* q,
                                   const int32_t* block_table, int32_t max_blocks_per_seq, const int32_t* seq_lens,
                                   int32_t batch, int32_t max_seq_len, const int32_t* cu_groups,
                                   const int32_t* shared_lens, int32_t num_groups, int32_t max_shared_len, void* out,
                                   void* workspace, size_t workspace_bytes, void* stream)
{
    return decode_shared_any(cfg, cache, false, q, block_table, max_blocks_per_seq, seq_lens, batch, max_seq_len, cu_groups,
                             shared_lens, num_groups, max_shared_len, out, workspace, workspace_bytes, stream);
}

kvattn_status kvattn_decode_shared_fp8(const kvattn_config* cfg, const kvattn_cache_fp8* cache, const void* q,
                                       const int32_t* block_table, int32_t max_blocks_per_seq,
                                       const int32_t* seq_lens, int32_t batch, int32_t max_seq_len,
                                       const int32_t* cu_groups, const int32_t* shared_lens, int32_t num_groups,
                                       int32_t max_shared_len, void* out, void* workspace, size_t workspace_bytes,
                                       void* stream)
{
    if (!cache) return KVATTN_ERR_INVALID_ARG;
    const kvattn_cache c{cache->pool, cache->pool, cache->num_blocks, cache->block_size};
    return decode_shared_any(cfg, &c, true, q, block_table, max_blocks_per_seq, seq_lens, batch, max_seq_len, cu_groups,
                             shared_lens, num_groups, max_shared_len, out, workspace, workspace_bytes, stream);
}

kvattn_status kvattn_rope_append_fp8(const kvattn_config* cfg, const kvattn_cache_fp8* cache, void* q,
                                     const void* k, const void* v, const int32_t* positions, const int32_t* seq_ids,
                                     const int32_t* block_table, int32_t num_seqs, int32_t max_blocks_per_seq,
                                     int32_t num_tokens, void* stream)
{
    if (!config_ok(cfg) || num_tokens < 0 || num_seqs <= 0 || !cache) return KVATTN_ERR_INVALID_ARG;
    kvattn_status st = config_supported(cfg);
    if (st != KVATTN_OK) return st;
    if (cfg->dtype != KVATTN_BF16 || cfg->head_dim != 128) return KVATTN_ERR_UNSUPPORTED;
    const kvattn_cache c{cache->pool, cache->pool, cache->num_blocks, cache->block_size};
    if (!cache_ok(&c, max_blocks_per_seq) || cache->block_size % 16 != 0) return KVATTN_ERR_INVALID_ARG;
    if (num_tokens == 0) return KVATTN_OK;
    if (!q || !k || !v || !positions || !seq_ids || !block_table) return KVATTN_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(v)) & 15u)
        return KVATTN_ERR_INVALID_ARG;
    RopeArgs a;
    std::memset(&a, 0, sizeof(a));
    const int64_t qrow = (int64_t)cfg->num_q_heads * cfg->head_dim * 2;
    const int64_t kvrow = (int64_t)cfg->num_kv_heads * cfg->head_dim * 2;
    a.q = q;
    a.k = k;
    a.v = v;
    a.q_stride = qrow;
    a.k_stride = kvrow;
    a.v_stride = kvrow;
    a.q_out = q;
    a.q_out_stride = qrow;
    a.k_pool = cache->pool;
    a.v_pool = cache->pool;
    a.fp8 = 1;
    a.positions = positions;
    a.seq_ids = seq_ids;
    a.block_table = block_table;
    a.num_blocks = cache->num_blocks;
    a.block_size = cache->block_size;
    a.num_seqs = num_seqs;
    a.max_blocks = max_blocks_per_seq;
    a.num_tokens = num_tokens;
    a.hq = cfg->num_q_heads;
    a.hkv = cfg->num_kv_heads;
    a.d = cfg->head_dim;
    a.dtype = cfg->dtype;
    a.status = device_status_ptr();
    if (!a.status) return KVATTN_ERR_CUDA;
    rope_tables((double)cfg->rope_base, cfg->head_dim, a);
    return launch_rope_append_fp8(a, static_cast<cudaStream_t>(stream));
}

kvattn_status kvattn_prefill_chunk(const kvattn_config* cfg, const kvattn_cache* cache, const void* q,
                                   const int32_t* cu_q_lens, const int32_t* prefix_lens,
                                   const int32_t* block_table, int32_t max_blocks_per_seq, int32_t num_chunks,
                                   int32_t max_q_len, int32_t total_q, void* out, void* stream)
{
    if (!config_ok(cfg) || num_chunks < 0 || max_q_len < 0 || total_q < 0) return KVATTN_ERR_INVALID_ARG;
    kvattn_status st = config_supported(cfg);
    if (st != KVATTN_OK) return st;
    if (cfg->dtype != KVATTN_BF16 || (cfg->head_dim != 128 && cfg->head_dim != 64)) return KVATTN_ERR_UNSUPPORTED;
    if (!cache_ok(cache, max_blocks_per_seq)) return KVATTN_ERR_INVALID_ARG;
    if (cache->block_size % 16 != 0) return KVATTN_ERR_UNSUPPORTED;
    if (num_chunks == 0 || total_q == 0) return KVATTN_OK;
    if (!q || !cu_q_lens || !prefix_lens || !block_table || !out) return KVATTN_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(out)) & 15u) return KVATTN_ERR_INVALID_ARG;
    PrefillArgs a;
    std::memset(&a, 0, sizeof(a));
    a.q = q;
    a.k_pool = cache->k_pool;
    a.v_pool = cache->v_pool;
    a.cu_q_lens = cu_q_lens;
    a.prefix_lens = prefix_lens;
    a.block_table = block_table;
    a.out = out;
    a.num_blocks = cache->num_blocks;
    a.block_size = cache->block_size;
    a.max_blocks = max_blocks_per_seq;
    a.num_chunks = num_chunks;
    a.max_q_len = max_q_len;
    a.total_q = total_q;
    a.hq = cfg->num_q_heads;
    a.hkv = cfg->num_kv_heads;
    a.d = cfg->head_dim;
    a.scale_log2 = scale_of(cfg) * 1.4426950408889634f;
    a.status = device_status_ptr();
    if (!a.status) return KVATTN_ERR_CUDA;
    return launch_prefill(a, static_cast<cudaStream_t>(stream));
}

size_t kvattn_prefill_fp8_workspace_size(const kvattn_config* cfg, int32_t block_size, int32_t max_blocks_per_seq,
                                         int32_t num_chunks, int64_t max_kv_tokens)
{
    if (!config_ok(cfg) || config_supported(cfg) != KVATTN_OK) return 0;
    if (cfg->dtype != KVATTN_BF16 || cfg->head_dim != 128) return 0;
    return fp8_prefill_layout(cfg->num_kv_heads, block_size, max_blocks_per_seq, num_chunks, max_kv_tokens).bytes;
}

kvattn_status kvattn_prefill_chunk_fp8(const kvattn_config* cfg, const kvattn_cache_fp8* cache, const void* q,
                                       const int32_t* cu_q_lens, const int32_t* prefix_lens,
                                       const int32_t* block_table, int32_t max_blocks_per_seq, int32_t num_chunks,
                                       int32_t max_q_len, int32_t total_q, int64_t max_kv_tokens, void* out,
                                       void* workspace, size_t workspace_bytes, void* stream)
{
    if (!config_ok(cfg) || num_chunks < 0 || max_q_len < 0 || total_q < 0 || max_kv_tokens < 0 || !cache)
        return KVATTN_ERR_INVALID_ARG;
    kvattn_status st = config_supported(cfg);
    if (st != KVATTN_OK) return st;
    if (cfg->dtype != KVATTN_BF16 || cfg->head_dim != 128) return KVATTN_ERR_UNSUPPORTED;
    const kvattn_cache c{cache->pool, cache->pool, cache->num_blocks, cache->block_size};
    if (!cache_ok(&c, max_blocks_per_seq) || cache->block_size % 16 != 0) return KVATTN_ERR_INVALID_ARG;
    if (num_chunks == 0 || total_q == 0) return KVATTN_OK;
    if (!q || !cu_q_lens || !prefix_lens || !block_table || !out || !workspace) return KVATTN_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(out)) & 15u) return KVATTN_ERR_INVALID_ARG;
    const Fp8PrefillLayout L =
        fp8_prefill_layout(cfg->num_kv_heads, cache->block_size, max_blocks_per_seq, num_chunks, max_kv_tokens);
    if (L.bytes == 0) return KVATTN_ERR_INVALID_ARG;
    if (workspace_bytes < L.bytes) return KVATTN_ERR_WORKSPACE_TOO_SMALL;
    PrefillArgs a;
    std::memset(&a, 0, sizeof(a));
    a.q = q;
    a.cu_q_lens = cu_q_lens;
    a.prefix_lens = prefix_lens;
    a.block_table = block_table;
    a.out = out;
    a.num_blocks = cache->num_blocks;
    a.block_size = cache->block_size;
    a.max_blocks = max_blocks_per_seq;
    a.num_chunks = num_chunks;
    a.max_q_len = max_q_len;
    a.total_q = total_q;
    a.hq = cfg->num_q_heads;
    a.hkv = cfg->num_kv_heads;
    a.d = cfg->head_dim;
    a.scale_log2 = scale_of(cfg) * 1.4426950408889634f;
    a.status = device_status_ptr();
    if (!a.status) return KVATTN_ERR_CUDA;
    return launch_prefill_fp8(a, cache->pool, L, workspace, static_cast<cudaStream_t>(stream));
}

namespace {

// Checks shared by the two windowed prefills, and their kernel arguments.
// Nothing to do (*todo false) is KVATTN_OK.
kvattn_status prefill_window_args(const kvattn_config* cfg, const kvattn_cache* cache, const void* q,
                                  const int32_t* cu_q_lens, const int32_t* prefix_lens, const int32_t* block_table,
                                  int32_t max_blocks_per_seq, int32_t num_chunks, int32_t max_q_len, int32_t total_q,
                                  int32_t window, int32_t num_sinks, void* out, PrefillArgs& a, bool* todo)
{
    *todo = false;
    if (!config_ok(cfg) || num_chunks < 0 || max_q_len < 0 || total_q < 0 || window < 1 || num_sinks < 0)
        return KVATTN_ERR_INVALID_ARG;
    const kvattn_status st = config_supported(cfg);
    if (st != KVATTN_OK) return st;
    if (cfg->dtype != KVATTN_BF16) return KVATTN_ERR_UNSUPPORTED;
    if (!cache_ok(cache, max_blocks_per_seq)) return KVATTN_ERR_INVALID_ARG;
    if (cache->block_size % 16 != 0) return KVATTN_ERR_UNSUPPORTED;
    if (num_chunks == 0 || total_q == 0 || max_q_len == 0) return KVATTN_OK;
    if (!q || !cu_q_lens || !prefix_lens || !block_table || !out) return KVATTN_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(out)) & 15u) return KVATTN_ERR_INVALID_ARG;
    std::memset(&a, 0, sizeof(a));
    a.q = q;
    a.k_pool = cache->k_pool;
    a.v_pool = cache->v_pool;
    a.cu_q_lens = cu_q_lens;
    a.prefix_lens = prefix_lens;
    a.block_table = block_table;
    a.out = out;
    a.num_blocks = cache->num_blocks;
    a.block_size = cache->block_size;
    a.max_blocks = max_blocks_per_seq;
    a.num_chunks = num_chunks;
    a.max_q_len = max_q_len;
    a.total_q = total_q;
    a.hq = cfg->num_q_heads;
    a.hkv = cfg->num_kv_heads;
    a.d = cfg->head_dim;
    a.scale_log2 = scale_of(cfg) * 1.4426950408889634f;
    a.window = std::min(window, kMaxWindowKeys);
    a.sinks = std::min(num_sinks, kMaxWindowKeys);
    *todo = true;
    return KVATTN_OK;
}

}  // namespace

kvattn_status kvattn_prefill_window(const kvattn_config* cfg, const kvattn_cache* cache, const void* q,
                                    const int32_t* cu_q_lens, const int32_t* prefix_lens, const int32_t* block_table,
                                    int32_t max_blocks_per_seq, int32_t num_chunks, int32_t max_q_len,
                                    int32_t total_q, int32_t window, int32_t num_sinks, void* out, void* stream)
{
    PrefillArgs a;
    bool todo;
    const kvattn_status st = prefill_window_args(cfg, cache, q, cu_q_lens, prefix_lens, block_table,
                                                 max_blocks_per_seq, num_chunks, max_q_len, total_q, window, num_sinks,
                                                 out, a, &todo);
    if (!todo) return st;
    a.status = device_status_ptr();
    if (!a.status) return KVATTN_ERR_CUDA;
    return launch_prefill_window(a, static_cast<cudaStream_t>(stream));
}

size_t kvattn_prefill_window_fp8_workspace_size(const kvattn_config* cfg, int32_t block_size,
                                                int32_t max_blocks_per_seq, int32_t num_chunks, int32_t max_q_len,
                                                int32_t window, int32_t num_sinks)
{
    if (!config_ok(cfg) || config_supported(cfg) != KVATTN_OK) return 0;
    if (cfg->dtype != KVATTN_BF16 || cfg->head_dim != 128) return 0;
    return fp8_window_layout(cfg->num_kv_heads, block_size, max_blocks_per_seq, num_chunks, max_q_len, window,
                             num_sinks).bytes;
}

kvattn_status kvattn_prefill_window_fp8(const kvattn_config* cfg, const kvattn_cache_fp8* cache, const void* q,
                                        const int32_t* cu_q_lens, const int32_t* prefix_lens,
                                        const int32_t* block_table, int32_t max_blocks_per_seq, int32_t num_chunks,
                                        int32_t max_q_len, int32_t total_q, int32_t window, int32_t num_sinks,
                                        void* out, void* workspace, size_t workspace_bytes, void* stream)
{
    if (!cache) return KVATTN_ERR_INVALID_ARG;
    const kvattn_cache c{cache->pool, cache->pool, cache->num_blocks, cache->block_size};
    PrefillArgs a;
    bool todo;
    const kvattn_status st = prefill_window_args(cfg, &c, q, cu_q_lens, prefix_lens, block_table, max_blocks_per_seq,
                                                 num_chunks, max_q_len, total_q, window, num_sinks, out, a, &todo);
    if (st != KVATTN_OK) return st;
    if (cfg->head_dim != 128) return KVATTN_ERR_UNSUPPORTED;
    if (!todo) return st;
    if (!workspace) return KVATTN_ERR_INVALID_ARG;
    const Fp8WindowLayout L = fp8_window_layout(cfg->num_kv_heads, cache->block_size, max_blocks_per_seq, num_chunks,
                                                max_q_len, window, num_sinks);
    if (L.bytes == 0) return KVATTN_ERR_INVALID_ARG;
    if (workspace_bytes < L.bytes) return KVATTN_ERR_WORKSPACE_TOO_SMALL;
    a.status = device_status_ptr();
    if (!a.status) return KVATTN_ERR_CUDA;
    return launch_prefill_window_fp8(a, cache->pool, L, workspace, static_cast<cudaStream_t>(stream));
}

kvattn_status kvattn_selftest_wait_timeout(int32_t limit_us, void* stream)
{
    if (limit_us < 1 || limit_us > 1000000) return KVATTN_ERR_INVALID_ARG;
    int* st = device_status_ptr();
    if (!st) return KVATTN_ERR_CUDA;
    selftest_timeout_kernel<<<1, 32, 0, static_cast<cudaStream_t>(stream)>>>(st, (uint64_t)limit_us * 1000ull);
    return cuda_status(cudaGetLastError());
}

kvattn_status kvattn_get_device_status(void* stream, int32_t* out)
{
    if (!out) return KVATTN_ERR_INVALID_ARG;
    int* p = device_status_ptr();
    if (!p) return KVATTN_ERR_CUDA;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (cudaStreamSynchronize(s) != cudaSuccess) return KVATTN_ERR_CUDA;
    int v = 0;
    if (cudaMemcpy(&v, p, sizeof(int), cudaMemcpyDeviceToHost) != cudaSuccess) return KVATTN_ERR_CUDA;
    const int zero = 0;
    if (cudaMemcpy(p, &zero, sizeof(int), cudaMemcpyHostToDevice) != cudaSuccess) return KVATTN_ERR_CUDA;
    *out = v;
    return KVATTN_OK;
}

}  // extern "C"
