// Split-KV decode attention over the whole cache of each sequence: split plan
// and launch (kernels: decode_kernel.cuh).
#include "decode_kernel.cuh"

namespace kvattn {

DecodePlan decode_plan(int32_t batch, int32_t hkv, int32_t group, int32_t max_seq_len, int32_t splits)
{
    DecodePlan p;
    const int max_tiles = std::max(1, (max_seq_len + kTile - 1) / kTile);
    if (splits > 0) {
        p.slots = splits;
    } else {
        // Flat decomposition with at most `slots` pieces per segment: a CTA
        // range holds ceil(total / grid) tiles, and the piece cap forces at
        // least ceil(max_tiles / (slots - 1)) per range.  With lengths spread
        // up to max_seq_len the total is about batch*segments*max_tiles/2, so
        // slots - 1 >= 4 * grid / (batch * segments) keeps the cap inactive
        // with a factor-2 margin.
        const int nsub = group > 4 ? group / 4 : 1;
        const int64_t segs = std::max<int64_t>(1, (int64_t)batch * hkv * nsub);
        const int64_t grid = (int64_t)num_sms() * 3;
        const int64_t want = 1 + (4 * grid + segs - 1) / segs;
        p.slots = (int32_t)std::max<int64_t>(3, std::min<int64_t>(16, want));
    }
    p.slots = std::min(p.slots, max_tiles + 1);
    if (p.slots < 1) p.slots = 1;
    return p;
}

kvattn_status launch_decode(const DecodeArgs& a, cudaStream_t s) { return dispatch<false>(a, s); }

}  // namespace kvattn
