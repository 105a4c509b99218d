// gdn_attn_bf16.cu -- gdn_attn_decode over a bf16 cache: mma.sync with the keys (and the channels of the values)
// on the 16-row side and 8 or 16 query rows a warp on the other, so that the few rows of a decode step
// fill the instruction; see gdn_attn.cuh.
#include "gdn_attn.cuh"

namespace gdn {
namespace attn {

namespace {

using bf16 = __nv_bfloat16;

// Warps by rows: 4 key groups as long as the rows fit two warps of 16, then 2 and 1 (8 warps hold 224 registers each).
// More than 32 rows only come here with an fp32 result.
template <int D, int PIECES>
cudaError_t by_rows(const AttnParams& p, bool out_bf16, int sms, cudaStream_t stream) {
    const int n = block_rows(p.G * p.K, true);
    if (n == 8) return launch<Shape<bf16, D, 1, 1, 4, PIECES>>(p, out_bf16, sms, stream);
    if (n == 16) return launch<Shape<bf16, D, 2, 1, 4, PIECES>>(p, out_bf16, sms, stream);
    if constexpr (PIECES == 3) {
        if (n == 64) return launch<Shape<bf16, D, 2, 4, 2, PIECES>>(p, out_bf16, sms, stream);
        if (n == 128) return launch<Shape<bf16, D, 2, 8, 1, PIECES>>(p, out_bf16, sms, stream);
    }
    return launch<Shape<bf16, D, 2, 2, 4, PIECES>>(p, out_bf16, sms, stream);
}

template <int D>
cudaError_t by_out(const AttnParams& p, bool out_bf16, int sms, cudaStream_t stream) {
    return out_bf16 ? by_rows<D, 2>(p, true, sms, stream) : by_rows<D, 3>(p, false, sms, stream);
}

}  // namespace

cudaError_t launch_bf16(const AttnParams& p, int head_dim, bool out_bf16, int sms, cudaStream_t stream) {
    if (head_dim == 64) return by_out<64>(p, out_bf16, sms, stream);
    if (head_dim == 128) return by_out<128>(p, out_bf16, sms, stream);
    return by_out<256>(p, out_bf16, sms, stream);
}

}  // namespace attn
}  // namespace gdn
