// gdn_attn_bf16.cu -- gdn_attn_decode over a bf16 cache: mma.sync with the keys (and the channels of the values)
// on the 16-row side and 8 query rows a warp (16 where more would not fit the registers) on the other, so that the
// few rows of a decode step fill the instruction; see gdn_attn.cuh.
//
// Measured, 64 ragged sequences of up to 8192 keys (0.54 GB), 16/2 heads of 256: 8 rows 94 us, 16 rows 96, 24 rows 108, 32 rows
// 121; of up to 16384 keys, 24/4 heads (2.2 GB): 333 us (6.5 TB/s).  fp32 results, three parts a weight: 24 rows 125, 64 rows 278, 128
// rows 576 (floors 81 to 85).  Eight rows a warp and more warps hide the
// products' latencies better than 16 rows a warp, which read the keys and values from shared memory once for twice the
// rows: 16 rows took 123 us that way against 103, 24 rows 131 against 117 (before the groups' cost was weighed as it is
// now); at 32 rows the registers of 16 computing warps no longer suffice.
#include "gdn_attn.cuh"

namespace gdn {
namespace attn {

namespace {

using bf16 = __nv_bfloat16;

// 4 key groups as long as the rows fit, then 2 and 1.  More than 32 rows only come here with an fp32 result.
template <int D, int PIECES>
cudaError_t by_rows(const AttnParams& p, bool out_bf16, int sms, cudaStream_t stream) {
    const int R = p.G * p.K;
    if (R <= 8) return launch<Shape<bf16, D, 1, 1, 4, PIECES>>(p, out_bf16, sms, stream);
    if (R <= 16) return launch<Shape<bf16, D, 1, 2, 4, PIECES>>(p, out_bf16, sms, stream);
    if (R <= 24) return launch<Shape<bf16, D, 1, 3, 4, PIECES>>(p, out_bf16, sms, stream);
    if constexpr (PIECES == 3) {
        if (R > 64) return launch<Shape<bf16, D, 2, 8, 1, PIECES>>(p, out_bf16, sms, stream);
        if (R > 32) return launch<Shape<bf16, D, 2, 4, 2, PIECES>>(p, out_bf16, sms, stream);
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
