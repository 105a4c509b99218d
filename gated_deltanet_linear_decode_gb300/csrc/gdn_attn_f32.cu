// gdn_attn_f32.cu -- gdn_attn_decode over an fp32 cache: fp32 products and sums on the CUDA cores, 2 to 8 rows a
// warp; see gdn_attn.cuh.
//
// But for heads of 256 with up to 4 rows, the products bind and not the memory: every row that a warp has costs its products, the
// reduction over the lanes and the weights' way to them whether a query stands in it or not, and a second warp a scheduler
// hides their latencies.  16 ragged sequences of up to 4096 keys, 8 kv heads, us (floors 21, 43, 86 for heads of 64,
// 128, 256): up to 4 rows by one warp of 8 rows 63, 72, 115, of 4 rows 41, 53, 96, by two of 2 rows 36, 52; 5 to 8 rows
// by one warp of 8 64, 73, 124, by two of 4 rows 52, 64, 112, with a group's cost at 3 tiles; as it is now up to 4 rows 35, 53, 94
// (6.2 TB/s at heads of 256), 5 to 8 rows 50, 64, 102.  9 to 16 rows 80, 104, 171; 24 rows, heads of 64, 139; 24 rows, 2 kv heads of 256, up to
// 8192 keys 164 (floor 43).  9 sequences, 2 tokens, up to 5001 keys, 6/3 heads of 64: 15.1 us (floor 5.2).
#include "gdn_attn.cuh"

namespace gdn {
namespace attn {

namespace {

template <int D>
cudaError_t by_rows(const AttnParams& p, bool out_bf16, int sms, cudaStream_t stream) {
    const int R = p.G * p.K;
    if (R <= 4) return launch<Shape<float, D, 1, D == 64 ? 2 : 1, 4, 1, D == 64 ? 2 : 4>>(p, out_bf16, sms, stream);
    if (R <= 8) return launch<Shape<float, D, 1, 2, 4, 1, 4>>(p, out_bf16, sms, stream);
    switch (block_rows(R, false)) {
        case 16: return launch<Shape<float, D, 1, 2, 4, 1>>(p, out_bf16, sms, stream);
        case 32: return launch<Shape<float, D, 1, 4, 2, 1>>(p, out_bf16, sms, stream);
        default: return launch<Shape<float, D, 1, 8, 1, 1>>(p, out_bf16, sms, stream);
    }
}

}  // namespace

cudaError_t launch_f32(const AttnParams& p, int head_dim, bool out_bf16, int sms, cudaStream_t stream) {
    if (head_dim == 64) return by_rows<64>(p, out_bf16, sms, stream);
    if (head_dim == 128) return by_rows<128>(p, out_bf16, sms, stream);
    return by_rows<256>(p, out_bf16, sms, stream);
}

}  // namespace attn

size_t attn_workspace_bytes(int, int K, int Hq, int Hkv, int head_dim, int act_dtype) {
    const size_t parts = 2 * static_cast<size_t>(attn::kMaxCtas);   // two of each CTA
    const size_t rows = attn::block_rows(Hq / Hkv * K, act_dtype == GDN_BF16);
    return attn::kCounterBytes + parts * rows * (head_dim * 4 + 8);
}

cudaError_t launch_attn_decode(const AttnParams& p, int head_dim, int act_dtype, int out_dtype, cudaStream_t stream) {
    const int sms = attn::grid_ctas();
    if (sms == 0) return cudaErrorInvalidDevice;
    const bool out_bf16 = out_dtype == GDN_BF16;
    if (act_dtype != GDN_BF16) return attn::launch_f32(p, head_dim, out_bf16, sms, stream);
    // 64 ragged sequences of up to 8192 keys, 16/2 heads of 256, both with a group's cost at 3 tiles: 24 rows 131 us on
    // mma.sync and 137 on tcgen05, 64 rows 253 and 204, 128 rows 465 and 324; heads of 64: 32 rows 173 and 231, 64 rows
    // 352 and 305.
    // (fp32 results stay on mma.sync: the sums in tensor memory lose bits over a long sequence, see gdn_attn.cuh.)
    return p.G * p.K > 32 && out_bf16 ? attn::launch_tc(p, head_dim, sms, stream) : attn::launch_bf16(p, head_dim, out_bf16, sms, stream);
}

}  // namespace gdn
