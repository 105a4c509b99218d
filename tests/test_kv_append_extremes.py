"""gdn_kv_append without a norm: an infinite channel that is not rotated is stored as it is, and does not reach the others."""
import pytest
import torch

import gated_deltanet_linear_decode_gb300 as gdn

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d,rope", [(64, 32), (128, 16), (256, 64)])
def test_infinite_channels_beside_the_rotated_ones(d, rope, dtype):
    g = torch.Generator().manual_seed(d)
    T, Hq, Hkv, ps = 5, 4, 2, 4
    q, k = (torch.randn(T, h * d, generator=g).to(dtype).cuda() for h in (Hq, Hkv))
    cos, sin = torch.randn(2, 8, rope // 2, generator=g).cuda()
    kc, vc = torch.zeros(2, 2, ps, Hkv, d, dtype=dtype, device="cuda")
    i = torch.arange(T, dtype=torch.int32, device="cuda")
    outs = []
    for x in (0.0, float("inf"), float("-inf")):
        for t in (q, k):
            t.view(T, -1, d)[:, 1, rope] = x
            t.view(T, -1, d)[2, 0, d - 1] = x
        out = torch.empty_like(q)
        gdn.gdn_kv_append(gdn.make_attn_dims(Hq, Hkv, d, dtype, dtype, rope_dim=rope), gdn.KvCache(kc, vc), q, k, k, i, i, out,
                          rope_cos=cos, rope_sin=sin)
        outs.append((x, out.clone().view(T, Hq, d), kc.view(-1, Hkv, d)[:T].clone()))
    for x, qo, ko in outs:
        for got, base in ((qo, outs[0][1]), (ko, outs[0][2])):
            want = base.clone()
            want[:, 1, rope] = x
            want[2, 0, d - 1] = x
            assert torch.equal(got, want)
