"""The sigmoid gate where it is a result's only rounding: h' = 0 + 1 * sigmoid(gate).  Its error stays within 2^-21 of it whatever
the gate's size (2^-22 and 2^-23 of an approximate power and reciprocal, 2^-24 of a sum), and extremes are what they are."""
import numpy as np
import pytest
import torch

import gated_deltanet_linear_decode_gb300 as gdn

pytestmark = pytest.mark.gpu
F32, BF = torch.float32, torch.bfloat16


@pytest.mark.parametrize("H", [512, 509])     # 16 bytes at a time, and one element
@pytest.mark.parametrize("dtype", [F32, BF])
def test_norms(H, dtype):
    T = 400
    g = torch.linspace(-85, 85, T * H, dtype=torch.float64).view(T, H).to(dtype).cuda()
    one, zero, out = torch.ones(T, H, dtype=dtype, device="cuda"), torch.zeros(T, H, device="cuda"), torch.empty(T, H, device="cuda")
    gdn.gdn_norm_residual(gdn.make_norm_dims(H, dtype, F32), zero, out, y=one, gate=g)
    want = torch.sigmoid(g.double())
    assert float(((out.double() - want).abs() / want).max()) <= 2.0 ** -21


@pytest.mark.parametrize("dtype", [F32, BF])
def test_attention(dtype):
    """One key, values of one: out = sigmoid(gate)."""
    B, Hq, d = 64, 8, 128
    k, v = torch.zeros(1, 4, 1, d, dtype=dtype, device="cuda"), torch.ones(1, 4, 1, d, dtype=dtype, device="cuda")
    g = torch.linspace(-85, 85, B * Hq * d, dtype=torch.float64).view(B, Hq * d).to(dtype).cuda()
    dims = gdn.make_attn_dims(Hq, 1, d, dtype, F32)
    ws = torch.zeros(gdn.gdn_attn_decode_workspace_bytes(dims, B, 1), dtype=torch.uint8, device="cuda")
    out = torch.empty(B, Hq * d, device="cuda")
    gdn.gdn_attn_decode(dims, gdn.KvCache(k, v), 1, torch.zeros_like(g), torch.zeros(B, 1, dtype=torch.int32, device="cuda"),
                        torch.ones(B, dtype=torch.int32, device="cuda"), out, gate=g, workspace=ws)
    want = torch.sigmoid(g.double())
    assert float(((out.double() - want).abs() / want).max()) <= 2.0 ** -21


@pytest.mark.parametrize("dtype", [F32, BF])
def test_extreme_gates(dtype):
    x = torch.tensor([[float("inf"), float("-inf"), float("nan"), 3e38, -3e38, 0.0, -0.0, 100.0, -100.0, -1000.0, 1e-30, 88.0]], device="cuda").to(dtype)
    one, zero, out = torch.ones_like(x), torch.zeros(1, 12, device="cuda"), torch.empty(1, 12, device="cuda")
    gdn.gdn_norm_residual(gdn.make_norm_dims(12, dtype, F32), zero, out, y=one, gate=x)
    got = out[0].tolist()
    assert got[0] == 1 and got[1] == 0 and np.isnan(got[2]) and got[3] == 1 and got[4] == 0
    assert got[5] == got[6] == 0.5 and got[7] == 1 and 0 <= got[8] <= 1e-38 and got[9] == 0 and got[10] == 0.5 and got[11] == 1
