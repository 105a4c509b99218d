"""Calls of one row: its pitch is of no account, whatever tensor it is a slice of."""
import pytest
import torch

import gated_deltanet_linear_decode_gb300 as gdn

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def slice_of(n, extra):
    """[1][n] of a tensor whose rows are n + extra apart."""
    return torch.randn(3, n + extra, device="cuda").to(BF)[:1, :n]


@pytest.mark.parametrize("extra", [0, 1, 3, 8])
def test_one_row_of_any_pitch(extra):
    d = gdn.make_attn_dims(2, 1, 64, BF, BF)
    k, v = (torch.randn(1, 4, 1, 64, device="cuda").to(BF) for _ in range(2))
    cache, i = gdn.KvCache(k, v), torch.zeros(1, dtype=torch.int32, device="cuda")
    q, nk, gate = slice_of(128, extra), slice_of(64, extra), slice_of(128, extra)
    out = torch.empty(1, 128, dtype=BF, device="cuda")
    gdn.gdn_kv_append(d, cache, q, nk, nk, i, i, out)
    assert torch.equal(out, q) and torch.equal(k[0, 0], nk)
    ws = torch.zeros(gdn.gdn_attn_decode_workspace_bytes(d, 1, 1), dtype=torch.uint8, device="cuda")
    gdn.gdn_attn_decode(d, cache, 1, q, i.view(1, 1), i + 1, out, gate=gate, workspace=ws)
    want = torch.empty_like(out)
    gdn.gdn_attn_decode(d, cache, 1, q.contiguous(), i.view(1, 1), i + 1, want, gate=gate.contiguous(), workspace=ws)
    assert torch.equal(out, want)
    n = gdn.make_norm_dims(128, BF, BF)
    h, x = torch.zeros(1, 128, dtype=BF, device="cuda"), torch.empty(1, 128, dtype=BF, device="cuda")
    gdn.gdn_norm_residual(n, h, x, y=q, gate=gate)
    gdn.gdn_norm_residual(n, h, want, y=q.contiguous(), gate=gate.contiguous())
    assert torch.equal(x, want)
