"""Where gdn_attn_decode could lose bits, or let one row's numbers into another's."""
import numpy as np
import pytest
import torch

import gated_deltanet_linear_decode_gb300 as gdn
from tests import attn_ref as R
from tests.test_attn_decode import BF, F32, Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 128, 256])
def test_bf16_results_of_long_sums_are_the_nearest_ones(d):
    """Up to 8 rows a kv head: sums of 16,000 values of one sign walked by one SM (more sequences than SMs, all on the same pages).
    A relative error e of the sum moves it past a rounding boundary of bf16 in at most e / 2^-8 of the results.  e = 4e-6 (five times
    2^-21, the weights' products and the exponents' rounding) leaves one in a thousand; a sum that rounds one way every 16 keys drifts
    by up to 2^-24 a step, 1.5e-5 over the 250 steps of a warp."""
    n, ps, Hq, B = 16000, 16, 8, 160
    c = Case([n], 1, Hq, 1, d, ps, BF, seed=18, gate=False)
    c.v.abs_()
    g = torch.Generator().manual_seed(19)
    q = torch.randn(B, Hq * d, generator=g).to(BF).cuda()
    dims = gdn.make_attn_dims(Hq, 1, d, BF, BF)
    ws = torch.zeros(gdn.gdn_attn_decode_workspace_bytes(dims, B, 1), dtype=torch.uint8, device="cuda")
    out = torch.empty(B, Hq * d, dtype=BF, device="cuda")
    gdn.gdn_attn_decode(dims, gdn.KvCache(c.k, c.v), 1, q, c.table.repeat(B, 1).cuda(), torch.full((B,), n, dtype=torch.int32, device="cuda"),
                        out, workspace=ws)
    rows = c.table[0].long().cuda()
    k, v = (x[rows].reshape(-1, d)[:n].double() for x in (c.k, c.v))
    s = q.double().view(-1, d) @ k.T / np.sqrt(d)
    ref = (torch.softmax(s, -1) @ v).view(B, -1)
    assert float((out != ref.to(BF)).double().mean()) <= 1e-3
