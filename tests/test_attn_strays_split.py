"""gdn_attn_decode: infinite and NaN values of drafted tokens on both sides of a border between two CTAs' parts of a group."""
import math

import pytest
import torch

import gated_deltanet_linear_decode_gb300 as gdn
from tests.test_attn_decode import Case
from tests.test_attn_numerics import FORMS

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,out_dtype,Hq,Hkv,K,d", [f for f in FORMS if f[4] > 3])
@pytest.mark.parametrize("peak", [False, True])
def test_rows_get_the_infinities_that_they_see(dtype, out_dtype, Hq, Hkv, K, d, peak):
    """A tile begins inside the last K - 1 tokens of each of B sequences (tiles are of 32 to 128 keys), all of one length, B prime and no
    divisor of the number of SMs: so in some sequence every border between two of its tiles is one between two CTAs, the last one among
    them.  Rows get the infinity that they see, whatever other rows see; with `peak` also where a score of an earlier part leaves
    the others no weight."""
    B, n = 67, 256 + K // 2
    c = Case([n] * B, K, Hq, Hkv, d, 16, dtype, seed=61)
    table = c.table.cuda().long()
    slot = lambda j: (table[:, j // 16], j % 16)
    if peak:   # the first key's score: 40 * 40 / sqrt(d), at least 100
        c.q[:, ::d] = 40.0
        page, at = slot(0)
        c.k[page, at, :, 0] = 40.0
    clean = c.run(out_dtype).clone()
    assert torch.isfinite(clean).all()
    want = torch.zeros(B, K, Hkv, Hq // Hkv, d, device="cuda")
    first = n - K   # the last key that the first token sees
    for j, ch, x in ((255, 5, math.inf), (256, 6, -math.inf), (256, 7, math.nan), (256, 5, math.inf), (n - 1, 8, math.inf)):
        page, at = slot(j)
        c.v[page, at, :, ch] = x
        want[:, j - first:, :, :, ch] += x
    want = want.view(clean.shape)
    hit = want != 0   # (a NaN is)
    inf = hit & ~torch.isnan(want)
    assert inf.any()
    for _ in range(3):
        got = c.run(out_dtype)
        assert torch.all((got == clean) | hit)
        assert torch.all(got[inf].float() == want[inf]) and torch.all(torch.isnan(got[hit & ~inf]))
