"""Where gdn_attn_decode could lose bits, or let one row's numbers into another's."""
import numpy as np
import pytest
import torch

import gated_deltanet_linear_decode_gb300 as gdn
from tests import attn_ref as R
from tests import gpu_util as G
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


FORMS = [  # dtype, result, Hq, Hkv, K, d: every kernel form that holds more than one token
    (BF, BF, 4, 2, 2, 256), (BF, BF, 2, 2, 7, 64), (BF, BF, 10, 2, 3, 128), (BF, BF, 16, 2, 3, 256), (BF, BF, 16, 2, 4, 128),
    (BF, BF, 16, 2, 8, 256), (BF, BF, 16, 2, 16, 64), (BF, BF, 16, 1, 16, 128), (BF, BF, 8, 2, 16, 128), (BF, BF, 16, 2, 16, 256),
    (BF, F32, 16, 2, 3, 256), (BF, F32, 16, 2, 4, 64), (BF, F32, 16, 2, 8, 128), (BF, F32, 16, 2, 16, 256),
    (F32, F32, 2, 2, 2, 64), (F32, F32, 2, 2, 3, 128), (F32, F32, 4, 2, 3, 256), (F32, BF, 8, 2, 4, 64), (F32, F32, 8, 2, 8, 128),
    (F32, F32, 4, 2, 16, 256), (F32, F32, 16, 2, 16, 64)]


@pytest.mark.parametrize("dtype,out_dtype,Hq,Hkv,K,d", FORMS)
@pytest.mark.parametrize("lens", [[130, 2, 65, 1, 0, 33, 17, 300], [5000, 16], [129] * 170], ids=["short", "split", "many"])
def test_rows_are_kept_from_later_tokens_that_are_not_finite(dtype, out_dtype, Hq, Hkv, K, d, lens):
    """Infinities and NaN in the drafted tokens' keys and values reach the rows that see them, in those channels, and no other.  Where
    nothing infinite is seen the bounds are those of test_attn_decode."""
    c = Case(lens, K, Hq, Hkv, d, 13, dtype, seed=31)
    at = lambda t, b, j, h: t[int(c.table[b, j // 13]), j % 13, h]
    bad = np.zeros((len(lens), K, Hkv, d), dtype=bool)   # by the first drafted token ...
    for b, n in enumerate(lens):
        plants = [(n - 1, 0, 3, float("inf")), (n - 1, 0, 8, float("nan")), (n - 1, Hkv - 1, slice(d - 5, d), float("nan"))]
        if K > 2:
            plants += [(n - K + 1, 0, d - 1, float("-inf")), (n - 2, 0, 17, float("inf"))]
        for j, h, ch, x in plants:
            if j < 0 or j <= n - K:      # (a key that every row sees)
                continue
            at(c.v, b, j, h)[ch] = x
            bad[b, j - n + K:, h, ch] = True   # ... token p sees keys up to n - K + p
        if n > 2 and b % 2 and K > 1:
            at(c.k, b, n - 1, 0)[5] = float("nan")
            bad[b, K - 1, 0] = True
    v = R.f64(c.v)
    fin = lambda x: np.nan_to_num(x, nan=0.0, posinf=0.0, neginf=0.0)
    gate = None if c.gate is None else R.f64(c.gate)
    ref = R.attn(R.f64(c.q), fin(R.f64(c.k)), fin(v), c.table.numpy(), lens, K, Hq, Hkv, d, gate)
    got = R.f64(c.run(out_dtype))
    bad = np.repeat(bad.reshape(len(lens) * K, Hkv, 1, d), Hq // Hkv, 2).reshape(got.shape)
    assert (np.isfinite(got) == ~bad).all(), (np.argwhere(np.isfinite(got) == bad)[:4], int((np.isfinite(got) == bad).sum()))
    big = float(np.abs(fin(v)).max())
    bound = 1e-5 * big if out_dtype == F32 else G.half_ulp_bf16(ref) + 2.0 ** -16 * big
    assert (np.abs(got - ref) <= bound)[~bad].all()


def test_infinite_values_that_a_row_sees():
    """One infinite value among the drafted tokens', the rows that see it get that infinity, whatever the gate."""
    c = Case([50], 4, 4, 2, 64, 16, F32, seed=32)
    c.v[int(c.table[0, 48 // 16]), 48 % 16, 1, 9] = float("-inf")
    out = R.f64(c.run(F32)).reshape(4, 4, 64)
    assert np.isfinite(out[:2]).all() and (out[2:, 2:, 9] == -np.inf).all()
    assert np.isfinite(out[2:, :2]).all() and np.isfinite(np.delete(out[2:, 2:], 9, -1)).all()


def rising(lens, K, Hq, d, dtype, per_tile, seed):
    """Scores that rise by `per_tile` (base 2) every 128 keys in a third of the rows, half as much in another, fall in the last."""
    c = Case(lens, K, Hq, 1, d, 16, dtype, seed=seed, gate=False)
    g = torch.Generator().manual_seed(seed + 1)
    T, step = len(lens) * K, per_tile / 128 / 1.4427 * d ** 0.5
    q = torch.randn(T, Hq, d, generator=g)
    sign = torch.tensor([1.0, 0.5, -1.0])[torch.randint(0, 3, (T, Hq), generator=g)]
    q[..., 0] = 4 * sign
    c.q = q.view(T, Hq * d).to(dtype).cuda()
    for b, n in enumerate(lens):
        j = torch.arange(n, device="cuda")
        page = c.table[b].long().cuda()[j // 16]
        c.k[page, j % 16, 0, 0] = (step / 4 * j).to(dtype)
    return c


@pytest.mark.parametrize("dtype,out_dtype,Hq,K,d", [
    (BF, BF, 16, 4, 64), (BF, BF, 16, 4, 128), (BF, BF, 16, 4, 256), (BF, BF, 8, 9, 128), (BF, BF, 8, 16, 64), (BF, BF, 8, 16, 128),
    (BF, BF, 8, 16, 256), (BF, BF, 16, 16, 128), (BF, BF, 8, 1, 128), (BF, F32, 16, 8, 256), (F32, F32, 4, 2, 64)])
@pytest.mark.parametrize("per_tile", [3, 12, 40])
@pytest.mark.parametrize("lens", [[9000], [700, 130, 0, 1500, 129], [1000] * 160], ids=["split", "few", "whole"])
def test_scores_that_rise_along_the_sequence(dtype, out_dtype, Hq, K, d, per_tile, lens):
    """The running maximum changes in most tiles, in some lanes by far and in others not at all.  An error of 2^-20 of a score moves a
    weight by as much (see test_attn_decode.test_large_scores); scores reach per_tile * 70 / 1.44."""
    c = rising(lens, K, Hq, d, dtype, per_tile, seed=40)
    first = [0, len(lens) // 2, len(lens) - 1] if len(lens) > 10 else range(len(lens))
    k, v = np.nan_to_num(R.f64(c.k)), np.nan_to_num(R.f64(c.v))
    got = R.f64(c.run(out_dtype)).reshape(len(lens), K, -1)
    big, s = float(np.abs(v).max()), per_tile * (max(lens) / 128) / 1.44 + 20
    for b in first:
        ref = R.attn(R.f64(c.q).reshape(len(lens), K, -1)[b], k, v, c.table.numpy()[b:b + 1], [lens[b]], K, Hq, 1, d).reshape(K, -1)
        bound = 2 * s * 2.0 ** -20 * big + (G.half_ulp_bf16(ref) + 2.0 ** -16 * big if out_dtype == BF else 1e-5 * big)
        err = np.abs(got[b] - ref)
        assert np.isfinite(got[b]).all() and (err <= bound).all(), float((err - bound).max())
