"""gdn_norm_residual against the 64-bit definition.  fp32: 1e-5 of the row's largest value (sums of up to 16384
squares, pairwise over a block); a bf16 result may be half a bf16 ulp further off."""
import numpy as np
import pytest
import torch

import gated_deltanet_linear_decode_gb300 as gdn
from tests import attn_ref as R
from tests import gpu_util as G

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def close(got, ref):
    bound = 1e-5 * np.maximum(1.0, np.abs(ref).max(-1, keepdims=True)) + (G.half_ulp_bf16(ref) if got.dtype == BF else 0)
    err = np.abs(R.f64(got) - ref)
    assert (err <= bound).all(), f"worst excess {float((err - bound).max()):.3e}"


def run(T, H, dtype, res, y=True, gate=0, post=True, chan=False, pre=True, store=True, in_place=False, pitch=0, seed=0,
        alpha=0.75):
    g = torch.Generator().manual_seed(seed)
    ht = (3 * torch.randn(T, H, generator=g)).to(res).cuda()
    wide = torch.randn(T, H + pitch, generator=g).to(dtype).cuda()
    yt = wide[:, pitch:] if pitch % 8 == 0 else wide[:, :H]
    gt = torch.randn(T, gate + (pitch if gate else 0), generator=g).to(dtype).cuda()[:, :gate] if gate else None
    w = [(1 + 0.1 * torch.randn(H, generator=g)).cuda() for _ in range(3)]
    pw, cs, nw = (w[0] if post and y else None), (w[1] if chan and y else None), (w[2] if pre else None)
    hr, xr = R.norm_residual(R.f64(ht), R.f64(yt) if y else None, None if gt is None else R.f64(gt),
                             None if pw is None else R.f64(pw), None if cs is None else R.f64(cs),
                             None if nw is None else R.f64(nw), alpha=alpha)
    d = gdn.make_norm_dims(H, dtype, res, alpha=alpha)
    ho = ht if in_place else torch.full((T, H), 7.0, dtype=res, device="cuda") if store else None
    x = torch.full((T, H), 7.0, dtype=dtype, device="cuda") if pre else None
    gdn.gdn_norm_residual(d, ht, ho, y=yt if y else None, gate=gt, post_w=pw, chan_scale=cs, pre_w=nw, x=x)
    if ho is not None:
        close(ho, hr)
    if pre:
        close(x, xr)


@pytest.mark.parametrize("dtype,res", [(BF, BF), (BF, F32), (F32, F32)])
@pytest.mark.parametrize("T,H", [(1, 1), (3, 7), (64, 2048), (5, 5120), (17, 1000), (300, 64), (2, 16384), (9, 2047),
                                 (1000, 8), (4, 8200)])
def test_sizes(T, H, dtype, res):
    run(T, H, dtype, res, gate=[0, 1, H][T % 3], chan=T % 2 == 0, seed=T * 7 + H)


@pytest.mark.parametrize("dtype,res", [(BF, BF), (BF, F32), (F32, F32)])
@pytest.mark.parametrize("T,H", [(608, 1024), (609, 1024), (2100, 264), (311, 4096), (400, 4104), (700, 1992), (305, 8192)])
def test_many_rows(T, H, dtype, res):
    """Either side of one and two chunks a thread, rows enough for a look-ahead, widths that leave threads without a chunk."""
    run(T, H, dtype, res, gate=[0, 1, H][T % 3], chan=T % 2 == 0, pitch=8 * (T % 2), seed=T + H)


@pytest.mark.parametrize("H", [256, 255])
@pytest.mark.parametrize("kw", [
    dict(y=False), dict(y=False, store=False), dict(post=False), dict(pre=False), dict(store=False),
    dict(in_place=True), dict(in_place=True, gate=1, chan=True), dict(post=False, gate=-1), dict(gate=-1, pitch=8),
    dict(gate=1, pitch=3), dict(pitch=16), dict(gate=-1, pitch=5, pre=False), dict(alpha=0.0)])
def test_forms(H, kw):
    kw = dict(kw)
    if kw.get("gate") == -1:
        kw["gate"] = H
    run(33, H, BF, BF, seed=5, **kw)
    run(33, H, BF, F32, seed=6, **kw)


def test_extremes():
    """Rows of zeros, and gates at plus and minus infinity (fully open and shut)."""
    T, H = 4, 512
    d = gdn.make_norm_dims(H, F32, F32)
    y, h = torch.zeros(T, H, device="cuda"), torch.zeros(T, H, device="cuda")
    y[1:] = torch.randn(T - 1, H, device="cuda")
    gate = torch.tensor([[0.0], [float("inf")], [float("-inf")], [-200.0]], device="cuda")
    w = torch.ones(H, device="cuda")
    ho, x = torch.empty_like(h), torch.empty_like(h)
    gdn.gdn_norm_residual(d, h, ho, y=y, gate=gate, pre_w=w, x=x)
    assert (ho[0] == 0).all() and (x[0] == 0).all() and torch.equal(ho[1], y[1]) and (ho[2:].abs() < 1e-30).all()
    assert torch.isfinite(x).all()
