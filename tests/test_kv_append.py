"""gdn_kv_append against the 64-bit definition.  fp32: 1e-5 relative to the row's largest value (a norm over
<= 256 squares, two products and a sum); bf16: half a bf16 ulp more.  v is a copy, and everything that no token
names keeps its bits."""
import numpy as np
import pytest
import torch

import gated_deltanet_linear_decode_gb300 as gdn
from tests import attn_ref as R
from tests import gpu_util as G

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def close(got, ref, dtype):
    got = R.f64(got)
    bound = 1e-5 * max(1.0, np.abs(ref).max()) + (G.half_ulp_bf16(ref) if dtype == BF else 0)
    err = np.abs(got - ref)
    assert (err <= bound).all(), f"worst excess {float((err - bound).max()):.3e}"


def run(T, Hq, Hkv, d, rope, ps, dtype, layout="thd", norm=True, seed=0, slots=None, pos=None, pitched=True):
    g = torch.Generator().manual_seed(seed)
    pages = -(-T // ps) + 3
    shape = (pages, ps, Hkv, d) if layout == "thd" else (pages, Hkv, ps, d)
    k, v = torch.randn(2, *shape, generator=g).to(dtype).cuda()
    if layout != "thd":
        k, v = k.transpose(1, 2), v.transpose(1, 2)
    nq, nk = Hq * d, Hkv * d
    qkv = torch.randn(T, nq + 2 * nk, generator=g).to(dtype).cuda()
    q, xk, xv = qkv[:, :nq], qkv[:, nq:nq + nk], qkv[:, nq + nk:]
    if not pitched:
        q, xk, xv = q.contiguous(), xk.contiguous(), xv.contiguous()
    n_pos = 700
    slots = torch.randperm(pages * ps, generator=g)[:T].to(torch.int32) if slots is None else slots
    pos = torch.randint(0, n_pos, (T,), generator=g).to(torch.int32) if pos is None else pos
    wq, wk = 1 + 0.1 * torch.randn(2, d, generator=g)
    ang = torch.arange(n_pos)[:, None].double() * 1e4 ** (-torch.arange(rope // 2).double() * 2 / max(rope, 1))
    cos, sin = ang.cos().float(), ang.sin().float()
    dims = gdn.make_attn_dims(Hq, Hkv, d, dtype, dtype, rope_dim=rope)
    out = torch.full((T, nq), 7.0, dtype=dtype, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    k0, v0 = k.clone(), v.clone()
    gdn.gdn_kv_append(dims, gdn.KvCache(k, v), q, xk, xv, pos.cuda(), slots.cuda(), out,
                      q_norm_w=wq.cuda() if norm else None, k_norm_w=wk.cuda() if norm else None,
                      rope_cos=cos.cuda() if rope else None, rope_sin=sin.cuda() if rope else None, dev_status=st)
    cap = pages * ps
    good = (slots < cap) & (((pos >= 0) & (pos < n_pos)) if rope else torch.ones(T, dtype=torch.bool))
    sel = good.numpy()
    kept = (good & (slots >= 0)).numpy()
    p = pos.clamp(0, n_pos - 1).long().numpy()
    co, si = (R.f64(cos)[p], R.f64(sin)[p]) if rope else (None, None)
    qr = R.heads(R.f64(q), d, R.f64(wq) if norm else None, co, si).reshape(T, -1)
    kr = R.heads(R.f64(xk), d, R.f64(wk) if norm else None, co, si)
    close(out[torch.from_numpy(sel).cuda()], qr[sel], dtype)
    assert (out[torch.from_numpy(~sel).cuda()] == 7.0).all()
    where = torch.zeros(cap, dtype=torch.bool)
    where[slots[torch.from_numpy(kept)].long()] = True
    m = where.view(pages, ps).cuda()
    assert torch.equal(k[~m], k0[~m]) and torch.equal(v[~m], v0[~m])
    s = slots[torch.from_numpy(kept)].long()
    close(k[(s // ps).cuda(), (s % ps).cuda()], kr[kept], dtype)
    assert torch.equal(v[(s // ps).cuda(), (s % ps).cuda()], xv.reshape(T, Hkv, d)[torch.from_numpy(kept).cuda()])
    assert int(st) == (0 if sel.all() else 64)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,Hq,Hkv,d,rope,ps,layout,norm", [
    (1, 16, 2, 256, 64, 16, "thd", True), (64, 16, 2, 256, 64, 16, "htd", True), (37, 5, 5, 64, 64, 7, "thd", True),
    (300, 3, 1, 128, 0, 1, "thd", True), (50, 6, 3, 128, 128, 20, "htd", False), (9, 1, 1, 64, 16, 64, "thd", True),
    (1000, 8, 4, 256, 256, 16, "thd", True), (257, 12, 2, 64, 32, 16, "htd", False)])
def test_against_the_definition(T, Hq, Hkv, d, rope, ps, layout, norm, dtype):
    run(T, Hq, Hkv, d, rope, ps, dtype, layout, norm, seed=T, pitched=T % 2 == 1)


@pytest.mark.parametrize("rope", [0, 32])
def test_padding_and_bad_indices(rope):
    """Padding (slot -1) is not stored; a slot past the cache or a position past the table skips the token."""
    T = 40
    slots = torch.arange(T, dtype=torch.int32)
    slots[[3, 39]] = -1
    slots[7], slots[8] = 16 * 6, 2 ** 31 - 1
    pos = torch.arange(T, dtype=torch.int32)
    pos[11], pos[12] = 700, -1
    run(T, 4, 2, 64, rope, 16, BF, seed=2, slots=slots, pos=pos)


def test_zero_row():
    """A head of zeros stays zero (eps keeps the norm finite)."""
    d = gdn.make_attn_dims(1, 1, 64, F32, F32)
    k, v = torch.ones(2, 1, 4, 1, 64, device="cuda")
    z, w = torch.zeros(1, 64, device="cuda"), torch.ones(64, device="cuda")
    out = torch.ones(1, 64, device="cuda")
    i = torch.zeros(1, dtype=torch.int32, device="cuda")
    gdn.gdn_kv_append(d, gdn.KvCache(k, v), z, z, z, i, i, out, q_norm_w=w, k_norm_w=w)
    assert (out == 0).all() and (k[0, 0] == 0).all() and (v[0, 0] == 0).all() and (k[0, 1:] == 1).all()
