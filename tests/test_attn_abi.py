"""include/gdn_attn.h and include/gdn_norm.h: plain C, every declared symbol exported, and bad arguments refused
before anything reaches a device (CPU only: no call here launches a kernel)."""
import ctypes
import os
import re
import subprocess

import pytest
import torch

import gated_deltanet_linear_decode_gb300 as gdn

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
INCLUDE = os.path.join(ROOT, "include")
OK, INVALID, UNSUPPORTED, ALIGNMENT, WORKSPACE = 0, 1, 2, 3, 5
A = lambda i: 0x100000000 * (i + 1)   # far apart, aligned, never dereferenced on these paths


def test_declared_symbols_are_exported_and_bound():
    src = "".join(open(os.path.join(INCLUDE, f)).read() for f in ("gdn_attn.h", "gdn_norm.h"))
    names = set(re.findall(r"\b(gdn_[a-z0-9_]+)\s*\(", re.sub(r"/\*.*?\*/", "", src, flags=re.S)))
    assert names == set(gdn.EXPORTED_SYMBOLS_ATTN)
    out = subprocess.run(["nm", "-D", "--defined-only", gdn._build.build()], capture_output=True, text=True, check=True).stdout
    assert names <= {line.split()[-1] for line in out.splitlines() if line.strip()}
    assert all(hasattr(gdn, n) for n in names)


def test_headers_compile_as_c_and_match_the_bindings():
    checks = [("gdn_attn_dims", gdn.GdnAttnDims), ("gdn_kv_cache", gdn.GdnKvCache), ("gdn_norm_dims", gdn.GdnNormDims)]
    src = '#include "gdn_attn.h"\n#include "gdn_norm.h"\n' + "".join(
        f"_Static_assert(sizeof({c}) == {ctypes.sizeof(p)}, \"size\");\n" for c, p in checks)
    src += f"_Static_assert(GDN_KV_REFUSED == {gdn.GDN_KV_REFUSED} && GDN_KV_BAD_INDEX == {gdn.GDN_KV_BAD_INDEX}, \"bits\");\n"
    src += "int main(void){ return (int)GDN_OK; }\n"
    r = subprocess.run(["gcc", "-std=c11", "-Wall", "-Werror", "-fsyntax-only", "-I", INCLUDE, "-x", "c", "-"], input=src,
                       text=True, capture_output=True)
    assert r.returncode == 0, r.stderr


def adims(Hq=16, Hkv=2, d=256, rope=0, scale=0.0625, eps=1e-6, act=1, out=1, flags=0):
    return gdn.GdnAttnDims(Hq, Hkv, d, rope, scale, eps, act, out, flags)


def cache(k=A(0), v=A(1), pages=100, ps=16, s=None, dims=None):
    d = dims or adims()
    s = s or (ps * d.H_kv * d.head_dim, d.H_kv * d.head_dim, d.head_dim)
    return gdn.GdnKvCache(k, v, pages, ps, *s)


def attn(dims=None, kc=None, B=4, K=1, P=10, q=A(2), ldq=4096, gate=A(3), ldg=4096, table=A(4), lens=A(5), out=A(6),
         ws=A(7), n=1 << 31, st=None):
    dims = adims() if dims is None else dims
    kc = cache(dims=dims) if kc is None else kc
    lib = gdn.library()
    gdn.gdn_attn_decode_workspace_bytes(adims(), 1, 1)   # sets the signatures
    return lib.gdn_attn_decode(ctypes.byref(dims) if dims else None, ctypes.byref(kc) if kc else None, B, K, P, q, ldq, gate,
                               ldg, table, lens, out, ws, n, st, None)


BAD_DIMS = [
    (dict(Hq=0), INVALID), (dict(Hkv=0), INVALID), (dict(Hq=5, Hkv=2), INVALID), (dict(act=2), INVALID),
    (dict(out=-1), INVALID), (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID), (dict(eps=0.0), INVALID),
    (dict(rope=-16), INVALID), (dict(rope=272), INVALID), (dict(d=96), UNSUPPORTED), (dict(d=512), UNSUPPORTED),
    (dict(Hq=34, Hkv=2), UNSUPPORTED), (dict(rope=24), UNSUPPORTED), (dict(flags=1), INVALID), (dict(flags=8), INVALID)]


@pytest.mark.parametrize("kw,status", BAD_DIMS)
def test_attention_dims(kw, status):
    d = adims(**kw)
    assert attn(dims=d, kc=cache()) == status
    assert gdn.gdn_attn_decode_workspace_bytes(d, 4, 1) == 0


def test_attention_arguments():
    assert attn(B=0) == OK
    assert attn(B=-1) == INVALID and attn(K=0) == INVALID and attn(K=17) == INVALID and attn(P=0) == INVALID
    for name in ("q", "table", "lens", "out"):
        assert attn(**{name: None}) == INVALID
        assert attn(**{name: A(20) + 8}) == ALIGNMENT
    assert attn(gate=A(20) + 2) == ALIGNMENT and attn(st=A(20) + 4) == ALIGNMENT and attn(ws=A(20) + 8) == ALIGNMENT
    assert attn(ldq=4095) == INVALID and attn(ldq=4100) == ALIGNMENT and attn(ldg=1) == INVALID
    assert attn(ldq=1 << 41) == INVALID
    assert attn(out=A(2)) == INVALID and attn(out=A(0) + 4096) == INVALID and attn(out=A(5)) == INVALID
    assert attn(ws=A(6), out=A(6)) == INVALID and attn(st=A(5)) == INVALID
    assert attn(B=1 << 30, K=16) == INVALID          # rows past 31 bits


def test_cache_description():
    d = adims()
    assert attn(kc=cache(k=None)) == INVALID and attn(kc=cache(v=A(0))) == INVALID and attn(kc=cache(k=A(0) + 8)) == ALIGNMENT
    assert attn(kc=cache(pages=0)) == INVALID and attn(kc=cache(ps=0)) == INVALID
    assert attn(kc=cache(pages=1 << 27, ps=16)) == INVALID           # slots past 31 bits
    for s in [(8192, 512, 255), (8192, 511, 256), (8191, 512, 256), (8192, 512, 0), (0, 512, 256), (8192, 256, 256),
              (-8192, 512, 256), (4096, 512, 256), (8192, 512, 512)]:
        assert attn(kc=cache(s=s)) in (INVALID, ALIGNMENT), s
    assert attn(kc=cache(s=(8192, 512, 260))) == ALIGNMENT


def test_workspace():
    n = gdn.gdn_attn_decode_workspace_bytes(adims(), 4, 1)
    assert gdn.gdn_attn_decode_workspace_bytes(adims(), 0, 1) == 0 and gdn.gdn_attn_decode_workspace_bytes(adims(), 1, 17) == 0
    if n:
        assert attn(n=n - 1) == WORKSPACE and attn(ws=None, n=0) == WORKSPACE


def extend(ps=16, pages=100, B=4, P=10, T=8, **kw):
    a = dict(new=A(0), lens=A(1), held=A(2), table=A(3), free=A(4), fc=A(5), lens_o=A(1), held_o=A(2), fc_o=A(5), slots=A(6),
             pos=A(7), cu=A(8), st=None)
    a.update(kw)
    gdn.gdn_attn_decode_workspace_bytes(adims(), 1, 1)
    return gdn.library().gdn_kv_extend(ps, pages, B, P, T, *a.values(), None)


def truncate(ps=16, pages=100, B=4, P=10, **kw):
    a = dict(keep=A(0), lens=A(1), held=A(2), table=A(3), free=A(4), fc=A(5), lens_o=A(1), held_o=A(2), fc_o=A(5), st=None)
    a.update(kw)
    gdn.gdn_attn_decode_workspace_bytes(adims(), 1, 1)
    return gdn.library().gdn_kv_truncate(ps, pages, B, P, *a.values(), None)


@pytest.mark.parametrize("f", [extend, truncate])
def test_page_bookkeeping_arguments(f):
    assert f(ps=0) == INVALID and f(pages=0) == INVALID and f(B=-1) == INVALID and f(P=0) == INVALID
    assert f(pages=1 << 28) == INVALID and f(B=16385) == UNSUPPORTED
    for name in ("lens", "held", "table", "free", "fc", "lens_o", "held_o", "fc_o"):
        assert f(**{name: None}) == INVALID
        assert f(**{name: A(20) + 4}) == ALIGNMENT
    assert f(st=A(20) + 4) == ALIGNMENT
    assert f(lens_o=A(2)) == INVALID and f(st=A(1)) == INVALID and f(B=64, lens_o=A(1) + 16) == INVALID
    assert f(free=A(3)) == INVALID


def test_extend_arguments():
    assert extend(T=-1) == INVALID and extend(new=None) == INVALID and extend(cu=None) == INVALID
    assert extend(slots=None) == INVALID and extend(pos=A(6)) == INVALID and extend(slots=A(0)) == INVALID
    assert extend(cu=A(3)) == INVALID


def append(dims=None, kc=None, T=4, q=A(2), ldq=4096, k=A(3), ldk=512, v=A(4), ldv=512, pos=A(5), slots=A(6), wq=A(7), wk=A(8),
           cos=A(9), sin=A(10), n_pos=100, out=A(11), st=None):
    dims = adims(rope=64) if dims is None else dims
    gdn.gdn_attn_decode_workspace_bytes(adims(), 1, 1)
    return gdn.library().gdn_kv_append(ctypes.byref(dims), ctypes.byref(kc or cache(dims=adims())), T, q, ldq, k, ldk, v, ldv, pos,
                                       slots, wq, wk, cos, sin, n_pos, out, st, None)


@pytest.mark.parametrize("kw,status", BAD_DIMS)
def test_append_dims(kw, status):
    assert append(dims=adims(**kw)) == status


def test_append_arguments():
    assert append(T=0) == OK and append(T=-1) == INVALID
    for name in ("q", "k", "v", "pos", "slots", "out"):
        assert append(**{name: None}) == INVALID
        assert append(**{name: A(20) + 8}) == ALIGNMENT
    for name in ("wq", "wk", "cos", "sin", "st"):
        assert append(**{name: A(20) + 8}) == ALIGNMENT
    assert append(cos=None) == INVALID and append(sin=None) == INVALID and append(n_pos=0) == INVALID
    assert append(ldq=4000) == INVALID and append(ldk=511) == INVALID and append(ldv=516) == ALIGNMENT
    assert append(out=A(2)) == INVALID and append(k=A(0)) == INVALID and append(v=A(1)) == INVALID and append(st=A(5)) == INVALID
    assert append(out=A(0)) == INVALID and append(kc=cache(ps=0)) == INVALID


def norm(H=2048, eps=1e-6, alpha=1.0, act=1, res=1, T=4, y=A(0), ldy=2048, gate=A(1), ldg=2048, cols=2048, h=A(2), post=A(3),
         chan=A(4), pre=A(5), ho=A(6), x=A(7), dims=True):
    d = gdn.GdnNormDims(H, eps, alpha, act, res)
    gdn.gdn_attn_decode_workspace_bytes(adims(), 1, 1)
    return gdn.library().gdn_norm_residual(ctypes.byref(d) if dims else None, T, y, ldy, gate, ldg, cols, h, post, chan, pre, ho, x, None)


def test_norm_arguments():
    assert norm(T=0) == OK and norm(T=-1) == INVALID and norm(dims=False) == INVALID
    assert norm(H=0) == INVALID and norm(eps=0.0) == INVALID and norm(alpha=float("inf")) == INVALID
    assert norm(act=3) == INVALID and norm(res=2) == INVALID and norm(act=0, res=1) == UNSUPPORTED
    assert norm(H=16385, ldy=16385, cols=1) == UNSUPPORTED
    assert norm(cols=2) == INVALID and norm(cols=0) == INVALID and norm(gate=None) == INVALID and norm(y=None) == INVALID
    assert norm(h=None) == INVALID and norm(ho=None, x=None, pre=None) == INVALID and norm(x=None) == INVALID
    assert norm(pre=None) == INVALID and norm(ldy=2047) == INVALID and norm(ldg=2000) == INVALID
    for name in ("y", "gate", "h", "post", "chan", "pre", "ho", "x"):
        assert norm(**{name: A(20) + 8}) == ALIGNMENT
    assert norm(ho=A(0)) == INVALID and norm(x=A(2)) == INVALID and norm(x=A(6)) == INVALID and norm(ho=A(2) + 16) == INVALID


def test_bindings_refuse_what_is_not_on_a_device():
    t = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError):
        gdn.KvCache(torch.zeros(2, 4, 1, 64), torch.zeros(2, 4, 1, 64))
    with pytest.raises(ValueError):
        gdn.gdn_kv_extend(16, t, t, t, t.view(4, 1), t, t[:1], t, t, t)
    with pytest.raises(ValueError):
        gdn.gdn_norm_residual(gdn.make_norm_dims(8), torch.zeros(2, 8, dtype=torch.bfloat16))
    with pytest.raises(TypeError):
        gdn.make_attn_dims(2, 2, 64, torch.float16)
