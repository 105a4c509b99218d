"""include/gdn_pages.h and gdn_attn_chunk: plain C, every declared symbol exported, and bad arguments refused before anything
reaches a device (CPU only: no call here launches a kernel)."""
import ctypes
import os
import re
import subprocess

import pytest
import torch

import gated_deltanet_linear_decode_gb300 as gdn
from tests.test_attn_abi import ALIGNMENT, BAD_DIMS, INCLUDE, INVALID, OK, UNSUPPORTED, WORKSPACE, A, adims, cache


def lib():
    gdn._attn._fn("gdn_attn_chunk")
    gdn._pages._fn("gdn_kv_fork")   # sets the signatures
    return gdn.library()


def test_declared_symbols_are_exported_and_bound():
    src = open(os.path.join(INCLUDE, "gdn_pages.h")).read()
    names = set(re.findall(r"^gdn_status (gdn_[a-z0-9_]+)\s*\(", src, flags=re.M))
    assert names == set(gdn.EXPORTED_SYMBOLS_PAGES)
    out = subprocess.run(["nm", "-D", "--defined-only", gdn._build.build()], capture_output=True, text=True, check=True).stdout
    assert names <= {line.split()[-1] for line in out.splitlines() if line.strip()}
    assert all(hasattr(gdn, n) for n in names)


def test_header_compiles_as_c():
    src = '#include "gdn_pages.h"\nint main(void){ return (int)GDN_OK; }\n'
    r = subprocess.run(["gcc", "-std=c11", "-Wall", "-Werror", "-fsyntax-only", "-I", INCLUDE, "-x", "c", "-"], input=src,
                       text=True, capture_output=True)
    assert r.returncode == 0, r.stderr


def chunk(dims=None, kc=None, B=4, T=40, P=10, q=A(2), ldq=4096, gate=A(3), ldg=4096, cu=A(4), table=A(5), lens=A(6), out=A(7),
          ws=A(8), n=1 << 31, st=None):
    dims = adims() if dims is None else dims
    kc = cache(dims=dims) if kc is None else kc
    return lib().gdn_attn_chunk(ctypes.byref(dims) if dims else None, ctypes.byref(kc) if kc else None, B, T, P, q, ldq, gate, ldg,
                                cu, table, lens, out, ws, n, st, None)


@pytest.mark.parametrize("kw,status", BAD_DIMS)
def test_chunk_dims(kw, status):
    d = adims(**kw)
    assert chunk(dims=d, kc=cache()) == status
    assert gdn.gdn_attn_chunk_workspace_bytes(d, 4, 40) == 0


def test_chunk_arguments():
    assert chunk(B=0) == OK and chunk(T=0) == OK
    assert chunk(B=-1) == INVALID and chunk(T=-1) == INVALID and chunk(P=0) == INVALID
    for name in ("q", "cu", "table", "lens", "out"):
        assert chunk(**{name: None}) == INVALID
        assert chunk(**{name: A(20) + 8}) == ALIGNMENT
    assert chunk(gate=A(20) + 2) == ALIGNMENT and chunk(st=A(20) + 4) == ALIGNMENT and chunk(ws=A(20) + 8) == ALIGNMENT
    assert chunk(ldq=4095) == INVALID and chunk(ldq=4100) == ALIGNMENT and chunk(ldg=1) == INVALID and chunk(ldq=1 << 41) == INVALID
    assert chunk(out=A(2)) == INVALID and chunk(out=A(0) + 4096) == INVALID and chunk(out=A(5)) == INVALID and chunk(out=A(4)) == INVALID
    assert chunk(ws=A(7), out=A(7)) == INVALID and chunk(st=A(6)) == INVALID
    assert chunk(T=1 << 28) == INVALID               # rows past 31 bits
    assert chunk(kc=cache(k=None)) == INVALID and chunk(kc=cache(ps=0)) == INVALID and chunk(kc=cache(s=(8192, 512, 260))) == ALIGNMENT


def test_chunk_workspace():
    n = gdn.gdn_attn_chunk_workspace_bytes(adims(), 4, 40)
    assert n > 0 and n == gdn.gdn_attn_chunk_workspace_bytes(adims(), 1, 100000)
    assert gdn.gdn_attn_chunk_workspace_bytes(adims(), 0, 1) == 0 and gdn.gdn_attn_chunk_workspace_bytes(adims(), 1, 0) == 0
    assert chunk(n=n - 1) == WORKSPACE and chunk(ws=None, n=0) == WORKSPACE


def fork(ps=16, pages=100, B=4, P=10, N=3, **kw):
    a = dict(src=A(0), dst=A(1), len=A(2), lens=A(3), held=A(4), table=A(5), refs=A(6), free=A(7), fc=A(8), cs=A(9), cd=A(10), st=None)
    a.update(kw)
    return lib().gdn_kv_fork(ps, pages, B, P, N, *a.values(), None)


def release(ps=16, pages=100, B=4, P=10, **kw):
    a = dict(keep=A(0), lens=A(1), held=A(2), table=A(3), refs=A(4), free=A(5), fc=A(6), cs=A(7), cd=A(8), st=None)
    a.update(kw)
    return lib().gdn_kv_release(ps, pages, B, P, *a.values(), None)


def compact(pages=100, B=4, P=10, most=50, **kw):
    a = dict(held=A(0), table=A(1), table_out=A(1), refs=A(2), free=A(3), fc=A(4), map=A(5))
    b = dict(cs=A(6), cd=A(7), n=A(8), st=None)
    for k, v in kw.items():
        (a if k in a else b)[k] = v
    return lib().gdn_kv_compact(pages, B, P, *a.values(), most, *b.values(), None)


@pytest.mark.parametrize("f,names", [
    (fork, ("src", "dst", "len", "lens", "held", "table", "refs", "free", "fc", "cs", "cd")),
    (release, ("keep", "lens", "held", "table", "refs", "free", "fc", "cs", "cd")),
    (compact, ("held", "table", "table_out", "refs", "free", "fc", "map", "cs", "cd", "n"))])
def test_book_pointers(f, names):
    for name in names:
        assert f(**{name: None}) == INVALID, name
        assert f(**{name: A(20) + 4}) == ALIGNMENT, name
    assert f(st=A(20) + 8) == ALIGNMENT
    for a in names:          # nothing that is written shares bytes with anything else
        for b in names:
            if a != b and (f, a, b) not in ((compact, "table", "table_out"), (compact, "table_out", "table")):
                i = names.index(b)
                base = {fork: i, release: i, compact: max(0, i - 1)}[f]
                written = [x for x in (a, b) if x not in ("src", "dst", "len", "keep") and not (f is fork and x == "free")
                           and not (f is compact and x in ("held", "table"))]
                if written:
                    assert f(**{a: A(base)}) == INVALID, (a, b)
    assert f(st=A(3)) == INVALID


@pytest.mark.parametrize("f", [fork, release, compact])
def test_book_sizes(f):
    assert f(pages=0) == INVALID and f(B=-1) == INVALID and f(P=0) == INVALID
    assert f(B=16385) == UNSUPPORTED and f(B=16384, P=1 << 17) == UNSUPPORTED
    if f is not compact:
        assert f(ps=0) == INVALID and f(pages=1 << 28) == INVALID


def test_book_edges():
    assert fork(N=0) == OK and fork(N=-1) == INVALID and fork(N=16385) == UNSUPPORTED and release(B=0) == OK
    assert compact(most=49) == INVALID and compact(most=-1) == INVALID and compact(pages=(1 << 30) + 2, most=1 << 30) == UNSUPPORTED
    assert compact(table_out=A(1) + 16) == INVALID


def copies(dims=None, kc=None, n=4, src=A(2), dst=A(3), st=None):
    dims = adims() if dims is None else dims
    return lib().gdn_kv_copy_pages(ctypes.byref(dims), ctypes.byref(kc or cache()), n, src, dst, st, None)


@pytest.mark.parametrize("kw,status", BAD_DIMS)
def test_copy_dims(kw, status):
    assert copies(dims=adims(**kw)) == status


def test_copy_arguments():
    assert copies(n=0) == OK and copies(n=-1) == INVALID
    assert copies(src=None) == INVALID and copies(dst=None) == INVALID and copies(src=A(20) + 4) == ALIGNMENT
    assert copies(st=A(20) + 8) == ALIGNMENT and copies(src=A(0)) == INVALID and copies(dst=A(1) + 4096) == INVALID
    assert copies(st=A(2)) == INVALID and copies(st=A(1)) == INVALID
    assert copies(kc=cache(pages=0)) == INVALID and copies(kc=cache(s=(8192, 512, 260))) == ALIGNMENT
    big = cache(v=A(30), pages=1, ps=1 << 25, dims=adims())
    assert copies(kc=big, src=A(60), dst=A(61)) == UNSUPPORTED


def test_bindings_refuse_what_is_not_on_a_device():
    t = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError):
        gdn.gdn_kv_fork(16, t, t, t, t, t, t.view(4, 1), t, t, t[:1], t, t)
    with pytest.raises(ValueError):
        gdn.gdn_kv_release(16, t, t, t, t.view(4, 1), t, t, t[:1], t, t)
    with pytest.raises(ValueError):
        gdn.gdn_kv_compact(t, t.view(4, 1), t, t, t[:1], t, t, t, t[:1])
