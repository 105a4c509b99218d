"""The two halves of a cache share no element, wherever they lie inside one another (CPU only: argument checks)."""
import itertools
import random

import pytest

import gated_deltanet_linear_decode_gb300 as gdn
from tests.test_attn_abi import A, INVALID, OK, adims, append, attn, cache, norm


def status(k, v, pages, ps, strides, **kw):
    d = adims(**kw)
    return attn(dims=d, kc=gdn.GdnKvCache(A(0) + k, A(0) + v, pages, ps, *strides), B=0)   # B = 0: the cache is looked at, nothing runs


@pytest.mark.parametrize("delta", [16, 512, 8192 - 16, 8192, 50 * 8192, 100 * 8192 - 16])
def test_a_half_within_the_other(delta):
    """Dense halves [100][16][2][256] of bf16, 1,638,400 bytes each."""
    kc = cache(k=A(0), v=A(0) + delta)
    assert attn(B=0, kc=kc) == INVALID and append(T=0, kc=kc) == INVALID
    assert attn(B=0, kc=cache(k=A(0) + delta, v=A(0))) == INVALID
    assert attn(B=0, kc=cache(k=A(0), v=A(0) + 100 * 16 * 2 * 256 * 2)) == OK


def test_halves_side_by_side():
    row, page = 2 * 256, 16 * 2 * 256                                            # elements
    assert status(0, page * 2, 100, 16, (2 * page, row, 256)) == OK              # page by page
    assert status(0, row * 2, 100, 16, (2 * page, 2 * row, 256)) == OK           # token by token
    assert status(0, 256 * 2, 100, 16, (2 * page, 2 * row, 512)) == OK           # head by head
    assert status(0, row * 2, 100, 16, (2 * page, row, 256)) == INVALID
    assert status(0, page * 2 + 16, 100, 16, (2 * page, row, 256)) == INVALID
    assert status(page * 2 * 3, 0, 100, 16, (2 * page, row, 256)) == OK          # v first, pages apart by an odd number


def test_against_all_elements():
    """Small caches of 64 channels: the answer is that of the sets of 16-byte pieces themselves."""
    rng, seen = random.Random(5), set()
    for _ in range(3000):
        n = [rng.randint(1, 3), rng.randint(1, 4), rng.randint(1, 3)]
        order, span, st = rng.sample(range(3), 3), 8, [8, 8, 8]                  # in pieces of 8 elements
        for i in order:
            if n[i] > 1:
                st[i] = span + rng.choice([0, 0, 1, 8, 16, 24])
                span += (n[i] - 1) * st[i]
        delta = rng.choice([rng.randint(1, span + 8), 8 * rng.randint(1, 1 + span // 8)])
        at = {sum(i * s for i, s in zip(idx, st)) + c for idx in itertools.product(*map(range, n)) for c in range(8)}
        want = INVALID if at & {x + delta for x in at} else OK
        got = {status(*kv, n[0], n[1], [8 * s for s in st], Hq=n[2], Hkv=n[2], d=64) for kv in ((0, 16 * delta), (16 * delta, 0))}
        assert got == {want}, (n, st, delta)
        seen.add(want)
    assert seen == {OK, INVALID}


def test_spans_past_64_bits():
    """Pitches and strides whose products pass 64 bits: what the rows cover is not taken for what is left of the product."""
    assert status(0, 1 << 33, 1 << 26, 16, (1 << 38, 512, 256)) == INVALID       # 2^64 elements from page to page
    T = (1 << 24) + 1                                                            # rows 2^40 elements apart: y covers all that lies after it
    assert norm(T=T, y=A(0), ldy=1 << 40, gate=None, cols=0, post=None, chan=None, ho=A(90), x=None, pre=None, h=A(90)) == INVALID
    assert attn(q=A(0) + (1 << 20), kc=cache(k=A(2), v=A(3)), B=T, ldq=1 << 40, out=A(90), ws=A(7)) == INVALID
