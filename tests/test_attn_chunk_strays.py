"""gdn_attn_chunk with infinite and NaN values among tokens that some rows see and others do not: many parts one after another in a
worker, units that several workers hold."""
import math

import pytest
import torch

from tests import chunk_ref as R
from tests.test_attn_chunk import BF, F32, KINDS, run

pytestmark = pytest.mark.gpu


def plant(b, spots):
    """spots: (sequence, key, kv head, channel, value).  The elements of the result whose rows see one of them."""
    G = b.Hq // b.Hkv
    hit = torch.zeros(b.T, b.Hq, b.d, dtype=torch.bool, device="cuda")
    for s, j, h, c, x in spots:
        b.v[int(b.table[s, j // b.ps]), j % b.ps, h, c] = x
        first = int(b.cu[s]) + max(0, j - (b.len_list[s] - b.new[s]))
        hit[first:int(b.cu[s + 1]), h * G:(h + 1) * G, c] = True
    return hit


@pytest.mark.parametrize("dt,odt", [(BF, BF), (BF, F32)])
@pytest.mark.parametrize("d,G,Hkv,new,lens", [(128, 8, 16, [600, 350], [700, 3000]), (64, 8, 16, [900], [1100]), (256, 6, 8, [500, 260], [500, 1500]),
                                              (128, 3, 24, [700, 90, 1], [700, 2500, 4000]), (256, 1, 24, [513, 700], [600, 700])])
def test_many_parts_a_worker_some_with_strays(dt, odt, d, G, Hkv, new, lens):
    """What one unit's tokens hold does not reach the units before and after it in a worker."""
    b = R.Batch(new, lens, G * Hkv, Hkv, d, 16, dt, gate=True, seed=22)
    clean = run(b, odt).clone().view(b.T, -1, d)
    g = torch.Generator().manual_seed(23)
    pick = lambda n: int(torch.randint(0, n, (1,), generator=g))
    spots = []
    for s, n in enumerate(new):
        for _ in range(6):
            spots.append((s, lens[s] - n + pick(n), pick(Hkv), pick(d), (math.nan, math.inf, -math.inf)[pick(3)]))
        spots.append((s, lens[s] - 1, pick(Hkv), pick(d), math.inf))   # the last row alone sees it
    hit = plant(b, spots)
    for _ in range(20):
        got = run(b, odt).view(b.T, -1, d)
        assert torch.all(~torch.isfinite(got[hit]))
        same = (got == clean) | hit
        assert torch.all(same), torch.argwhere(~same)[:5].tolist()


@pytest.mark.parametrize("dt,odt", KINDS)
@pytest.mark.parametrize("d,G,new,lens", [(256, 4, 70, 20000), (128, 8, 31, 9000), (64, 1, 256, 6000), (128, 2, 3, 4000)])
@pytest.mark.parametrize("gate", [False, True])
def test_split_units_with_strays(dt, odt, d, G, new, lens, gate):
    """Few rows over many keys, joined from many workers' parts; the strays lie in the last of them."""
    b = R.Batch([new], [lens], G, 1, d, 16, dt, gate=gate, seed=24)
    clean = run(b, odt).clone().view(b.T, -1, d)
    off = lens - new
    hit = plant(b, [(0, off + 1, 0, 3, math.inf), (0, off + new // 2, 0, 9, math.nan), (0, lens - 1, 0, d - 1, -math.inf), (0, lens - 1, 0, 0, math.nan)])
    for _ in range(3):
        got = run(b, odt).view(b.T, -1, d)
        assert torch.all(~torch.isfinite(got[hit]))
        same = (got == clean) | hit
        assert torch.all(same), torch.argwhere(~same)[:5].tolist()
