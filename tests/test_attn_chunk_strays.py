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


def late_borders(b, d, odt):
    """(sequence, kv head, key): keys of a unit that some of its rows do not see, at which another worker's part begins (csrc/gdn_chunk_plan.h;
    one unit a sequence and kv head, a worker is a pair of SMs)."""
    G, heads = b.Hq // b.Hkv, b.Hkv * (d // 64 if odt == F32 else 1)
    cost, workers = 768 if d == 256 else 512, torch.cuda.get_device_properties(0).multi_processor_count // 2
    at = [0]
    for n in b.len_list:
        at += [at[-1] + (cost + n) * (h + 1) for h in range(heads)]
    total = at[-1]
    W = max(1, min(workers, total // 512))
    out = set()
    for s, (new, n) in enumerate(zip(b.new, b.len_list)):
        assert new <= 2 * (128 // G)
        for h in range(heads):
            first = at[s * heads + h] + cost
            owner = lambda t: ((first + 128 * t + 1) * W - 1) // total
            for t in range((n - new + 1) // 128 + 1, (n - 1) // 128 + 1):
                if owner(t) != owner(t - 1):
                    out.add((s, h // (heads // b.Hkv), 128 * t))
    return sorted(out)


@pytest.mark.parametrize("dt,odt,peak", [(BF, BF, False), (BF, F32, False), (F32, F32, False), (BF, BF, True), (BF, F32, True)])
@pytest.mark.parametrize("d,G,Hkv,new,lens", [(256, 1, 3, [256] * 12, [700] * 12), (128, 1, 6, [250] * 12, [900, 1100, 2000] * 4),
                                              (64, 1, 2, [256] * 20, [1000] * 20), (128, 2, 8, [128] * 9, [1000 + 37 * i for i in range(9)])])
def test_strays_on_both_sides_of_a_border_between_workers(dt, odt, d, G, Hkv, new, lens, peak):
    """Rows that see an infinity in the one worker's part and no key in the other's get that infinity, whatever the other's tokens hold;
    over a bf16 cache also where a score of another part leaves the part of the infinity no weight (peak)."""
    b = R.Batch(new, lens, G * Hkv, Hkv, d, 16, dt, gate=True, seed=25)
    if peak:
        b.q[:, ::d] = 40.0   # the first key's score: 40 * 40 / sqrt(d), at least 100 above the others
        for s in range(len(new)):
            b.k[int(b.table[s, 0]), 0, :, 0] = 40.0
    clean = run(b, odt).clone().view(b.T, -1, d)
    assert torch.all(torch.isfinite(clean))
    borders = late_borders(b, d, odt)
    assert len(borders) > 0
    want = torch.zeros(b.T, b.Hq, d, device="cuda")
    for s, h, j in borders:
        for key, ch, x in ((j - 1, 5, math.inf), (j, 6, -math.inf), (j, d - 1, math.nan), (j + 1, 5, math.inf)):
            if key < lens[s]:
                hit = plant(b, [(s, key, h, ch, x)])
                want[hit] += x
    for _ in range(3):
        got = run(b, odt).view(b.T, -1, d)
        hit = want != 0   # (a NaN is)
        same = (got == clean) | hit
        assert torch.all(same), torch.argwhere(~same)[:5].tolist()
        assert torch.all(torch.isnan(got[hit]) == torch.isnan(want[hit]))
        inf = hit & ~torch.isnan(want)
        assert inf.any() and torch.all(got[inf].float() == want[inf])
