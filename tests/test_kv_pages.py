"""gdn_kv_extend and gdn_kv_truncate against a sequential allocator: every output is a whole number and equal."""
import random

import pytest
import torch

import gated_deltanet_linear_decode_gb300 as gdn
from tests import attn_ref as R

pytestmark = pytest.mark.gpu


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


class State:
    """B sequences with random lengths, tables and a shuffled free stack, on the device and in the model."""

    def __init__(self, rng, B, ps, max_len, free, width=None, lens=None):
        self.ps = ps
        lens = [rng.randint(0, max_len) for _ in range(B)] if lens is None else lens
        held = [-(-n // ps) + (rng.random() < 0.2) for n in lens]   # now and then a page more than needed
        n = sum(held) + free
        perm = list(range(n))
        rng.shuffle(perm)
        self.P = width or max(held + [0]) + 3
        table, at = [], 0
        for h in held:
            table.append(perm[at:at + h] + [-9] * (self.P - h))
            at += h
        fl = perm[at:] + [-5] * at
        self.model = R.Pages(ps, table, fl, n - at, lens, held)
        self.table, self.free, self.n_free = i32(table).view(B, self.P), i32(fl), i32([n - at])
        self.lens, self.held = i32(lens), i32(held)

    def extend(self, new, T, in_place=True):
        B = len(new)
        o = {} if in_place else dict(seq_len_out=i32([-1] * B), n_pages_out=i32([-1] * B), free_count_out=i32([-1]))
        slots, pos, cu, st = i32([-3] * T), i32([-3] * T), i32([-3] * (B + 1)), i32([0] * B)
        before = (self.lens.clone(), self.held.clone(), self.n_free.clone())
        gdn.gdn_kv_extend(self.ps, i32(new), self.lens, self.held, self.table, self.free, self.n_free, slots, pos, cu,
                          dev_status=st, **o)
        want = self.model.extend(new, T)
        if not in_place:
            assert all(torch.equal(x, y) for x, y in zip(before, (self.lens, self.held, self.n_free)))
            self.lens, self.held, self.n_free = o["seq_len_out"], o["n_pages_out"], o["free_count_out"]
        assert (slots.tolist(), pos.tolist(), cu.tolist()) == want[:3]
        assert st.tolist() == [32 if b in want[3] else 0 for b in range(B)]
        self.same()
        return want

    def truncate(self, keep, in_place=True):
        B = len(keep)
        o = {} if in_place else dict(seq_len_out=i32([-1] * B), n_pages_out=i32([-1] * B), free_count_out=i32([-1]))
        st = i32([0] * B)
        gdn.gdn_kv_truncate(self.ps, i32(keep), self.lens, self.held, self.table, self.free, self.n_free,
                            dev_status=st, **o)
        refused = self.model.truncate(keep)
        if not in_place:
            self.lens, self.held, self.n_free = o["seq_len_out"], o["n_pages_out"], o["free_count_out"]
        assert st.tolist() == [32 if b in refused else 0 for b in range(B)]
        self.same()

    def same(self):
        m = self.model
        assert self.lens.tolist() == m.lens and self.held.tolist() == m.held
        assert self.n_free.tolist() == [len(m.free)]
        assert self.free.tolist()[: len(m.free)] == m.free
        assert self.table.tolist() == m.table


@pytest.mark.parametrize("B,ps,max_len", [(1, 16, 100), (3, 1, 5), (64, 16, 900), (33, 7, 300), (1025, 16, 60), (2500, 4, 30)])
@pytest.mark.parametrize("in_place", [True, False])
def test_steps_of_decode_verify_and_truncate(B, ps, max_len, in_place):
    rng = random.Random(B * 100 + ps)
    s = State(rng, B, ps, max_len, 6 * B + 10, width=-(-max_len // ps) + 12)
    for step in range(6):
        K = [1, 3, 16, 0, 2, 5][step]
        new = [K if rng.random() < 0.9 else 0 for _ in range(B)]
        s.extend(new, sum(new) + rng.randint(0, 9), in_place)
        keep = [x if rng.random() < 0.3 else max(0, x - rng.randint(0, K)) if rng.random() < 0.9 else 0 for x in s.model.lens]
        s.truncate(keep, in_place)


@pytest.mark.parametrize("B,ps,max_len", [(40, 2, 400), (300, 2, 60), (512, 2, 60), (513, 2, 60)])
def test_many_pages(B, ps, max_len):
    """Caches of more than 4096 pages, a few to a thread and more sequences than threads."""
    rng = random.Random(B)
    s = State(rng, B, ps, max_len, 4200, width=-(-max_len // ps) + 12)
    for step in range(3):
        new = [rng.randint(0, 8) for _ in range(B)]
        s.extend(new, sum(new) + 5)
        s.truncate([rng.randint(0, x) for x in s.model.lens])


@pytest.mark.parametrize("lens", [[8000, 1, 0, 500], [65536], [1] * 9, [4097, 4095, 4096]])
def test_prompts_into_an_empty_cache(lens):
    ps = 16
    s = State(random.Random(3), len(lens), ps, 0, sum(-(-n // ps) for n in lens) + 1, width=max(lens) // ps + 1,
              lens=[0] * len(lens))
    s.model.held, s.held = [0] * len(lens), i32([0] * len(lens))
    # the pages that the state gave away ahead of need are not in the stack: fine, they are just not used
    s.extend(lens, sum(lens) + 3)
    s.truncate([0] * len(lens))


def test_extend_then_truncate_restores_the_stack():
    rng = random.Random(8)
    s = State(rng, 50, 8, 200, 400)
    stack, lens = s.free.tolist(), list(s.model.lens)
    held = list(s.model.held)
    s.extend([rng.randint(0, 20) for _ in range(50)], 1000)
    s.truncate(lens)
    n = len(s.model.free)
    # an extra page that a sequence held before the extend is given back too, on top of the old stack
    assert [h - x for h, x in zip(held, s.model.held)] == [h - -(-n_ // 8) for h, n_ in zip(held, lens)]
    s2 = State(rng, 20, 8, 200, 400)
    s2.truncate(list(s2.model.lens))          # nothing held past the need
    stack, n = s2.free.tolist(), len(s2.model.free)
    lens = list(s2.model.lens)
    s2.extend([rng.randint(0, 20) for _ in range(20)], 1000)
    s2.truncate(lens)
    assert s2.free.tolist()[:n] == stack[:n] and len(s2.model.free) == n


@pytest.mark.parametrize("free,T", [(0, 500), (5, 500), (23, 500), (400, 37), (400, 0), (11, 60)])
def test_refusals_in_order(free, T):
    """Too few free pages, too few rows, a narrow table, negative requests: refused ones keep what they had."""
    rng = random.Random(free * 1000 + T)
    s = State(rng, 40, 8, 60, free, width=12)
    new = [rng.choice([0, 1, 4, 9, 20, 70, -1]) for _ in range(40)]
    want = s.extend(new, T)
    assert want[3]
    s.extend([0] * 40, 4)
    s.truncate([rng.choice([x, x + 1, -1, 0, x // 2]) for x in s.model.lens])


def test_no_sequences():
    slots, pos, cu, fc = i32([5, 5]), i32([5, 5]), i32([7]), i32([3])
    e = torch.empty(0, dtype=torch.int32, device="cuda")
    gdn.gdn_kv_extend(16, e, e, e, torch.empty(0, 4, dtype=torch.int32, device="cuda"), i32([0, 1, 2]), fc, slots, pos, cu)
    assert slots.tolist() == [-1, -1] and pos.tolist() == [0, 0] and cu.tolist() == [0] and fc.tolist() == [3]


def test_a_full_stack_takes_nothing_more():
    """Pages given back twice do not run past the free list."""
    s = State(random.Random(1), 4, 4, 40, 3, lens=[40, 40, 40, 40])
    s.n_free.fill_(s.free.numel() - 12)
    s.model.free = s.free.tolist()[: s.free.numel() - 12]
    s.truncate([0, 0, 0, 0])
