"""gdn_kv_fork, gdn_kv_release, gdn_kv_compact and gdn_kv_copy_pages against lists: whole numbers and copies, all equal."""
import random

import pytest
import torch

import gated_deltanet_linear_decode_gb300 as gdn
from tests import pages_ref as R

pytestmark = pytest.mark.gpu


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


class Books:
    """The same books on the device and in lists."""

    def __init__(self, rng, B, ps, lens, free, width=None):
        held = [-(-n // ps) for n in lens]
        n = sum(held) + free
        perm = list(range(n))
        rng.shuffle(perm)
        P = width or max(held + [0]) + 2
        table, at = [], 0
        for h in held:
            table.append(perm[at:at + h] + [-9] * (P - h))
            at += h
        self.m = R.Shared(ps, table, perm[at:] + [-5] * at, n - at, lens, held, [0] * n)
        self.put()

    def put(self):
        m = self.m
        self.table, self.free, self.n_free = i32(m.table).view(len(m.lens), m.P), i32(m.free), i32([m.n_free])
        self.lens, self.held, self.refs = i32(m.lens), i32(m.held), i32(m.refs)

    def same(self):
        m = self.m
        assert self.lens.tolist() == m.lens and self.held.tolist() == m.held
        assert self.refs.tolist() == m.refs
        assert self.n_free.tolist() == [m.n_free]
        assert self.free.tolist()[:m.n_free] == m.free[:m.n_free]
        assert self.table.tolist() == m.table

    def fork(self, src, dst, take):
        N = len(src)
        cs, cd, st = i32([-7] * N), i32([-7] * N), i32([0] * N)
        gdn.gdn_kv_fork(self.m.ps, i32(src), i32(dst), i32(take), self.lens, self.held, self.table, self.refs, self.free, self.n_free,
                        cs, cd, dev_status=st)
        want = self.m.fork(src, dst, take)
        assert (cs.tolist(), cd.tolist(), st.tolist()) == want
        self.same()
        return want

    def release(self, keep):
        B = len(keep)
        cs, cd, st = i32([-7] * B), i32([-7] * B), i32([0] * B)
        gdn.gdn_kv_release(self.m.ps, i32(keep), self.lens, self.held, self.table, self.refs, self.free, self.n_free, cs, cd, dev_status=st)
        want = self.m.release(keep)
        assert (cs.tolist(), cd.tolist(), st.tolist()) == want
        self.same()
        return want

    def compact(self, in_place=True, extra=0):
        m = self.m
        N, C = m.N, m.N // 2 + extra
        page_map, cs, cd, n, st = i32([-7] * N), i32([-7] * max(1, C)), i32([-7] * max(1, C)), i32([-7]), i32([0] * len(m.lens))
        old, out = self.table.clone(), None if in_place else self.table.clone()
        gdn.gdn_kv_compact(self.held, self.table, self.refs, self.free, self.n_free, page_map, cs, cd, n, block_table_out=out,
                           dev_status=st)
        new, moves = m.compact()
        if not in_place:
            assert torch.equal(self.table, old)
            self.table = out
        assert page_map.tolist() == new and n.tolist() == [len(moves)]
        pad = [-1] * (len(cs) - len(moves))
        assert cs.tolist() == [a for a, _ in moves] + pad and cd.tolist() == [z for _, z in moves] + pad
        self.same()
        return st.tolist()


@pytest.mark.parametrize("B,ps,max_len", [(4, 16, 100), (64, 16, 900), (33, 7, 300), (300, 1, 40), (1025, 16, 60), (40, 2, 600)])
def test_forks_releases_and_compactions(B, ps, max_len):
    """Several rounds: random forks (full, in the middle of a page, empty), random shortening, now and then a compaction."""
    rng = random.Random(B * 100 + ps)
    parents = max(1, B // 4)
    s = Books(rng, B, ps, [rng.randint(1, max_len) for _ in range(parents)] + [0] * (B - parents), 3 * B + 4, width=-(-max_len // ps) + 2)
    for step in range(5):
        m = s.m
        empty = [b for b in range(B) if m.lens[b] == 0 and m.held[b] == 0]
        full = [b for b in range(B) if m.lens[b] > 0]
        rng.shuffle(empty)
        empty = empty[: max(1, len(empty) * 2 // 3)] if empty else []
        src = [rng.choice(full) for _ in empty] if full else []
        take = [rng.choice([m.lens[a], rng.randint(0, m.lens[a]), m.lens[a] // ps * ps]) for a in src]
        if src:
            s.fork(src, empty[:len(src)], take)
        keep = [rng.choice([n, n, rng.randint(0, n), 0]) for n in m.lens]
        s.release(keep)
        if step % 2:
            s.compact(in_place=step == 1, extra=step)
    s.release([0] * B)
    assert s.m.n_free == s.m.N and not any(s.m.refs)
    assert sorted(s.free.tolist()) == list(range(s.m.N))


@pytest.mark.parametrize("B,ps,max_len", [(400, 1, 300), (64, 16, 20000), (8000, 16, 60)])
def test_large_tables(B, ps, max_len):
    """As above with tables of 48,000 to 120,000 entries: clusters of 16 CTAs, and more blocks of entries a warp than it holds."""
    test_forks_releases_and_compactions(B, ps, max_len)


def test_fork_then_release_restores_the_stack():
    rng = random.Random(5)
    s = Books(rng, 40, 8, [200, 77, 64] + [0] * 37, 60)
    stack, n = s.free.tolist(), s.m.n_free
    s.fork([i % 3 for i in range(37)], list(range(3, 40)), [[200, 199, 13][i // 3 % 3] if i % 3 == 0 else [77, 70][i % 2] if i % 3 == 1 else 64 for i in range(37)])
    s.release(list(s.m.lens[:3]) + [0] * 37)
    assert s.m.n_free == n and s.free.tolist()[:n] == stack[:n]


def test_release_without_sharing_is_truncation():
    for ps, B in ((16, 64), (3, 700)):
        rng = random.Random(ps)
        a = Books(rng, B, ps, [rng.randint(0, 150) for _ in range(B)], 20)
        keep = [rng.randint(0, n) for n in a.m.lens]
        lens, held, free, nf = a.lens.clone(), a.held.clone(), a.free.clone(), a.n_free.clone()
        gdn.gdn_kv_truncate(ps, i32(keep), lens, held, a.table, free, nf)
        a.release(keep)
        assert torch.equal(lens, a.lens) and torch.equal(held, a.held) and torch.equal(nf, a.n_free)
        assert torch.equal(free[: int(nf)], a.free[: int(nf)])


def test_shared_middle_of_a_page_is_copied():
    """Three holders of a page end inside it, two of them in the call in which the third gives it up."""
    s = Books(random.Random(1), 4, 4, [12, 0, 0, 0], 9)
    s.fork([0, 0, 0], [1, 2, 3], [12, 12, 8])
    want = s.release([12, 7, 6, 0])
    assert want[0][1] >= 0 and want[0][2] == want[0][1] and want[0][0] == -1
    s.release([5, 7, 6, 0])
    s.release([0, 0, 0, 0])
    assert s.m.n_free == s.m.N


def test_all_holders_end_inside_a_page():
    """Each gets a copy, and the page itself goes back."""
    s = Books(random.Random(2), 3, 4, [8, 0, 0], 6)
    s.fork([0, 0], [1, 2], [8, 8])
    want = s.release([3, 2, 1])
    assert min(want[1]) >= 0
    s.release([0, 0, 0])


@pytest.mark.parametrize("free", [0, 1, 4, 100])
def test_refusals(free):
    rng = random.Random(free)
    s = Books(rng, 12, 8, [50, 33, 16, 8, 1, 0, 0, 0, 0, 0, 0, 0], free)
    st = s.fork([0, 0, 1, 2, 9, -1, 12, 0, 1, 3, 0, 4, 5], [5, 5, 6, 7, 8, 8, 8, 0, 3, -1, 12, 8, 9], [50, 20, 34, 16, 0, 1, 1, 1, 1, 1, 1, 1, 0])[2]
    assert st.count(32) >= 8
    s.fork([0, 1, 4, 2], [9, 9, 10, 11], [49, 33, 1, -1])
    s.release([51, 33, -1, 0, 1] + [rng.randint(0, n) if n else 0 for n in s.m.lens[5:]])
    s.release([9] + [n // 2 for n in s.m.lens[1:]])


def test_bad_pages():
    """Pages outside the cache are handed on without a count, and end nowhere."""
    s = Books(random.Random(7), 6, 4, [14, 16, 9, 0, 0, 0], 5)
    m = s.m
    m.table[0][1], m.table[0][3], m.table[2][0] = 10 ** 9, -3, m.N
    s.put()
    st = s.fork([0, 2, 0], [3, 4, 5], [14, 9, 7])[2]
    assert st == [64, 64, 64]
    s.release([14, 16, 0, 0, 5, 0])
    assert s.compact() == [64, 0, 0, 0, 64, 0]
    s.release([0] * 6)
    m.held[1] = m.P + 1
    m.lens[1] = 3
    s.put()
    assert s.release([0, 2, 0, 0, 0, 0])[2][1] == 32
    st = i32([0] * 6)
    N = m.N
    gdn.gdn_kv_compact(s.held, s.table, s.refs, s.free, s.n_free, i32([0] * N), i32([0] * N), i32([0] * N), i32([0]), dev_status=st)
    assert st.tolist() == [0, 64, 0, 0, 0, 0]


def test_a_page_in_the_stack_and_in_a_table():
    """Wrong books: a page that has no room on the stack is dropped, and the stack stays within its bounds."""
    s = Books(random.Random(9), 3, 4, [16, 8, 0], 2)
    s.m.n_free = s.m.N - 1
    s.m.free = list(range(s.m.N))
    s.put()
    st = s.release([0, 0, 0])[2]
    assert 64 in st and s.m.n_free == s.m.N


@pytest.mark.parametrize("N,fill", [(1, 1), (2, 1), (33, 5), (64, 64), (5000, 1700), (70001, 30000)])
def test_compaction_of_caches(N, fill):
    rng = random.Random(N)
    B = min(fill, 50)
    each = [fill // B + (b < fill % B) for b in range(B)]
    perm = rng.sample(range(N), fill)
    P, table, at = max(each) + 1, [], 0
    for h in each:
        table.append(perm[at:at + h] + [-9] * (P - h))
        at += h
    s = Books(rng, 1, 1, [0], 1)
    s.m = R.Shared(1, table, [0] * N, 0, each, each, [0] * N)
    s.put()
    s.compact(in_place=N % 2 == 0)
    s.compact()   # nothing is left to move
    assert s.m.n_free == N - fill


def test_nothing_held():
    s = Books(random.Random(1), 3, 4, [0, 0, 0], 7)
    s.compact()
    assert s.m.n_free == 7


def _halves(layout, pages, ps, H, d, dt):
    g = torch.Generator(device="cuda").manual_seed(pages)
    rn = lambda *s: torch.randn(*s, generator=g, device="cuda").to(dt)
    if layout == "thd":
        return rn(pages, ps, H, d), rn(pages, ps, H, d)
    if layout == "htd":
        return rn(pages, H, ps, d).transpose(1, 2), rn(pages, H, ps, d).transpose(1, 2)
    if layout == "both":          # keys and values of a token side by side
        t = rn(pages, ps, H, 2 * d)
        return t[..., :d], t[..., d:]
    if layout == "pht":           # page and head outside, odd pitches
        t = rn(pages, H + 1, ps + 3, d + 8)
        return t[:, :H, :ps, :d].transpose(1, 2), t.clone()[:, :H, :ps, :d].transpose(1, 2)
    t = rn(H, pages, ps, d)       # a head's pages together
    return t.permute(1, 2, 0, 3), t.clone().permute(1, 2, 0, 3)


@pytest.mark.parametrize("layout", ["thd", "htd", "both", "pht", "hp"])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("ps,H,d,n", [(16, 2, 256, 20), (1, 1, 64, 300), (11, 3, 128, 7), (100, 8, 64, 3)])
def test_copies(layout, dt, ps, H, d, n):
    pages = 2 * n + 3
    k, v = _halves(layout, pages, ps, H, d, dt)
    perm = torch.randperm(pages, generator=torch.Generator().manual_seed(n)).to(torch.int32)
    src, dst = perm[:n].clone(), perm[n:2 * n].clone()
    src[::5], dst[1::7] = -1, -1
    there = (src >= 0) & (dst >= 0)
    want_k, want_v = k.clone(), v.clone()
    want_k[dst[there].long().cuda()] = k[src[there].long().cuda()]
    want_v[dst[there].long().cuda()] = v[src[there].long().cuda()]
    base_k = k._base.clone() if k._base is not None else None
    st = i32([0])
    dims = gdn.make_attn_dims(H, H, d, dt, dt)
    gdn.gdn_kv_copy_pages(dims, gdn.KvCache(k, v), src.cuda(), dst.cuda(), dev_status=st)
    bits = torch.int16 if dt == torch.bfloat16 else torch.int32
    eq = lambda a, b: torch.equal(a.contiguous().view(bits), b.contiguous().view(bits))
    assert eq(k, want_k) and eq(v, want_v) and st.tolist() == [0]
    if layout == "pht" and base_k is not None:   # what lies between the rows is not touched
        base_k[:, :H, :ps, :d] = k.transpose(1, 2)
        assert eq(base_k, k._base)


def test_copies_keep_the_bits_of_any_value():
    k = torch.randint(-2 ** 15, 2 ** 15, (9, 4, 2, 64), device="cuda", dtype=torch.int16).view(torch.bfloat16)
    v = torch.randint(-2 ** 15, 2 ** 15, (9, 4, 2, 64), device="cuda", dtype=torch.int16).view(torch.bfloat16)
    a, b = k.view(torch.int16).clone(), v.view(torch.int16).clone()
    gdn.gdn_kv_copy_pages(gdn.make_attn_dims(2, 2, 64), gdn.KvCache(k, v), i32([0, 8]), i32([4, 5]))
    a[[4, 5]], b[[4, 5]] = a[[0, 8]], b[[0, 8]]
    assert torch.equal(k.view(torch.int16), a) and torch.equal(v.view(torch.int16), b)


def test_copies_of_pages_outside():
    k, v = torch.randn(5, 2, 1, 64, device="cuda"), torch.randn(5, 2, 1, 64, device="cuda")
    k0, v0, st = k.clone(), v.clone(), i32([0])
    d = gdn.make_attn_dims(1, 1, 64, torch.float32)
    gdn.gdn_kv_copy_pages(d, gdn.KvCache(k, v), i32([5, 0, 2 ** 31 - 1, 1]), i32([1, 5, 0, -2 ** 31]), dev_status=st)
    assert torch.equal(k, k0) and torch.equal(v, v0) and st.tolist() == [64]
    gdn.gdn_kv_copy_pages(d, gdn.KvCache(k, v), i32([]), i32([]))


def test_replayed_in_a_graph_on_another_stream():
    """Fork, copies, release captured once: replays end where they began, with the copies made."""
    rng = random.Random(3)
    s = Books(rng, 20, 8, [100, 37] + [0] * 18, 40)
    g = torch.Generator(device="cuda").manual_seed(1)
    k, v = torch.randn(s.m.N, 8, 1, 64, generator=g, device="cuda"), torch.randn(s.m.N, 8, 1, 64, generator=g, device="cuda")
    dims, kv = gdn.make_attn_dims(1, 1, 64, torch.float32), gdn.KvCache(k, v)
    src, dst, take = i32([i % 2 for i in range(18)]), i32(list(range(2, 20))), i32([100, 37] * 9)
    keep, cs, cd, rs, rd = i32([100, 37] + [0] * 18), i32([0] * 18), i32([0] * 18), i32([0] * 20), i32([0] * 20)

    def step():
        gdn.gdn_kv_fork(8, src, dst, take, s.lens, s.held, s.table, s.refs, s.free, s.n_free, cs, cd)
        gdn.gdn_kv_copy_pages(dims, kv, cs, cd)
        gdn.gdn_kv_release(8, keep, s.lens, s.held, s.table, s.refs, s.free, s.n_free, rs, rd)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    want = s.m.fork(src.tolist(), dst.tolist(), take.tolist())
    s.m.release(keep.tolist())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(3):
        k[cd.long()] = 0
        graph.replay()
    torch.cuda.synchronize()
    assert (cs.tolist(), cd.tolist()) == want[:2]
    assert torch.equal(k[cd.long()], k[cs.long()])
    free, held = s.free.tolist()[: s.m.n_free], s.m.n_free
    assert free == s.m.free[:held] and s.n_free.tolist() == [held]
    assert s.refs.tolist() == s.m.refs and s.lens.tolist() == s.m.lens
