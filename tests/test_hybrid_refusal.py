"""examples/hybrid_decode.py with a sequence that is refused (its table is full) or idle: the caches, states and outputs of the others
are those of the same batch in which it is not."""
import pytest
import torch

from tests.test_hybrid_example import example

pytestmark = pytest.mark.gpu
B, LONG = 4, 1   # sequence LONG starts just under its most tokens


def cache_of(m, b):
    n = int(m.lens[b])
    rows = torch.arange(n, device="cuda")
    page = m.table[b].long()[rows // m.ps]
    return m.kv.k[page, rows % m.ps], m.kv.v[page, rows % m.ps]


def start(ex, K, full):
    m = ex.HybridDecoder(B, K, Hk=2, Hv=4, Hq=4, Hkv=2, D=64, rope=32, max_len=64, seed=3)
    if full:   # one token left for LONG: K = 1 is refused at the second step, K > 1 at the first
        m.lens[LONG], m.held[LONG] = 63, 4
        m.table[LONG, :4] = m.free[int(m.n_free) - 4:int(m.n_free)]
        m.n_free -= 4
    return m


@pytest.mark.parametrize("K", [1, 3])
@pytest.mark.parametrize("graph", [False, True])
def test_the_others_go_on_as_without_it(K, graph):
    if graph and K > 1:
        pytest.skip("the plain step is what is captured")
    ex = example()
    a, b = start(ex, K, False), start(ex, K, True)
    run = b.step
    g = torch.Generator(device="cuda").manual_seed(7)
    others = [i for i in range(B) if i != LONG]
    rows = [i * K + p for i in others for p in range(K)]
    for i in range(6):
        x = torch.randn(B * K, 2048, generator=g, device="cuda").to(torch.bfloat16)
        a.hidden.copy_(x)
        b.hidden.copy_(x)
        a.step()
        run()
        assert torch.equal(a.xn[rows], b.xn[rows])
        if K > 1:
            acc = torch.tensor([1 + (i + j) % K for j in range(B)], dtype=torch.int32, device="cuda")
            a.commit(acc)
            b.commit(acc)
        elif graph and i == 0:
            run = b.capture().replay
        assert a.lens[others].tolist() == b.lens[others].tolist() and a.held[others].tolist() == b.held[others].tolist()
        assert torch.equal(a.S[others], b.S[others]) and torch.equal(a.conv[others], b.conv[others])
        for j in others:
            assert all(torch.equal(x, y) for x, y in zip(cache_of(a, j), cache_of(b, j)))
    assert b.status.tolist() == [32 if j == LONG else 0 for j in range(B)] and int(a.status.max()) == 0
    assert int(b.lens[LONG]) == (64 if K == 1 else 63)


@pytest.mark.parametrize("K", [1, 3])
def test_a_refused_sequence_keeps_its_cache(K):
    ex = example()
    m = start(ex, K, True)
    m.lens[LONG] = 64
    m.kv.k.normal_()
    m.kv.v.normal_()
    before, state = [t.clone() for t in cache_of(m, LONG)], m.S[LONG].clone()
    m.hidden.normal_()
    m.step()
    if K > 1:
        m.commit(torch.full((B,), 2, dtype=torch.int32, device="cuda"))
        assert torch.equal(m.S[LONG], state)
    assert all(torch.equal(x, y) for x, y in zip(before, cache_of(m, LONG))) and int(m.lens[LONG]) == 64


def test_an_idle_sequence_leaves_the_others_alone():
    """n_new 0 for one sequence: no row of the others goes to its neighbour's slots."""
    ex = example()
    a, b = start(ex, 1, False), start(ex, 1, False)
    g = torch.Generator(device="cuda").manual_seed(8)
    b.n_new[LONG] = 0
    others = [i for i in range(B) if i != LONG]
    for _ in range(3):
        x = torch.randn(B, 2048, generator=g, device="cuda").to(torch.bfloat16)
        a.hidden.copy_(x)
        b.hidden.copy_(x)
        a.step()
        b.step()
        assert torch.equal(a.xn[others], b.xn[others])
    for j in others:
        assert all(torch.equal(x, y) for x, y in zip(cache_of(a, j), cache_of(b, j)))
    assert int(b.lens[LONG]) == 0 and int(b.status.max()) == 0


def test_drafts_that_are_all_accepted_give_the_lengths_and_states_of_plain_decoding():
    """Three tokens a step, all kept, beside the same tokens one a step: lengths, pages held and the page order are equal, the states and
    the cached keys and values of the accepted tokens agree to bf16 rounding of the projections' inputs."""
    ex = example()
    kw = dict(Hk=2, Hv=4, Hq=4, Hkv=2, D=64, rope=32, max_len=64, seed=3)
    a, b = ex.HybridDecoder(B, 1, **kw), ex.HybridDecoder(B, 3, **kw)
    g = torch.Generator(device="cuda").manual_seed(9)
    for _ in range(5):
        x = torch.randn(B, 3, 2048, generator=g, device="cuda").to(torch.bfloat16)
        for t in range(3):
            a.hidden.copy_(x[:, t])
            a.step()
        b.hidden.copy_(x.view(B * 3, 2048))
        b.step()
        b.commit(torch.full((B,), 3, dtype=torch.int32, device="cuda"))
    assert a.lens.tolist() == b.lens.tolist() == [15] * B and a.held.tolist() == b.held.tolist()
    rel = lambda x, y: float((x.double() - y.double()).norm() / y.double().norm())
    assert rel(b.S, a.S) <= 2e-2
    for j in range(B):
        assert all(rel(x, y) <= 2e-2 for x, y in zip(cache_of(b, j), cache_of(a, j)))
