"""gdn_attn_chunk against its definition in 64 bits."""
import math

import numpy as np
import pytest
import torch

import gated_deltanet_linear_decode_gb300 as gdn
from tests import chunk_ref as R

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
_ws = {}


def workspace(dims):
    """One a kind of call, zeroed once: calls of all shapes follow one another on it."""
    key = (dims.head_dim, dims.act_dtype, dims.out_dtype)
    if key not in _ws:
        _ws[key] = torch.zeros(gdn.gdn_attn_chunk_workspace_bytes(dims, 1, 1), dtype=torch.uint8, device="cuda")
    return _ws[key]


def run(b, out_dtype, scale=None, out=None, status=None, ws=None, **kw):
    dims = gdn.make_attn_dims(b.Hq, b.Hkv, b.d, b.dt, out_dtype, scale=scale, **kw)
    out = torch.full((b.T, b.Hq * b.d), 7.0, dtype=out_dtype, device="cuda") if out is None else out
    gdn.gdn_attn_chunk(dims, gdn.KvCache(b.k, b.v), b.q, b.cu, b.table, b.lens, out, gate=b.gate,
                       workspace=workspace(dims) if ws is None else ws, dev_status=status)
    return out


def check(b, out_dtype, scale=None, absent=(), tight=None, status=0):
    st = torch.zeros(len(b.len_list), dtype=torch.int32, device="cuda")
    out = run(b, out_dtype, scale, status=st)
    n = int(b.cu[-1])
    assert torch.all(out[n:] == 7.0)                     # rows of no sequence
    got, (want, size) = out.double().cpu().numpy()[:n], b.want(scale, absent)
    want, size = want[:n], size[:n]
    assert np.all(np.isfinite(got))
    err, lim = np.abs(got - want), R.bound(want, size, b, out_dtype, scale)
    assert np.all(err <= lim), (float((err / lim).max()), np.argwhere(err > lim)[:4].tolist())
    # the roundings of fp32 arithmetic are of either sign: sqrt(len) 2^-24 of the sizes summed, not len
    if out_dtype == F32 and n:
        rel = np.linalg.norm(got - want) / np.linalg.norm(want)
        assert rel <= (tight or 4e-6), rel
    if status is not None:
        assert st.tolist() == ([status] * len(st) if isinstance(status, int) else status)
    again = run(b, out_dtype, scale)
    assert torch.equal(again.view(torch.uint8), out.view(torch.uint8))   # the same from run to run
    return out


KINDS = [(BF, BF), (BF, F32), (F32, F32), (F32, BF)]


@pytest.mark.parametrize("dt,odt", KINDS)
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("G,Hkv", [(1, 3), (2, 1), (6, 2), (8, 2), (16, 1), (5, 2)])
def test_heads_and_types(dt, odt, d, G, Hkv):
    b = R.Batch([70, 1, 33, 0, 5], [70, 130, 300, 50, 5], G * Hkv, Hkv, d, 16, dt, gate=G % 2 == 0, pad=3, seed=d + G)
    check(b, odt)


@pytest.mark.parametrize("dt,odt", KINDS)
@pytest.mark.parametrize("ps", [1, 5, 11, 16, 64, 100, 256, 700])
def test_page_sizes(dt, odt, ps):
    check(R.Batch([140, 3], [333, 129], 4, 2, 128 if ps % 2 else 256, ps, dt, seed=ps), odt)


@pytest.mark.parametrize("dt,odt", KINDS)
@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 511, 513])
def test_lengths(dt, odt, n):
    """A prompt of n tokens, and n tokens behind others, on either side of the tiles' and units' borders."""
    check(R.Batch([n, n], [n, n + 128], 2, 1, 64, 16, dt, seed=n), odt)
    check(R.Batch([1, n], [n, 2 * n + 127], 8, 1, 256, 16, dt, seed=n), odt)


@pytest.mark.parametrize("dt,odt", [(BF, BF), (F32, F32), (BF, F32)])
@pytest.mark.parametrize("layout", ["thd", "htd", "both"])
@pytest.mark.parametrize("wide", [False, True])
def test_layouts(dt, odt, layout, wide):
    check(R.Batch([50, 90], [77, 290], 6, 2, 128, 16, dt, layout, gate=True, pad=1, seed=3, wide=wide), odt)


@pytest.mark.parametrize("dt,odt", KINDS)
def test_rows_without_keys(dt, odt):
    """Sequences shorter than their rows (the first rows see nothing), empty ones, ones without rows."""
    b = R.Batch([40, 300, 10, 0, 7], [25, 3, 0, 99, 7], 8, 2, 64, 16, dt, gate=True, seed=1)
    out = check(b, odt)
    assert torch.all(out[:15] == 0) and torch.all(out[40:337] == 0) and torch.all(out[340:350] == 0)


@pytest.mark.parametrize("dt,odt", KINDS)
@pytest.mark.parametrize("fill", [math.nan, math.inf, -math.inf, 3e38])
def test_what_no_sequence_has_does_not_matter(dt, odt, fill):
    b = R.Batch([37, 1, 150, 2], [37, 100, 400, 9], 8, 2, 128, 16, dt, seed=2, fill=fill)
    clean = R.Batch([37, 1, 150, 2], [37, 100, 400, 9], 8, 2, 128, 16, dt, seed=2)
    assert torch.equal(check(b, odt), run(clean, odt))


@pytest.mark.parametrize("dt,odt", KINDS)
@pytest.mark.parametrize("d,G", [(256, 8), (64, 1), (128, 5)])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_infinite_and_nan_tokens_reach_only_the_rows_that_see_them(dt, odt, d, G, bad):
    """Values: a channel of the rows that see them becomes infinite or NaN; keys: the rows; nothing else changes."""
    b = R.Batch([200, 60], [260, 60], 2 * G, 2, d, 16, dt, seed=5)
    clean = run(b, odt).clone()
    slot = lambda s, j: (int(b.table[s, j // 16]), j % 16)
    spots = [(0, 59 + 1 + 130, 0, 3), (0, 259, 1, d - 1), (0, 10, 0, 7), (1, 31, 1, 0)]   # sequence, key, kv head, channel
    for s, j, h, c in spots:
        b.v[slot(s, j)][h, c] = bad
    got = run(b, odt).view(-1, 2 * G, d)
    hit = torch.zeros_like(got, dtype=torch.bool)
    for s, j, h, c in spots:
        first = int(b.cu[s]) + max(0, j - (b.len_list[s] - b.new[s]))
        hit[first:int(b.cu[s + 1]), h * G:(h + 1) * G, c] = True
    assert torch.all(~torch.isfinite(got[hit]))
    same = (got == clean.view(-1, 2 * G, d)) | hit
    assert torch.all(same), torch.argwhere(~same)[:5].tolist()
    for s, j, h, c in spots:
        b.v[slot(s, j)][h, c] = 0.5
    base = run(b, odt).clone().view(-1, 2 * G, d)
    b.k[slot(0, 60 + 77)][1, 2] = bad
    got = run(b, odt).view(-1, 2 * G, d)
    untouched = torch.ones_like(got, dtype=torch.bool)
    untouched[77:200, G:] = False
    assert torch.equal(got[untouched], base[untouched]) and torch.all(torch.isfinite(base))
    if math.isnan(bad):
        assert torch.all(torch.isnan(got[77:200, G:]))


@pytest.mark.parametrize("dt,odt", KINDS)
def test_pages_outside_the_cache(dt, odt):
    b = R.Batch([100, 20], [300, 150], 8, 2, 64, 16, dt, seed=4)
    b.table[0, 2], b.table[0, 17], b.table[1, 3] = 10 ** 8, -1, b.k.shape[0]
    check(b, odt, absent=(10 ** 8, -1, b.k.shape[0]), status=64)


@pytest.mark.parametrize("dt,odt", [(BF, BF), (F32, F32)])
def test_lengths_and_rows_outside(dt, odt):
    """A length past the table counts as the table; rows outside 0..T or falling ones are no rows."""
    b = R.Batch([30, 10, 5], [64, 80, 40], 4, 2, 64, 16, dt, seed=6)
    b.table = b.table[:, :4].contiguous()
    b.lens[1], b.len_list[1] = 1000, 64
    check(b, odt, status=[0, 64, 0])
    b = R.Batch([30, 10, 5], [64, 80, 40], 4, 2, 64, 16, dt, seed=6)
    good = run(b, odt).clone()
    for cu, kept in [([0, 30, 40, 46], 40), ([-1, 30, 40, 45], None), ([0, 30, 29, 45], None), ([0, 2 ** 31 - 1, -2 ** 31, 3], None)]:
        b.cu = torch.tensor(cu, dtype=torch.int32, device="cuda")
        st = torch.zeros(3, dtype=torch.int32, device="cuda")
        out = run(b, odt, status=st)
        bad = [i for i in range(3) if not 0 <= cu[i] <= cu[i + 1] <= b.T]
        assert st.tolist() == [64 if i in bad else 0 for i in range(3)]
        if kept:
            assert torch.equal(out[:kept], good[:kept]) and torch.all(out[kept:] == 7.0)


@pytest.mark.parametrize("dt,odt", KINDS)
@pytest.mark.parametrize("new,lens", [([3], [9000]), ([1, 1, 1], [5000, 1, 2500]), ([300], [6000]), ([1] * 40, [257] * 40)])
def test_long_and_split(dt, odt, new, lens):
    """Few rows over many keys: parts of one unit in many workers, joined."""
    check(R.Batch(new, lens, 8, 1, 64, 16, dt, seed=7), odt)
    check(R.Batch(new, lens, 4, 1, 256, 64, dt, seed=8), odt)


@pytest.mark.parametrize("dt,odt", [(BF, BF), (BF, F32)])
@pytest.mark.parametrize("d,G,Hkv,new,lens", [(128, 8, 16, [600, 350], [700, 3000]), (64, 8, 16, [900], [1100]), (256, 6, 8, [500, 260], [500, 1500]),
                                              (128, 3, 24, [700, 90, 1], [700, 2500, 4000])])
def test_many_parts_and_tiles_a_worker(dt, odt, d, G, Hkv, new, lens):
    """Workers with several units one after another, of one tile to dozens of tiles."""
    check(R.Batch(new, lens, G * Hkv, Hkv, d, 16, dt, seed=21), odt)


@pytest.mark.parametrize("dt,odt", KINDS)
@pytest.mark.parametrize("rise", [0.02, -0.02])
def test_scores_that_rise_along_the_sequence(dt, odt, rise):
    """The running maximum is raised in most tiles (or set by the first)."""
    b = R.Batch([90], [1200], 2, 1, 64, 16, dt, seed=9)
    step = torch.zeros_like(b.k)
    for j in range(1200):
        step[int(b.table[0, j // 16]), j % 16, :, 0] = j * rise
    b.k = (b.k.float() * 0.3 + step.float()).to(dt)
    b.q = b.q.clone()
    b.q[:, 0] = 8.0
    b.q[:, 64] = 8.0
    check(b, odt, tight=2e-5)   # scores of up to 24 units: their own rounding, 24 * 2^-24 * sqrt(64)


@pytest.mark.parametrize("dt,odt", KINDS)
@pytest.mark.parametrize("scale", [0.0, -0.1, 0.7])
def test_scales(dt, odt, scale):
    check(R.Batch([40, 9], [140, 9], 4, 2, 64, 16, dt, seed=10), odt, scale=scale, tight=1e-5)


@pytest.mark.parametrize("dt,odt", KINDS)
def test_infinite_gate_and_large_values(dt, odt):
    """Gates of +-inf are 1 and 0; large values do not overflow on the way."""
    b = R.Batch([20], [50], 2, 1, 64, 16, dt, gate=True, seed=11)
    b.gate[:, 0], b.gate[:, 1] = math.inf, -math.inf
    b.v = (b.v.float().clamp(-1, 1) * 2.0 ** 110).to(dt)
    out = check(b, odt)
    assert torch.all(out[:, 1] == 0)


def test_agrees_with_decode_on_single_tokens():
    """One token of each sequence: what gdn_attn_decode gives, up to the weights' rounding."""
    b = R.Batch([1] * 9, [1, 5, 17, 100, 300, 64, 65, 128, 1000], 16, 2, 256, 16, seed=12, gate=True)
    dims = gdn.make_attn_dims(16, 2, 256, BF, F32)
    ws = torch.zeros(gdn.gdn_attn_decode_workspace_bytes(dims, 9, 1), dtype=torch.uint8, device="cuda")
    one = torch.empty(9, 16 * 256, device="cuda")
    gdn.gdn_attn_decode(dims, gdn.KvCache(b.k, b.v), 1, b.q, b.table, b.lens, one, gate=b.gate, workspace=ws)
    assert float((run(b, F32) - one).norm() / one.norm()) < 2e-6
    assert float((run(b, BF).float() - one).norm() / one.norm()) < 2.0 ** -8


def test_many_sequences():
    """More sequences than threads, most with nothing to do."""
    rng = np.random.default_rng(0)
    new = [int(x) for x in rng.choice([0, 0, 0, 1, 2, 9], 3000)]
    lens = [n + int(x) for n, x in zip(new, rng.integers(0, 30, 3000))]
    check(R.Batch(new, lens, 2, 1, 64, 16, seed=13), BF)
    check(R.Batch([0] * 2999 + [5], [3] * 2999 + [40], 2, 1, 64, 16, F32, seed=13), F32)


def test_no_rows():
    b = R.Batch([0, 0], [5, 0], 2, 1, 64, 16, pad=4, seed=14)
    assert torch.all(run(b, BF) == 7.0)
    e = torch.empty(0, 128, device="cuda", dtype=BF)
    dims = gdn.make_attn_dims(2, 1, 64, BF, BF)
    gdn.gdn_attn_chunk(dims, gdn.KvCache(b.k, b.v), e, b.cu, b.table, b.lens, e, workspace=workspace(dims))


@pytest.mark.parametrize("dt,odt", KINDS)
def test_offsets_past_31_bits(dt, odt):
    """A cache whose last pages lie more than 2^31 elements from its start."""
    pages, ps, H, d = (1 << 31) // (16 * 2 * 256) + 40, 16, 2, 256
    k = torch.empty(pages, ps, H, d, dtype=dt, device="cuda")
    v = torch.empty_like(k)
    b = R.Batch([30], [100], 4, H, d, ps, dt, seed=15)
    n = b.k.shape[0]
    k[-n:], v[-n:] = b.k, b.v
    want = run(b, odt)
    b.k, b.v = k, v
    b.table = b.table + (pages - n)
    assert torch.equal(run(b, odt), want)


@pytest.mark.parametrize("dt,odt", KINDS)
def test_captured_and_replayed_beside_another_stream(dt, odt):
    """Two graphs with a workspace each, replayed at the same time on two streams, with new inputs in place."""
    bs = [R.Batch([150, 4], [400, 900], 8, 2, 128, 16, dt, seed=s) for s in (1, 2)]
    outs, graphs, streams = [], [], [torch.cuda.Stream() for _ in bs]
    for b, s in zip(bs, streams):
        dims = gdn.make_attn_dims(b.Hq, b.Hkv, b.d, b.dt, odt)
        ws = torch.zeros(gdn.gdn_attn_chunk_workspace_bytes(dims, 2, b.T), dtype=torch.uint8, device="cuda")
        out = torch.empty(b.T, b.Hq * b.d, dtype=odt, device="cuda")
        run(b, odt, out=out, ws=ws)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            run(b, odt, out=out, ws=ws)
        outs.append((out, ws))
        graphs.append(graph)
    for round_ in range(3):
        for b in bs:
            b.q.mul_(0.9)
        torch.cuda.synchronize()
        for _ in range(4):
            for g, s in zip(graphs, streams):
                with torch.cuda.stream(s):
                    g.replay()
        torch.cuda.synchronize()
        for b, (out, _) in zip(bs, outs):
            assert torch.equal(out, run(b, odt))


def test_a_prompt_as_it_would_be_run():
    """Pages, append, attention of the prompt in two pieces, a fork with its copies, a token of each, a release: every
    attention equal to the definition over what was appended."""
    B, Hq, Hkv, d, ps = 4, 8, 2, 128, 16
    g = torch.Generator(device="cuda").manual_seed(0)
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")
    dims = gdn.make_attn_dims(Hq, Hkv, d, BF, BF)
    N = 64
    k, v = (torch.full((N, ps, Hkv, d), math.nan, dtype=BF, device="cuda") for _ in range(2))
    kv, table = gdn.KvCache(k, v), torch.full((B, 16), -1, dtype=torch.int32, device="cuda")
    lens, held, free, nf = i32(0, 0, 0, 0), i32(0, 0, 0, 0), torch.arange(N, dtype=torch.int32, device="cuda"), i32(N)
    refs, st, ws = torch.zeros(N, dtype=torch.int32, device="cuda"), i32(0, 0, 0, 0), workspace(dims)
    keys, vals = [[] for _ in range(B)], [[] for _ in range(B)]

    def step(new):
        T = sum(new) + 3
        q, kx, vx = (torch.randn(T, h * d, generator=g, device="cuda").to(BF) for h in (Hq, Hkv, Hkv))
        slots, pos, cu = (torch.empty(n, dtype=torch.int32, device="cuda") for n in (T, T, B + 1))
        gdn.gdn_kv_extend(ps, i32(*new), lens, held, table, free, nf, slots, pos, cu, dev_status=st)
        qo, out = torch.empty_like(q), torch.zeros(T, Hq * d, dtype=BF, device="cuda")
        gdn.gdn_kv_append(dims, kv, q, kx, vx, pos, slots, qo)
        gdn.gdn_attn_chunk(dims, kv, qo, cu, table, lens, out, workspace=ws, dev_status=st)
        at, c = 0, cu.tolist()
        for b, n in enumerate(new):
            keys[b] += list(kx[at:at + n].view(n, Hkv, d).cpu())
            vals[b] += list(vx[at:at + n].view(n, Hkv, d).cpu())
            at += n
        for b, n in enumerate(new):
            if n == 0:
                continue
            x = R.Batch([n], [len(keys[b])], Hq, Hkv, d, 4096, seed=0)
            x.k, x.v = torch.stack(keys[b])[None], torch.stack(vals[b])[None]
            x.ps, x.q, x.table = len(keys[b]), qo[c[b]:c[b + 1]].cpu(), torch.zeros(1, 2, dtype=torch.int32)
            want, size = x.want()
            err = np.abs(out[c[b]:c[b + 1]].double().cpu().numpy() - want)
            assert np.all(err <= R.bound(want, size, x, BF)), (b, n)

    step([100, 37, 0, 0])
    step([60, 1, 0, 0])
    cs, cd, fst = i32(0, 0), i32(0, 0), i32(0, 0)
    gdn.gdn_kv_fork(ps, i32(0, 1), i32(2, 3), i32(150, 38), lens, held, table, refs, free, nf, cs, cd, dev_status=fst)
    gdn.gdn_kv_copy_pages(dims, kv, cs, cd)
    keys[2], vals[2], keys[3], vals[3] = keys[0][:150], vals[0][:150], list(keys[1]), list(vals[1])
    step([1, 1, 1, 1])
    step([0, 3, 40, 1])
    rs, rd = i32(0, 0, 0, 0), i32(0, 0, 0, 0)
    gdn.gdn_kv_release(ps, i32(70, 0, 141, 20), lens, held, table, refs, free, nf, rs, rd, dev_status=st)
    gdn.gdn_kv_copy_pages(dims, kv, rs, rd)
    for b, n in enumerate((70, 0, 141, 20)):
        keys[b], vals[b] = keys[b][:n], vals[b][:n]
    assert rd.tolist()[0] >= 0   # its kept page is another's too
    page_map, ms, md, nm = (torch.empty(n, dtype=torch.int32, device="cuda") for n in (N, N, N, 1))
    gdn.gdn_kv_compact(held, table, refs, free, nf, page_map, ms, md, nm, dev_status=st)
    gdn.gdn_kv_copy_pages(dims, kv, ms, md)
    step([5, 20, 1, 2])
    assert st.tolist() == [0] * 4 and fst.tolist() == [0, 0]


@pytest.mark.parametrize("dt,odt", [(BF, BF), (BF, F32), (F32, F32)])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_units_of_dozens_of_parts(dt, odt, d):
    """Many rows over a long sequence: more parts of a unit than are joined at a time."""
    check(R.Batch([70], [20000], 4, 1, d, 16, dt, gate=True, seed=d), odt)
    check(R.Batch([3, 33], [4000, 9000], 8, 1, d, 64, dt, seed=d + 1), odt)


@pytest.mark.parametrize("dt,odt", [(BF, BF), (BF, F32)])
@pytest.mark.parametrize("order,pad", [((0, 1, 2, 3), 3), ((0, 2, 1, 3), 5), ((1, 0, 2, 3), 0), ((2, 0, 1, 3), 0), ((1, 2, 0, 3), 0), ((2, 1, 0, 3), 1)])
@pytest.mark.parametrize("d,ps", [(64, 16), (128, 24), (256, 6), (256, 8)])
def test_orders_of_the_cache(dt, odt, order, pad, d, ps):
    """Pages, tokens and heads in any order in memory, with room between."""
    b = R.Batch([90, 5], [200, 301], 6, 3, d, ps, dt, seed=31)
    want = run(b, odt)

    def laid(t):
        shape = [t.shape[i] for i in order]
        shape[1] += pad
        back = torch.empty(shape, dtype=dt, device="cuda").fill_(math.nan)
        view = back.permute([order.index(i) for i in range(4)])
        for i in range(3):
            view = view.narrow(i, 0, t.shape[i])
        view.copy_(t)
        return view

    b.k, b.v = laid(b.k), laid(b.v)
    assert torch.equal(run(b, odt), want)


@pytest.mark.parametrize("odt", [BF, F32])
@pytest.mark.parametrize("new,lens", [([40, 300], [500, 700]), ([3], [9000]), ([64], [9000])])
def test_a_wait_that_gives_up(odt, new, lens):
    """GDN_FLAG_TEST_STALL: the kernel ends, says so, and writes no result; with a workspace of zeros the next call is as ever."""
    b = R.Batch(new, lens, 8, 1, 128, 16, seed=41)
    want, st = run(b, odt), torch.zeros(len(new), dtype=torch.int32, device="cuda")
    ws = torch.zeros_like(workspace(gdn.make_attn_dims(8, 1, 128, BF, odt)))
    out = run(b, odt, status=st, ws=ws, test_stall=True)
    assert st.tolist() == [16] * len(new) and torch.all(out == 7.0)
    ws.zero_()
    st.zero_()
    assert torch.equal(run(b, odt, status=st, ws=ws), want) and not st.any()


@pytest.mark.parametrize("dt,odt", KINDS)
@pytest.mark.parametrize("d", [64, 256])
def test_buffers_on_16_bytes_only(dt, odt, d):
    """A workspace, a result, queries and gates that begin 16 bytes past a multiple of 32; nothing is written outside."""
    b = R.Batch([70, 3], [9000, 200], 4, 1, d, 16, dt, gate=True, seed=51)
    want = run(b, odt)
    dims = gdn.make_attn_dims(4, 1, d, dt, odt)
    need = gdn.gdn_attn_chunk_workspace_bytes(dims, 2, b.T)
    room = torch.full((need + 4096,), 0x5a, dtype=torch.uint8, device="cuda")
    ws = room[16:16 + need].zero_()

    def moved(t):
        n = 16 // t.element_size()
        x = torch.zeros(t.numel() + n, dtype=t.dtype, device="cuda")[n:].view(t.shape)
        return x.copy_(t)

    b.q, b.gate = moved(b.q), moved(b.gate)
    n = 16 // want.element_size()
    back = torch.full((want.numel() + 2 * n,), 7.0, dtype=odt, device="cuda")
    out = back[n:-n].view(want.shape)
    for t in (ws, b.q, b.gate, out):
        assert t.data_ptr() % 32 == 16
    for _ in range(2):
        run(b, odt, out=out, ws=ws)
        assert torch.equal(out, want)
    assert torch.all(room[:16] == 0x5a) and torch.all(room[16 + need:] == 0x5a)
    assert torch.all(back[:n] == 7.0) and torch.all(back[-n:] == 7.0)


def test_two_dtypes_share_a_workspace_in_turn():
    """A workspace that is large enough serves calls of any dims one after another."""
    a, b = R.Batch([70, 3], [9000, 200], 4, 1, 256, 16, BF, seed=52), R.Batch([40], [3000], 6, 3, 64, 11, F32, seed=53)
    kinds = [(a, BF), (b, F32), (a, F32), (b, F32), (a, BF)]
    need = max(gdn.gdn_attn_chunk_workspace_bytes(gdn.make_attn_dims(x.Hq, x.Hkv, x.d, x.dt, o), 1, 1) for x, o in kinds)
    ws = torch.zeros(need, dtype=torch.uint8, device="cuda")
    for x, o in kinds:
        assert torch.equal(run(x, o, ws=ws), run(x, o))
