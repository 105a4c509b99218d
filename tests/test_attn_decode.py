"""GPU parity of gdn_attn_decode with the 64-bit definition.

Inputs are exact in both.  An fp32 output has the accuracy contract of fp32 results, 1e-5, relative to the
largest value (an output is a weighted mean of values); a bf16 output may be half a bf16 ulp off, plus 2^-16 of
the largest value for weights held as two bf16 parts.  Everything the call must not read -- the rest of a
sequence's last page, the pages of nobody -- is NaN."""
import numpy as np
import pytest
import torch

import gated_deltanet_linear_decode_gb300 as gdn
from tests import attn_ref as R
from tests import gpu_util as G

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


class Case:
    def __init__(self, lens, K, Hq, Hkv, d, ps, dtype, seed=0, layout="thd", spare=2, gate=True, width=0, qscale=1.5):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.K, self.Hq, self.Hkv, self.d, self.ps, self.dtype = lens, K, Hq, Hkv, d, ps, dtype
        B, held = len(lens), [-(-n // ps) for n in lens]
        n = sum(held) + spare
        perm = torch.randperm(n, generator=g)
        P = max(1, max(held), width)
        # entries past the pages held mean nothing: they point nowhere
        self.table = torch.full((B, P), -7, dtype=torch.int32)
        kv = torch.full((2, n, ps, Hkv, d), float("nan"))
        at = 0
        for b, h in enumerate(held):
            self.table[b, :h] = perm[at:at + h].to(torch.int32)
            for i in range(h):
                m = min(ps, lens[b] - i * ps)
                kv[:, perm[at + i], :m] = torch.randn(2, m, Hkv, d, generator=g)
            at += h
        kv = kv.to(dtype).cuda()
        if layout == "htd":       # [page][head][token][channel] in memory
            kv = kv.transpose(2, 3).contiguous().transpose(2, 3)
        elif layout == "pair":    # [page][2][token][head][channel]: both halves in one buffer
            kv = kv.transpose(0, 1).contiguous().transpose(0, 1)
        elif layout == "pth":     # [token][page][head][channel]
            kv = kv.transpose(1, 2).contiguous().transpose(1, 2)
        self.k, self.v = kv[0], kv[1]
        T = B * K
        self.q = (qscale * torch.randn(T, Hq * d, generator=g)).to(dtype).cuda()
        self.gate = torch.randn(T, Hq * d, generator=g).to(dtype).cuda() if gate else None
        self.seq_len = torch.tensor(lens, dtype=torch.int32).cuda()

    def ref(self, absent=()):
        v = R.f64(self.v)
        return R.attn(R.f64(self.q), np.nan_to_num(R.f64(self.k)), np.nan_to_num(v), self.table.numpy(), self.lens, self.K, self.Hq,
                      self.Hkv, self.d, None if self.gate is None else R.f64(self.gate), absent=absent)

    def run(self, out_dtype, ws=None, table=None, status=None, stream=None, q=None, gate="own", out=None):
        d = gdn.make_attn_dims(self.Hq, self.Hkv, self.d, self.dtype, out_dtype)
        n = gdn.gdn_attn_decode_workspace_bytes(d, len(self.lens), self.K)
        ws = torch.zeros(n, dtype=torch.uint8, device="cuda") if ws is None else ws
        if out is None:
            out = torch.full((len(self.lens) * self.K, self.Hq * self.d), float("nan"), dtype=out_dtype, device="cuda")
        gdn.gdn_attn_decode(d, gdn.KvCache(self.k, self.v), self.K, self.q if q is None else q,
                            (self.table if table is None else table).cuda(), self.seq_len, out,
                            gate=self.gate if isinstance(gate, str) else gate, workspace=ws, dev_status=status,
                            stream=stream)
        return out

    def close(self, out, ref=None):
        ref = self.ref() if ref is None else ref
        big = float(np.nanmax(np.abs(np.where(np.isnan(R.f64(self.v)), 0, R.f64(self.v)))))
        got = R.f64(out)
        assert np.isfinite(got).all()
        bound = 1e-5 * big if out.dtype == F32 else G.half_ulp_bf16(ref) + 2.0 ** -16 * big
        err = np.abs(got - ref)
        assert (err <= bound).all(), f"worst excess {float((err - bound).max()):.3e} of {big:.2f}"


SHAPES = [
    # lens, K, Hq, Hkv, d, ps
    ([1], 1, 1, 1, 64, 1),
    ([777], 1, 16, 2, 256, 16),
    ([0, 1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 1000], 1, 6, 3, 64, 16),
    ([5, 0, 333, 31], 1, 24, 4, 256, 16),
    ([130, 1, 0, 700], 1, 16, 1, 128, 7),          # 16 query heads on one kv head
    ([257, 64], 1, 5, 5, 128, 64),                 # a kv head each
    ([2, 0, 1, 3, 4, 100, 513], 4, 8, 2, 128, 16),   # lengths under K: rows that see nothing
    ([95, 1, 400], 3, 16, 2, 256, 16),
    ([16, 15, 300, 90], 16, 16, 1, 64, 10),        # 256 rows a kv head
    ([40, 1000], 16, 16, 2, 256, 100),             # 128 rows a kv head
    ([33, 70], 7, 9, 3, 128, 33),
    ([12000], 1, 8, 1, 128, 48),                   # one long sequence
    ([7001, 3, 2900], 2, 12, 2, 64, 256),
    ([200] * 40, 1, 4, 2, 64, 16),
    ([5000] + [0] * 300 + [9], 1, 2, 2, 64, 16),   # many idle slots
    ([3] * 700, 2, 2, 1, 64, 5),                   # many short ones
]


@pytest.mark.parametrize("dtype,out_dtype", [(BF, BF), (BF, F32), (F32, F32), (F32, BF)])
@pytest.mark.parametrize("i", range(len(SHAPES)))
def test_against_the_definition(i, dtype, out_dtype):
    lens, K, Hq, Hkv, d, ps = SHAPES[i]
    c = Case(lens, K, Hq, Hkv, d, ps, dtype, seed=300 + i, gate=i % 2 == 0)
    c.close(c.run(out_dtype))


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("K,G_", [(1, 1), (2, 1), (1, 3), (2, 2), (1, 5), (3, 2), (2, 4), (3, 3), (1, 16)])
def test_few_rows_in_fp32(K, G_, d):
    """Every number of rows a warp may hold or leave empty: a group of many parts, one of one, one without keys."""
    c = Case([9000, 0, 1, 31, 2500], K, 2 * G_, 2, d, 11, F32, seed=K * 100 + G_ * 10 + d)
    c.close(c.run(F32))


@pytest.mark.parametrize("layout", ["htd", "pair", "pth"])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_cache_layouts(layout, dtype):
    c = Case([100, 1, 37, 222], 2, 6, 2, 128, 12, dtype, seed=41, layout=layout)
    c.close(c.run(F32))


def test_rows_without_keys_are_zero():
    c = Case([2, 0, 1], 4, 4, 2, 64, 16, BF, seed=5)
    out = R.f64(c.run(BF)).reshape(3, 4, -1)
    assert (out[0, :2] == 0).all() and (out[1] == 0).all() and (out[2, :3] == 0).all()
    assert (out[0, 2:] != 0).any() and (out[2, 3] != 0).any()


@pytest.mark.parametrize("qscale", [30.0, 300.0])
def test_large_scores(qscale):
    """Scores of hundreds to thousands: one key takes nearly all the weight; nothing overflows.  An error of
    2^-20 of a score (products of exact values summed in 32 bits over 128 channels) moves a weight by as much."""
    c = Case([500, 64, 1], 2, 8, 2, 128, 16, BF, seed=6, gate=False, qscale=qscale)
    ref = c.ref()
    got = R.f64(c.run(F32))
    big = float(np.nanmax(np.abs(np.nan_to_num(R.f64(c.v)))))
    s = qscale * np.sqrt(128.0) / np.sqrt(128.0) * 6 * 3   # a bound on |score|: 6 sigma of q.k / sqrt(d), 3 spare
    assert np.isfinite(got).all() and np.abs(got - ref).max() <= 2 * s * 2.0 ** -20 * big


def test_minus_infinity_in_a_seen_key():
    """A score of minus infinity (an infinite key) takes no weight, also when it is the first one."""
    c = Case([70], 1, 2, 1, 64, 16, F32, seed=7, gate=False)
    c.q.abs_()
    for j in (0, 33):
        c.k[int(c.table[0, j // 16]), j % 16] = float("-inf")
    kk = np.nan_to_num(R.f64(c.k), neginf=-1e300)
    ref = R.attn(R.f64(c.q), kk, np.nan_to_num(R.f64(c.v)), c.table.numpy(), c.lens, 1, 2, 1, 64)
    c.close(c.run(F32), ref)


def test_pitched_rows():
    """q and gate as column slices of one wider projection row."""
    c = Case([100, 9, 64], 2, 4, 2, 64, 16, BF, seed=8)
    wide = torch.randn(6, 2 * 256 + 64, device="cuda").to(BF)
    wide[:, :256], wide[:, 256:512] = c.q, c.gate
    c.close(c.run(BF, q=wide[:, :256], gate=wide[:, 256:512]))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_bad_indices_are_left_out_and_reported(dtype):
    c = Case([64, 200, 30, 40], 1, 4, 2, 64, 16, dtype, seed=9, gate=False)
    table = c.table.clone()
    ref_table = table.clone()
    table[1, 3], table[1, 7], table[3, 0] = -1, c.k.shape[0], 2 ** 31 - 1
    ref_table[1, 3] = ref_table[1, 7] = ref_table[3, 0] = c.k.shape[0] - 1   # a page of nobody
    st = torch.zeros(4, dtype=torch.int32, device="cuda")
    out = c.run(F32, table=table, status=st)
    keep, c.table = c.table, ref_table
    c.close(out, c.ref(absent=[c.k.shape[0] - 1]))
    c.table = keep
    assert st.tolist() == [0, 64, 0, 64]
    # a length past the table is taken as the table's; a negative one as none
    c.seq_len = torch.tensor([64, 13 * 16 + 1, -5, 40], dtype=torch.int32, device="cuda")
    st.zero_()
    out = c.run(F32, status=st)
    assert st.tolist()[0] == 0 and st.tolist()[2:] == [0, 0] and st.tolist()[1] == 64
    assert (out[2] == 0).all()


def test_workspace_is_reused_across_shapes_and_results_repeat():
    """One workspace, zeroed once, serves calls of different shapes in any order; the same call gives the same bits."""
    a = Case([3000, 17, 0, 900], 1, 8, 2, 128, 16, BF, seed=10)
    b = Case([50, 4000], 16, 16, 2, 64, 16, F32, seed=11)
    e = Case([20000], 1, 2, 1, 64, 64, BF, seed=12)
    n = max(gdn.gdn_attn_decode_workspace_bytes(gdn.make_attn_dims(c.Hq, c.Hkv, c.d, c.dtype, F32), len(c.lens), c.K) for c in (a, b, e))
    ws = torch.zeros(max(n, 16), dtype=torch.uint8, device="cuda")
    first = [c.run(F32, ws=ws) for c in (a, b, e)]
    for c, o in zip((a, b, e), first):
        c.close(o)
    for c, o in [(e, first[2]), (a, first[0]), (a, first[0]), (b, first[1]), (e, first[2])]:
        assert torch.equal(c.run(F32, ws=ws), o)


def test_another_stream():
    c = Case([300, 20], 1, 8, 2, 128, 16, BF, seed=13)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        out = c.run(F32)
    s.synchronize()
    c.close(out)
    out = c.run(F32, stream=s)
    torch.cuda.synchronize()
    c.close(out)


def test_offsets_past_32_bits():
    """A cache half of 2^31 elements and more: the last pages lie past what 32 bits address."""
    ps, Hkv, d = 64, 4, 256
    pages = (1 << 31) // (ps * Hkv * d) + 40
    k = torch.empty(pages, ps, Hkv, d, dtype=BF, device="cuda")
    v = torch.empty(pages, ps, Hkv, d, dtype=BF, device="cuda")
    c = Case([200, 130], 1, 8, Hkv, d, ps, BF, seed=14)
    at = torch.arange(pages - c.k.shape[0], pages, device="cuda")
    k[at], v[at] = c.k, c.v
    table = torch.where(c.table >= 0, c.table + pages - c.k.shape[0], c.table)
    ref = c.ref()
    small = (c.k, c.v)
    c.k, c.v = k, v
    out = c.run(F32, table=table)
    c.k, c.v = small
    c.close(out, ref)


def test_graph_replay_follows_the_lengths():
    """Lengths and tables are read on the device: one captured call serves them as they change."""
    c = Case([90, 300], 1, 8, 2, 128, 16, BF, seed=15)
    d = gdn.make_attn_dims(c.Hq, c.Hkv, c.d, BF, F32)
    ws = torch.zeros(gdn.gdn_attn_decode_workspace_bytes(d, 2, 1), dtype=torch.uint8, device="cuda")
    out, table, cache = torch.empty(2, c.Hq * c.d, device="cuda"), c.table.cuda(), gdn.KvCache(c.k, c.v)
    g = torch.cuda.CUDAGraph()
    gdn.gdn_attn_decode(d, cache, 1, c.q, table, c.seq_len, out, gate=c.gate, workspace=ws)
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        gdn.gdn_attn_decode(d, cache, 1, c.q, table, c.seq_len, out, gate=c.gate, workspace=ws)
    for lens in ([90, 300], [1, 299], [0, 17], [64, 128]):
        c.lens = lens
        c.seq_len.copy_(torch.tensor(lens, dtype=torch.int32))
        g.replay()
        torch.cuda.synchronize()
        c.close(out)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_a_wait_that_gives_up_writes_nothing(dtype):
    """GDN_FLAG_TEST_STALL: the computing warps first wait on a barrier that nothing arrives on.  Every sequence
    reports bit 4, no output byte changes, and with a zeroed workspace the next call is right."""
    c = Case([300, 0, 40, 4000, 17], 2, 8, 2, 128, 16, dtype, seed=16)
    d = gdn.make_attn_dims(c.Hq, c.Hkv, c.d, dtype, F32, test_stall=True)
    ws = torch.zeros(gdn.gdn_attn_decode_workspace_bytes(d, 5, 2), dtype=torch.uint8, device="cuda")
    out = torch.full((10, c.Hq * c.d), 7.0, device="cuda")
    st = torch.zeros(5, dtype=torch.int32, device="cuda")
    gdn.gdn_attn_decode(d, gdn.KvCache(c.k, c.v), 2, c.q, c.table.cuda(), c.seq_len, out, gate=c.gate, workspace=ws,
                        dev_status=st)
    torch.cuda.synchronize()
    assert st.tolist() == [16] * 5 and (out == 7.0).all()
    ws.zero_()
    c.close(c.run(F32, ws=ws))


@pytest.mark.parametrize("out_dtype", [BF, F32])
@pytest.mark.parametrize("d,Hq,K", [(256, 8, 10), (64, 16, 16), (128, 12, 16)])
def test_many_rows_give_up_and_repeat(d, Hq, K, out_dtype):
    """The same for more than 32 rows a kv head, and such calls give the same bits each time, also split over many CTAs."""
    c = Case([300, 0, 40, 9000, 17], K, Hq, 2, d, 16, BF, seed=17)
    st = torch.zeros(5, dtype=torch.int32, device="cuda")
    dims = gdn.make_attn_dims(Hq, 2, d, BF, out_dtype, test_stall=True)
    n = gdn.gdn_attn_decode_workspace_bytes(dims, 5, K)
    ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
    out = torch.full((5 * K, Hq * d), 7.0, dtype=out_dtype, device="cuda")
    gdn.gdn_attn_decode(dims, gdn.KvCache(c.k, c.v), K, c.q, c.table.cuda(), c.seq_len, out, gate=c.gate, workspace=ws,
                        dev_status=st)
    torch.cuda.synchronize()
    assert st.tolist() == [16] * 5 and (out == 7.0).all()
    ws.zero_()
    first = c.run(out_dtype, ws=ws)
    c.close(first)
    for _ in range(5):
        assert torch.equal(c.run(out_dtype, ws=ws), first)


@pytest.mark.parametrize("dtype,Hq,K", [(BF, 8, 1), (BF, 8, 2), (BF, 8, 3), (BF, 8, 8), (F32, 8, 1)])
def test_long_sums_keep_their_bits(dtype, Hq, K):
    """Sequences that one SM walks by itself (more of them than SMs, all on the same pages): values of one sign, so that
    a sum that always rounds one way would drift by 2^-25 a step; the fp32 contract holds all the same."""
    n, ps, d, B = 16000, 16, 64, 160
    c = Case([n], K, Hq, 1, d, ps, dtype, seed=18, gate=False)
    c.v.abs_()
    g = torch.Generator().manual_seed(19)
    q = torch.randn(B * K, Hq * d, generator=g).to(dtype).cuda()
    dims = gdn.make_attn_dims(Hq, 1, d, dtype, F32)
    ws = torch.zeros(gdn.gdn_attn_decode_workspace_bytes(dims, B, K), dtype=torch.uint8, device="cuda")
    out = torch.empty(B * K, Hq * d, device="cuda")
    gdn.gdn_attn_decode(dims, gdn.KvCache(c.k, c.v), K, q, c.table.repeat(B, 1).cuda(), torch.full((B,), n, dtype=torch.int32, device="cuda"),
                        out, workspace=ws)
    k, v = R.f64(c.k), R.f64(c.v)
    for b in (0, 77, B - 1):
        rows = slice(b * K, b * K + K)
        ref = R.attn(R.f64(q[rows]), k, v, c.table.numpy(), [n], K, Hq, 1, d)
        assert np.abs(R.f64(out[rows]) - ref).max() <= 1e-5 * np.nanmax(np.abs(v))
