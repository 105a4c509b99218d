"""examples/hybrid_decode.py: the two layers run together, its graph replays give the eager steps' bits, and the
attention layer's output of the last step is the 64-bit definition's on the cache as it stands."""
import importlib.util
import os

import numpy as np
import pytest
import torch

from tests import attn_ref as R
from tests import gpu_util as G

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def example():
    spec = importlib.util.spec_from_file_location("hybrid_decode", os.path.join(ROOT, "examples", "hybrid_decode.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def check_attention(m):
    """The last step's attention: bf16 output, half a bf16 ulp and 2^-16 of the largest value (as in test_attn_decode)."""
    k, v = R.f64(m.kv.k), R.f64(m.kv.v)
    ref = R.attn(R.f64(m.q), k, v, m.table.cpu().numpy(), m.lens.tolist(), m.K, m.ad.H_q, m.ad.H_kv, m.ad.head_dim,
                 gate=R.f64(m.qkvg[:, m.cuts[2]:]))
    err = np.abs(R.f64(m.o) - ref)
    assert (err <= G.half_ulp_bf16(ref) + 2.0 ** -16 * np.abs(v).max()).all()


def test_decode_eager_and_graph():
    ex = example()
    kw = dict(H=2048, max_len=256, seed=4)
    a, b = ex.HybridDecoder(5, **kw), ex.HybridDecoder(5, **kw)
    g = torch.Generator(device="cuda").manual_seed(1)
    graph = None
    for _ in range(40):
        x = torch.randn(5, 2048, generator=g, device="cuda").to(torch.bfloat16)
        a.hidden.copy_(x)
        b.hidden.copy_(x)
        a.step()
        if graph:
            graph.replay()
        else:
            b.step()
            graph = b.capture()
        assert torch.equal(a.xn, b.xn) and torch.equal(a.slots, b.slots)
    assert a.lens.tolist() == [40] * 5 and int(a.status.max()) == 0
    check_attention(b)


def test_verify_and_commit_follow_plain_decode():
    """Drafted tokens that are all accepted leave the lengths, slots' order and states of plain decoding; rejected ones leave
    the cache as long as what was kept."""
    ex = example()
    m = ex.HybridDecoder(4, 3, max_len=128, seed=5)
    g = torch.Generator(device="cuda").manual_seed(2)
    want = [0] * 4
    for i in range(12):
        m.hidden.copy_(torch.randn(12, 2048, generator=g, device="cuda").to(torch.bfloat16))
        m.step()
        check_attention(m)
        accept = [1 + (i + b) % 3 for b in range(4)]
        m.commit(torch.tensor(accept, dtype=torch.int32, device="cuda"))
        want = [w + a for w, a in zip(want, accept)]
        assert m.lens.tolist() == want and m.held.tolist() == [-(-w // 16) for w in want]
        assert int(m.n_free) == m.free.numel() - sum(m.held.tolist())
    assert int(m.status.max()) == 0


def test_command_line(capsys, monkeypatch):
    ex = example()
    for argv in (["--batch", "3", "--steps", "6"], ["--batch", "3", "--steps", "4", "--verify", "3"]):
        monkeypatch.setattr("sys.argv", ["hybrid_decode.py", *argv])
        ex.main()
        assert "us a step" in capsys.readouterr().out
