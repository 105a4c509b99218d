"""The page bookkeeping's large clusters captured in a graph: what is asked of the runtime before the launch does not end the capture."""
import random

import pytest
import torch

import gated_deltanet_linear_decode_gb300 as gdn
from tests.test_pages_shared import Books, i32

pytestmark = pytest.mark.gpu


def test_large_tables_captured():
    B, N = 20, 18
    s = Books(random.Random(3), B, 8, [100, 37] + [0] * N, 60, width=2000)   # 36,000 entries that there may be, 40,000 of the tables
    src, dst, take = i32([i % 2 for i in range(N)]), i32(list(range(2, B))), i32([100, 37] * (N // 2))
    keep, cs, cd, rs, rd = i32([100, 37] + [0] * N), i32([0] * N), i32([0] * N), i32([0] * B), i32([0] * B)
    pages = s.free.numel()
    page_map, ms, md, nm, refs, n_free = i32([0] * pages), i32([0] * pages), i32([0] * pages), i32([0]), i32([0] * pages), i32([0])
    free, table = i32([0] * pages), s.table.clone()

    def step():
        gdn.gdn_kv_fork(8, src, dst, take, s.lens, s.held, s.table, s.refs, s.free, s.n_free, cs, cd)
        gdn.gdn_kv_compact(s.held, s.table, refs, free, n_free, page_map, ms, md, nm, block_table_out=table)
        gdn.gdn_kv_release(8, keep, s.lens, s.held, s.table, s.refs, s.free, s.n_free, rs, rd)

    step()
    want = [t.clone() for t in (table, refs, n_free, page_map, ms, md, nm, s.free, s.n_free, s.refs, s.lens, s.held)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(3):
        for t in (refs, page_map, ms, md, nm):
            t.fill_(-3)
        graph.replay()
    torch.cuda.synchronize()
    got = (table, refs, n_free, page_map, ms, md, nm, s.free, s.n_free, s.refs, s.lens, s.held)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    w = s.m.fork(src.tolist(), dst.tolist(), take.tolist())
    assert (cs.tolist(), cd.tolist()) == w[:2]
    s.m.release(keep.tolist())
    assert s.refs.tolist() == s.m.refs and s.lens.tolist() == s.m.lens and s.free.tolist()[:s.m.n_free] == s.m.free[:s.m.n_free]
