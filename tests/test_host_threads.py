"""Calls of one entry point from two host threads at a time, of sizes whose kernels ask for different amounts of shared memory:
no call fails for what the other thread's asked for."""
import threading

import pytest
import torch

import gated_deltanet_linear_decode_gb300 as gdn

pytestmark = pytest.mark.gpu


def i32(n, v=0):
    return torch.full((n,), v, dtype=torch.int32, device="cuda")


def extend(B):
    a = dict(page_size=16, n_new=i32(B, 1), seq_len=i32(B), n_pages=i32(B), block_table=torch.zeros(B, 2, dtype=torch.int32, device="cuda"),
             free_list=torch.arange(B, dtype=torch.int32, device="cuda"), free_count=i32(1, B), slot_map=i32(B), positions=i32(B), cu_seqlens=i32(B + 1),
             seq_len_out=i32(B), n_pages_out=i32(B), free_count_out=i32(1))
    return lambda s: gdn.gdn_kv_extend(**a, stream=s)


def truncate(B):
    a = dict(page_size=16, new_len=i32(B), seq_len=i32(B), n_pages=i32(B), block_table=torch.zeros(B, 2, dtype=torch.int32, device="cuda"),
             free_list=i32(B), free_count=i32(1), seq_len_out=i32(B), n_pages_out=i32(B), free_count_out=i32(1))
    return lambda s: gdn.gdn_kv_truncate(**a, stream=s)


def norm(H):
    d = gdn.make_norm_dims(H, torch.float32, torch.float32)
    h, o = torch.randn(1, H, device="cuda"), torch.empty(1, H, device="cuda")
    return lambda s: gdn.gdn_norm_residual(d, h, o, stream=s)


@pytest.mark.parametrize("make,large,small", [(extend, 16384, 5300), (truncate, 16384, 10500), (norm, 16383, 10501)])
def test_two_threads_of_different_sizes(make, large, small):
    errors, calls = [], [make(large), make(small)]
    for c in calls:
        c(None)
    torch.cuda.synchronize()

    def loop(call):
        s = torch.cuda.Stream()
        for _ in range(4000):
            try:
                call(s)
            except gdn.GdnError as e:
                errors.append(e)
                return
        s.synchronize()

    threads = [threading.Thread(target=loop, args=(c,)) for c in calls]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors
