"""Page indices outside the cache in a block table or on the free stack: reported, and no slot is formed from them -- a product
past 31 bits would name the slot of another sequence."""
import pytest
import torch

import gated_deltanet_linear_decode_gb300 as gdn

pytestmark = pytest.mark.gpu


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("bad", [8, -1, 1 << 28, 2 ** 31 - 1, -2 ** 31])
def test_extend_forms_no_slot_from_a_page_outside_the_cache(bad):
    """Pages of 16 tokens: 2^28 pages on is slot 0 again in 32 bits."""
    lens, held = i32([3, 16, 5, 20]), i32([1, 1, 1, 2])
    table = i32([[bad, 0], [4, 0], [5, 0], [6, 7]])     # sequence 0 goes on in a page outside; sequence 1 is given one
    free, n_free = i32([0, bad, 0, 0, 0, 0, 0, 0]), i32([2])
    slots, pos, cu, st = i32([-3] * 6), i32([-3] * 6), i32([-3] * 5), i32([0] * 4)
    gdn.gdn_kv_extend(16, i32([2, 1, 1, 1]), lens, held, table, free, n_free, slots, pos, cu, dev_status=st)
    assert slots.tolist() == [-1, -1, -1, 5 * 16 + 5, 7 * 16 + 4, -1] and pos.tolist() == [3, 4, 16, 5, 20, 0]
    assert st.tolist() == [64, 64, 0, 0] and cu.tolist() == [0, 2, 3, 4, 5]
    assert lens.tolist() == [5, 17, 6, 21] and held.tolist() == [1, 2, 1, 2] and n_free.tolist() == [1]


@pytest.mark.parametrize("bad", [8, -1, 2 ** 31 - 1])
def test_truncate_reports_a_page_outside_the_cache(bad):
    lens, held, st = i32([40, 40, 40]), i32([3, 3, 3]), i32([0] * 3)
    table = i32([[0, 1, 2], [3, 4, bad], [bad, 6, 7]])
    free, n_free = i32([-5] * 8), i32([0])
    gdn.gdn_kv_truncate(16, i32([40, 32, 32]), lens, held, table, free, n_free, dev_status=st)
    assert st.tolist() == [0, 64, 0] and held.tolist() == [3, 2, 2] and n_free.tolist() == [2]
    assert free.tolist()[:2] == [7, bad]
