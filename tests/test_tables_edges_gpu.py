"""The tables of a paged cache's step at the ends of their ranges: bad pages."""
import pytest
import torch

import test_tables_gpu as T
from exact_attention_93_gb300 import fattn, kvcache

pytestmark = pytest.mark.gpu
I32 = torch.int32


@pytest.mark.parametrize("inplace", [False, True])
@pytest.mark.parametrize("where", ["held", "free"])
@pytest.mark.parametrize("rows", [1, 5, 9000])
def test_a_page_below_zero_is_recorded(where, rows, inplace):
    # Its rows would else be taken for ones that are not to be written, and lost without a word.
    new, lens, page = [rows, 20, 3], [20, 3, 0], 16
    table, free, count = T.state(new, lens, page)
    total = sum(new) + 2
    want = T.plain(new, lens, table, free.tolist(), count, page, total)
    if where == "held":  # keys 16 .. 31 of the first sequence
        table[0, 1] = -2
        bad = range(0, min(rows, 12))
    else:  # the last page taken: the third sequence's
        taken = count - want[4][0]
        free[count - taken] = -7
        bad = range(rows + 20, rows + 23)
    t = table.cuda()
    got = kvcache.kv_cache_reserve(T.i32(*new), T.i32(*lens), t, free.cuda(), T.i32(count), page, total,
                                   inplace=inplace)
    slots = [-1 if i in bad else s for i, s in enumerate(want[3])]
    assert got.slots.tolist() == slots
    assert got.positions.tolist() == want[2] and got.cu_seqlens.tolist() == want[0]
    assert fattn.fa_device_error() == fattn.FA_ERR_INVALID_ARG
    assert fattn.fa_device_error() == fattn.FA_OK


def test_a_page_below_zero_that_no_new_token_needs():
    table = torch.full((2, 4), -1, dtype=I32, device="cuda")
    table[0, 1] = 3
    got = kvcache.kv_cache_reserve(T.i32(2, 0), T.i32(20, 40), table, T.i32(5), T.i32(1), 16, 2)
    assert got.slots.tolist() == [3 * 16 + 4, 3 * 16 + 5]
    assert fattn.fa_device_error() == fattn.FA_OK
