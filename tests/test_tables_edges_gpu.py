"""The tables of a paged cache's step at the ends of their ranges: bad pages, tens of thousands
of rows, many sequences of several tokens each, results at odd addresses."""
import ctypes

import pytest
import torch

import test_decoder_host as host
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


LARGE = [([140000], [7], 16), ([70000, 1, 70001], [3, 0, 500], 64), ([0, 33333, 0], [9, 100, 9], 256),
         # a second chunk of sequences with more rows than threads, from a multiple of four and not
         ([20] * 2048 + [30] * 2000, [i % 40 for i in range(4048)], 16),
         ([20] * 2047 + [21] + [30] * 2000, [i % 40 for i in range(4048)], 16),
         ([7] * 2047 + [8] + [25] * 3000, [i % 90 for i in range(5048)], 32)]


@pytest.mark.parametrize("new,lens,page", LARGE)
@pytest.mark.parametrize("tail", [0, 9])
@pytest.mark.parametrize("inplace", [False, True])
def test_many_rows(new, lens, page, tail, inplace):
    T.test_reserve(new, lens, page, tail, inplace)


@pytest.mark.parametrize("inplace", [False, True])
def test_results_at_odd_addresses(inplace):
    new, lens, page = [40000, 3, 1], [5, 31, 0], 16
    table, free, count = T.state(new, lens, page)
    total = sum(new) + 3
    want = T.plain(new, lens, table, free.tolist(), count, page, total)
    t, f, n, l, c = table.cuda(), free.cuda(), T.i32(*new), T.i32(*lens), T.i32(count)
    pos, slots = torch.full((total + 4,), 5, dtype=I32, device="cuda"), torch.full(
        (total + 4,), 5, dtype=torch.int64, device="cuda")
    cu, out, left, missing = (torch.zeros(k, dtype=I32, device="cuda") for k in (4, 3, 1, 1))
    p = lambda x: x.data_ptr()  # noqa: E731
    r = host.Reserve(p(n), p(l), p(t), t.stride(0), t.shape[1], p(f), len(f), p(c), 3, page, total,
                     p(cu), p(l) if inplace else p(out), p(pos) + 4, p(slots) + 8,
                     p(c) if inplace else p(left), p(missing))
    stream = torch.cuda.current_stream().cuda_stream
    assert fattn.load().fa_cache_reserve(ctypes.addressof(r), stream) == fattn.FA_OK
    torch.cuda.synchronize()
    assert pos.tolist() == [5] + want[2] + [5] * 3 and slots.tolist() == [5] + want[3] + [5] * 3
    assert cu.tolist() == want[0] and (l if inplace else out).tolist() == want[1]
    assert (c if inplace else left).tolist() == want[4] and missing.tolist() == [0]
    assert t.tolist() == want[6] and fattn.fa_device_error() == fattn.FA_OK
