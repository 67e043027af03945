"""The tables of a paged cache's step built on the GPU, pages given back, and rows
written by slots: whole numbers, equal to a plain loop's."""
import pytest
import torch

import paged_ref as R
from exact_attention_93_gb300 import fattn, kvcache

pytestmark = pytest.mark.gpu
BF, HF = torch.bfloat16, torch.float16
I32 = torch.int32


def i32(*v):
    return torch.tensor(v, dtype=I32, device="cuda")


def plain(new, lens, table, free, count, page, total):
    """What the step's tables are, by a loop over the tokens."""
    table, cu, out, pos, slots = table.tolist(), [0], [], [], []
    for b, (n, l) in enumerate(zip(new, lens)):
        for p in range(l, l + n):
            if p % page == 0:
                count -= 1
                table[b][p // page] = free[count]
            pos.append(p)
            slots.append(table[b][p // page] * page + p % page)
        cu.append(cu[-1] + n)
        out.append(l + n)
    pos += [0] * (total - len(pos))
    slots += [-1] * (total - len(slots))
    return cu, out, pos, slots, [count], [0], table


def state(new, lens, page, width=None, spare=5, seed=0):
    g = torch.Generator().manual_seed(seed)
    held = [-(-x // page) for x in lens]
    need = sum(-(-(x + n) // page) - h for x, n, h in zip(lens, new, held))
    width = width or max([-(-(x + n) // page) for x, n in zip(lens, new)] + [1]) + 2
    order = torch.randperm(sum(held) + need + spare + 9, generator=g).to(I32)
    table = torch.full((len(new), width), -9, dtype=I32)
    at = 0
    for b, h in enumerate(held):
        table[b, :h] = order[at: at + h]
        at += h
    free = order[at:].contiguous()
    return table, free, need + spare


def check(got, want, table):
    for name, x, y in zip(got._fields, got, want):
        assert x.tolist() == y, name
    assert table.tolist() == want[6]


CASES = [([1], [0], 16), ([1], [16], 16), ([1], [15], 16), ([0], [0], 16), ([0, 0, 3], [5, 0, 0], 32),
         ([1] * 64, [i * 37 for i in range(64)], 64), ([17, 0, 256, 1], [0, 300, 256, 255], 256),
         ([700, 1300, 1, 900], [0, 5, 77, 128], 128), ([3] * 513, [i % 50 for i in range(513)], 16),
         ([1 + i % 3 for i in range(2048)], [i % 90 for i in range(2048)], 32),
         ([i % 2 for i in range(5000)], [i % 33 for i in range(5000)], 16),
         ([0] * 2047 + [1, 40, 0, 9], [16] * 2051, 16), ([30000], [7], 16)]


@pytest.mark.parametrize("new,lens,page", CASES)
@pytest.mark.parametrize("tail", [0, 7])
@pytest.mark.parametrize("inplace", [False, True])
def test_reserve(new, lens, page, tail, inplace):
    table, free, count = state(new, lens, page)
    total = sum(new) + tail
    want = plain(new, lens, table, free.tolist(), count, page, total)
    t, f = table.cuda(), free.cuda()
    n, l, c = i32(*new), i32(*lens), i32(count)
    for _ in range(1 if inplace else 2):  # the same again: nothing has been used up
        got = kvcache.kv_cache_reserve(n, l, t, f, c, page, total, inplace=inplace)
        check(got, want, t)
    assert fattn.fa_device_error() == fattn.FA_OK
    assert torch.equal(f, free.cuda()) and n.tolist() == list(new)
    if inplace:
        assert l.tolist() == want[1] and c.tolist() == want[4]
        assert got.seqlens.data_ptr() == l.data_ptr() and got.free_count.data_ptr() == c.data_ptr()
    else:
        assert l.tolist() == list(lens) and c.tolist() == [count]


def test_exactly_enough_pages_and_too_few():
    new, lens, page = [40, 1, 100], [0, 31, 16], 16
    table, free, count = state(new, lens, page, spare=0)
    t = table.cuda()
    got = kvcache.kv_cache_reserve(i32(*new), i32(*lens), t, free.cuda(), i32(count), page, 141)
    assert got.free_count.tolist() == [0] and got.missing.tolist() == [0]
    for less in (1, 4, count):
        for inplace in (False, True):
            t, l, c = table.cuda(), i32(*lens), i32(count - less)
            got = kvcache.kv_cache_reserve(i32(*new), l, t, free.cuda(), c, page, 150,
                                           inplace=inplace)
            assert got.missing.tolist() == [less] and torch.equal(t, table.cuda())
            assert got.cu_seqlens.tolist() == [0] * 4 and got.seqlens.tolist() == lens
            assert got.slots.tolist() == [-1] * 150 and got.positions.tolist() == [0] * 150
            assert got.free_count.tolist() == [count - less]
            assert l.tolist() == lens and c.tolist() == [count - less]
    assert fattn.fa_device_error() == fattn.FA_OK  # not an error: the caller makes room


@pytest.mark.parametrize("bad", ["new", "length", "table", "sum", "total", "count", "count more"])
def test_bad_lengths_change_nothing(bad):
    new, lens, page, total = [3, 5, 2], [10, 0, 40], 16, 10
    table, free, count = state(new, lens, page, width=4)
    count = {"count": -1, "count more": len(free) + 1}.get(bad, count)
    if bad == "new":
        new[1] = -1
    elif bad == "length":
        lens[2] = -3
    elif bad == "table":
        lens[0] = 62
    elif bad == "sum":
        new[0], lens[0] = (1 << 31) - 1, 64
    elif bad == "total":
        total = 9
    t, f = table.cuda(), free.cuda()
    got = kvcache.kv_cache_reserve(i32(*new), i32(*lens), t, f, i32(count), page, total)
    assert got.missing.tolist() == [-1] and torch.equal(t, table.cuda())
    assert got.cu_seqlens.tolist() == [0] * 4 and got.seqlens.tolist() == lens
    assert got.slots.tolist() == [-1] * total and got.free_count.tolist() == [count]
    assert fattn.fa_device_error() == fattn.FA_ERR_INVALID_ARG
    assert fattn.fa_device_error() == fattn.FA_OK


def test_tables_of_other_strides_an_empty_step_and_no_free_pages():
    wide = torch.full((3, 20), 4, dtype=I32, device="cuda")
    table = wide[:, 5:9]
    got = kvcache.kv_cache_reserve(i32(1, 20, 0), i32(0, 3, 9), table, i32(*range(50, 60)), i32(10),
                                   16, 21)
    assert got.missing.tolist() == [0]
    assert table.tolist() == [[59, 4, 4, 4], [4, 58, 4, 4], [4, 4, 4, 4]]
    assert (wide[:, :5] == 4).all() and (wide[:, 9:] == 4).all()
    none = torch.empty(0, dtype=I32, device="cuda")
    got = kvcache.kv_cache_reserve(i32(0, 2), i32(0, 3), wide[:2], none, i32(0), 32, 2)
    assert got.missing.tolist() == [0] and got.slots.tolist() == [4 * 32 + 3, 4 * 32 + 4]
    got = kvcache.kv_cache_reserve(i32(0, 0), i32(0, 3), wide[:2], none, i32(0), 32, 0)
    assert got.missing.tolist() == [0] and got.slots.numel() == 0
    assert got.cu_seqlens.tolist() == [0, 0, 0]


def test_slots_beyond_32_bits():
    page = (1 << 31) // 256 + 3  # page * 256 needs 64 bits
    table = torch.zeros(1, 2, dtype=I32, device="cuda")
    got = kvcache.kv_cache_reserve(i32(2), i32(255), table, i32(page), i32(1), 256, 2)
    assert got.slots.tolist() == [255, page * 256]


def test_reserve_in_graphs_and_on_streams():
    new, lens, page = [1] * 40, [i * 11 for i in range(40)], 16
    table, free, count = state(new, lens, page, spare=200, width=60)
    t, f, n, l, c = table.cuda(), free.cuda(), i32(*new), i32(*lens), i32(count)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):  # a loop of steps: lengths and count go on in place
        got = kvcache.kv_cache_reserve(n, l, t, f, c, page, 40, inplace=True)
    for _ in range(20):
        want = plain(new, lens, table, free.tolist(), count, page, 40)
        graph.replay()
        check(got, want, t)
        lens, count, table = want[1], want[4][0], torch.tensor(want[6], dtype=I32)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = kvcache.kv_cache_reserve(n, l, t, f, c, page, 40, inplace=True)
    s.synchronize()
    check(got, plain(new, lens, table, free.tolist(), count, page, 40), t)


@pytest.mark.parametrize("batch,page", [(1, 16), (5, 64), (600, 16), (3000, 32)])
@pytest.mark.parametrize("keeps", [False, True])
def test_release(batch, page, keeps):
    g = torch.Generator().manual_seed(batch)
    lens = torch.randint(0, 40 * page, (batch,), generator=g).tolist()
    lens[0] = 40 * page
    done = torch.randint(0, 2, (batch,), generator=g).bool()
    done[0] = True
    keep = torch.randint(0, 9, (batch,), generator=g).tolist() if keeps else [0] * batch
    table = torch.randint(0, 1 << 20, (batch, 43), generator=g, dtype=I32)
    back = [p for b in range(batch) if done[b]
            for p in table[b, keep[b]: -(-lens[b] // page)].tolist()]
    free = torch.arange(7 + len(back), dtype=I32)
    for kind in (torch.bool, torch.uint8):
        l, f, c = i32(*lens), free.cuda(), i32(7)
        kvcache.kv_cache_release(done.to(kind).cuda(), l, table.cuda(), f, c, page,
                                 keep_pages=i32(*keep) if keeps else None)
        assert c.tolist() == [7 + len(back)]
        assert f.tolist() == list(range(7)) + back
        assert l.tolist() == [0 if d else x for d, x in zip(done.tolist(), lens)]
    # one place too few, or a bad length: nothing happens
    for what in ("room", "length", "keep"):
        if what == "room" and not back:
            continue
        l, f, c = i32(*lens), free[:-1].contiguous().cuda() if what == "room" else free.cuda(), i32(7)
        if what == "length":
            l[0] = 44 * page
        kp = i32(*keep)
        kp[0] = -1 if what == "keep" else kp[0]
        before = l.clone(), f.clone()
        kvcache.kv_cache_release(done.cuda(), l, table.cuda(), f, c, page, keep_pages=kp)
        assert fattn.fa_device_error() == fattn.FA_ERR_INVALID_ARG
        assert c.tolist() == [7] and torch.equal(l, before[0]) and torch.equal(f, before[1])
    assert fattn.fa_device_error() == fattn.FA_OK


def test_reserve_and_release_give_every_page_back():
    g = torch.Generator().manual_seed(3)
    batch, page, pages = 9, 16, 200
    table = torch.zeros(batch, 40, dtype=I32, device="cuda")
    free, c, l = torch.randperm(pages, generator=g).to(I32).cuda(), i32(pages), i32(*[0] * batch)
    for step in range(30):
        new = torch.randint(0, 60, (batch,), generator=g, dtype=I32).cuda()
        got = kvcache.kv_cache_reserve(new, l, table, free, c, page, 600, inplace=True)
        held = -(-l // page)
        assert int(held.sum() + c) == pages
        mine = torch.cat([table[b, :held[b]] for b in range(batch)] + [free[:int(c)]])
        assert torch.equal(mine.sort().values, torch.arange(pages, dtype=I32, device="cuda"))
        if int(got.missing) or step % 4 == 3:
            done = torch.randint(0, 2, (batch,), generator=g).bool().cuda()
            kvcache.kv_cache_release(done, l, table, free, c, page)
    assert fattn.fa_device_error() == fattn.FA_OK


@pytest.mark.parametrize("D,Hk,dtype,fp8", [(64, 3, BF, False), (128, 8, HF, False), (128, 4, BF, True),
                                            (64, 9, HF, True)])
def test_write_is_append_by_slots(D, Hk, dtype, fp8):
    rows, ctx, page = [5, 0, 40, 1], [3, 9, 0, 31], 16
    b = R.Batch(rows, ctx, Hk, D, page, dtype, fp8, seed=1, tail=3, poison=False)
    g = torch.Generator().manual_seed(4)
    k, v = (torch.randn(b.total, Hk, D, generator=g).to(dtype).cuda() for _ in range(2))
    made = [kvcache.alloc_kv_cache(b.pool.shape[1], page, Hk, D, R.E4M3 if fp8 else dtype)
            for _ in range(2)]
    _, _, table, cu, lens, _ = b.gpu()
    first, second = made
    kvcache.kv_cache_append(k, v, *first[:2], table, cu, lens, *first[2:])
    slots = []
    for s, (n, c) in enumerate(zip(rows, ctx)):
        slots += [int(b.table[s, p // page]) * page + p % page for p in range(c, c + n)]
    slots = torch.tensor(slots + [-1, -1, -(1 << 40)], device="cuda")
    kvcache.kv_cache_write(k, v, *second[:2], slots, *second[2:])
    assert fattn.fa_device_error() == fattn.FA_OK
    same = lambda x, y: x is None or torch.equal(x.view(torch.uint8), y.view(torch.uint8))  # noqa: E731
    assert all(same(x, y) for x, y in zip(first, second))
    # beyond the cache: not written, recorded
    slots[2] = b.pool.shape[1] * page
    slots[3] = 1 << 45
    third = kvcache.alloc_kv_cache(b.pool.shape[1], page, Hk, D, R.E4M3 if fp8 else dtype)
    kvcache.kv_cache_write(k, v, *third[:2], slots, *third[2:])
    assert fattn.fa_device_error() == fattn.FA_ERR_INVALID_ARG
    kept = [i for i in range(len(slots) - 3) if i not in (2, 3)]
    fourth = kvcache.alloc_kv_cache(b.pool.shape[1], page, Hk, D, R.E4M3 if fp8 else dtype)
    kvcache.kv_cache_write(k[kept], v[kept], *fourth[:2], slots[kept].contiguous(), *fourth[2:])
    assert all(same(x, y) for x, y in zip(third, fourth))
    assert fattn.fa_device_error() == fattn.FA_OK
