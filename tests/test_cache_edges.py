"""GPU tests of the history cache where its calls meet less usual arguments: positions past the cache's slots,
splits with selected pages, padded batches. Bounds are test_cache.py's; a NaN fails them here."""
import copy
import ctypes
import threading

import numpy as np
import pytest
import torch

import block_sparse_attention_kunlun_b200 as ba
from oracle import cache as C
import test_cache
from cache_util import check
from parity_util import f64
from test_cache import ATTEND, MIDDLE, ROWS, build, i32, offsets, poison, queries

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("selected", [False, True])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("rows", ROWS)
def test_positions_past_the_cached_slots(rows, D, selected):
    """A row's window may start past the last slot of a short history: it sees itself and its tree, no cached slot
    (but selected pages). Beside it a sequence whose rows lie partly before and partly past that point."""
    lens, n = [100, 37], [rows, rows]
    cache, ref, rng = build(rows + D, [a + b for a, b in zip(lens, n)], 2, D, 16)
    q = queries(rng, 2 * rows, 2, D)
    pos = [600 + t for t in range(rows)] + [30 + 16 * t for t in range(rows)]
    mask = C.words(rng.random((2 * rows, 2, ref.table.shape[1])) < 0.3) if selected else None
    got = ba.cache_attention_fwd(cache, q.cuda(), i32(offsets(n)), i32(lens), 64, 2, positions=i32(pos),
                                 page_mask=None if mask is None else i32(mask))
    want = C.attend(ref, f64(q), offsets(n), lens, 64, 2, pos, None, mask)
    assert np.isfinite(want[1]).all()
    check(got, want, D)
    assert ba.ba_device_status(cache.status) == ba.BA_OK


def busy_block(like):
    """Leaves a freed block of `like`'s size whose last write, on the current stream, is still to come."""
    x = torch.empty_like(like)
    torch.cuda._sleep(50_000_000)
    x.view(torch.uint8).fill_(0x7F)


@pytest.mark.parametrize("as_number", [False, True])
def test_results_on_an_explicit_stream_do_not_lie_in_busy_memory(as_number):
    """Results that the binding allocates for a call on another stream must not be a block that work of the
    current stream has still to write (the allocator hands freed blocks out at once)."""
    cache, ref, rng = build(5, [3000, 2500], 2, 128, 16)
    offs, lens = i32([0, 1, 2]), i32([2900, 2400])
    q = queries(rng, 2, 4, 128).cuda()
    mean = torch.from_numpy(rng.normal(size=(ref.k.shape[0], 2, 128))).float().cuda()
    calls = {
        "attention": lambda **kw: ba.cache_attention_fwd(cache, q, offs, lens, 1 << 20, 1, **kw),
        "read": lambda **kw: ba.cache_read(cache, offs, lens, 2, **kw),
        "select": lambda **kw: (ba.cache_select(cache, q, offs, lens, mean, 64, 1, 4, **kw),),
    }
    side = torch.cuda.Stream()
    for name, call in calls.items():
        want = [t.clone() for t in call()]
        torch.cuda.synchronize()
        for t in want:
            busy_block(t)
        got = call(stream=side.cuda_stream if as_number else side)
        torch.cuda.synchronize()
        for x, y in zip(got, want):
            assert torch.equal(x, y), name


@pytest.mark.parametrize("rows", ROWS)
def test_calls_on_explicit_streams_share_no_workspace(rows):
    """Split attention on two explicit streams at once, workspaces from the binding, while the current stream
    fills freed blocks of the workspace's size: every result equals the call alone."""
    cache, _, rng = build(21, [5000, 4000], 2, 128, 64)
    args = []
    for lens in ([4900, 3900], [4800, 3950]):
        q = queries(rng, 2 * rows, 2, 128).cuda()
        args.append((q, i32([0, rows, 2 * rows]), i32(lens), 1 << 20, 1))
    need = ba.ba_cache_fwd_workspace_size(cache, ba.make_problem(args[0][0], args[0][1]), 1 << 20, 1)
    assert need > 0
    want = [ba.cache_attention_fwd(cache, *a) for a in args]
    streams = [torch.cuda.Stream() for _ in args]
    outs = [[(torch.empty_like(a[0]), torch.empty((2, 2 * rows), device="cuda")) for _ in range(40)] for a in args]
    torch.cuda.synchronize()
    for i in range(40):
        for s, a, o in zip(streams, args, outs):
            ba.cache_attention_fwd(cache, *a, out=o[i][0], lse=o[i][1], stream=s)
        for _ in range(3):
            ba.workspace_for(need, "cuda").fill_(0x7F)
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        for out, lse in o:
            assert torch.equal(out, w[0]) and torch.equal(lse, w[1])


@pytest.mark.parametrize("rows", [1, 9])
def test_threads_select_over_caches_of_different_sizes(rows):
    """Host threads, each with its own stream and cache: a call's shared memory is its own affair."""
    work = []
    for i in range(8):
        pages = (16384, 7000)[i % 2] if rows == 1 else (2048, 900)[i % 2]
        table = torch.arange(pages, dtype=torch.int32).reshape(1, pages).cuda()
        cache = ba.HistoryCache.empty(pages, 16, 1, 64, table)
        rng = np.random.default_rng(i)
        mean = torch.from_numpy(rng.normal(size=(pages, 1, 64))).float().cuda()
        q, offs, lens = queries(rng, rows, 1, 64).cuda(), i32([0, rows]), i32([1000])
        want = ba.cache_select(cache, q, offs, lens, mean, 64, 1, 3)
        mask, stream = torch.zeros_like(want), torch.cuda.Stream()
        args = (ctypes.byref(cache.struct), ctypes.byref(ba.make_problem(q, offs)), q.data_ptr(), offs.data_ptr(),
                lens.data_ptr(), None, mean.data_ptr(), 64, 1, 3, mask.data_ptr(), stream.cuda_stream)
        work.append((args, mask, want, (cache, q, offs, lens, mean, stream)))
    select, codes = ba._load().ba_cache_select, []

    def serve(args):
        codes.append({select(*args) for _ in range(5000)})

    torch.cuda.synchronize()
    threads = [threading.Thread(target=serve, args=(w[0],)) for w in work]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert codes == [{ba.BA_OK}] * len(work)
    for _, mask, want, _ in work:
        assert torch.equal(mask, want)


def test_a_cache_keeps_its_tensors():
    """The calls read the tensors' addresses as they were when the cache was made: none can be put in another's
    place. A wider page table is another cache on the same pools; a copy has tensors of its own."""
    cache, ref, rng = build(2, [40], 1, 64, 16)
    with pytest.raises(AttributeError):
        cache.page_table = torch.zeros((1, 9), dtype=torch.int32, device="cuda")
    wide = torch.full((1, 40), -1, dtype=torch.int32, device="cuda")
    wide[:, :cache.page_table.shape[1]] = cache.page_table
    wider = ba.HistoryCache(cache.k, cache.v, cache.k_scales, cache.v_scales, wide, status=cache.status)
    twin = copy.deepcopy(cache)
    assert twin.k.data_ptr() != cache.k.data_ptr() and twin.struct.k == twin.k.data_ptr()
    for c in (wider, twin):
        k, v = ba.cache_read(c, i32([0, 40]), i32([0]), 40)
        pages, at = ref.table[0, np.arange(40) // 16], np.arange(40) % 16
        assert np.array_equal(f64(k)[:, 0], ref.k[pages, 0, at]) and np.array_equal(f64(v)[:, 0], ref.v[pages, 0, at])


@pytest.mark.parametrize("group", [1, 4, 16, 20])
@pytest.mark.parametrize("slots", [200, 6000])
def test_empty_sequences_change_nothing(slots, group):
    """Single events of four sequences, alone and in a batch padded with sixty empty ones: the same kernel in the
    same splits, bit for bit."""
    lens = [slots, slots - 70, 3, slots // 2]
    cache, ref, rng = build(slots + group, [n + 1 for n in lens], 2, 64, 16)
    q = queries(rng, 4, 2 * group, 64)
    alone = ba.cache_attention_fwd(cache, q.cuda(), i32([0, 1, 2, 3, 4]), i32(lens), 1 << 20, 1)
    check(alone, C.attend(ref, f64(q), [0, 1, 2, 3, 4], lens, 1 << 20, 1), 64)
    at = [5, 6, 40, 63]
    n, padded = np.zeros(64, dtype=int), np.zeros(64, dtype=int)
    n[at], padded[at] = 1, lens
    table = torch.full((64, cache.page_table.shape[1]), -1, dtype=torch.int32, device="cuda")
    table[at] = cache.page_table
    wide = ba.HistoryCache(cache.k, cache.v, cache.k_scales, cache.v_scales, table)
    got = ba.cache_attention_fwd(wide, q.cuda(), i32(offsets(n)), i32(padded), 1 << 20, 1)
    assert torch.equal(got[0], alone[0]) and torch.equal(got[1], alone[1])


# test_cache.py's comparison passes a NaN in out: the same cases with the one that does not.

@pytest.mark.parametrize("D,size,kv,group,lens,n,block,window,kind,selected", ATTEND + MIDDLE)
def test_no_nan_where_the_oracle_has_none(monkeypatch, D, size, kv, group, lens, n, block, window, kind, selected):
    monkeypatch.setattr(test_cache, "check_attention", check)
    test_cache.test_attention_of_uneven_batches(D, size, kv, group, lens, n, block, window, kind, selected)


@pytest.mark.parametrize("rows,D", [(1, 128), (1, 64), (5, 128), (5, 64), (7, 128), (7, 64), (40, 128), (130, 64)])
def test_no_nan_from_joined_splits(monkeypatch, rows, D):
    monkeypatch.setattr(test_cache, "check_attention", check)
    test_cache.test_long_cache_split_over_blocks(rows, D)


@pytest.mark.parametrize("rows", ROWS)
def test_no_nan_in_rarer_cases(monkeypatch, rows):
    monkeypatch.setattr(test_cache, "check_attention", check)
    for D in (64, 128):
        test_cache.test_values_and_keys_of_any_scale(rows, D)
    test_cache.test_sequences_that_share_pages(rows)
    if rows < 32:   # (its tree is one word)
        test_cache.test_rows_that_see_nothing(rows)


@pytest.mark.parametrize("value", ["nan", "huge"])
@pytest.mark.parametrize("rows", ROWS)
def test_what_a_row_does_not_see_does_not_reach_it_through_splits(rows, value):
    """Selected pages of a long history, its slots split over blocks: NaN and overflowing values in unselected
    pages and behind the last row, and NaN left in the workspace, change no bit."""
    lens, chosen = [6000], [0, 3, 100, 101, 290, 370]
    cache, ref, rng = build(rows, [6000 + rows + 20], 2, 64, 16)
    q = queries(rng, rows, 4, 64)
    bits = np.zeros((rows, 2, ref.table.shape[1]), dtype=bool)
    bits[:, :, chosen] = True
    mask = C.words(bits)
    need = ba.ba_cache_fwd_workspace_size(cache, ba.make_problem(q, i32([0, rows])), 64, 1)
    assert need > 0
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")
    args = (cache, q.cuda(), i32([0, rows]), i32(lens), 64, 1)
    clean = ba.cache_attention_fwd(*args, page_mask=i32(mask), workspace=ws)
    check(clean, C.attend(ref, f64(q), [0, rows], lens, 64, 1, mask=mask), 64)
    ws0 = C.window_start(lens[0], 64, 1)
    poison(cache, [ref.slot(0, p) for p in range(6000 + rows + 20)
                   if (p < ws0 and p // 16 not in chosen) or p >= 6000 + rows], value)
    ws.fill_(0xFF)
    got = ba.cache_attention_fwd(*args, page_mask=i32(mask), workspace=ws)
    assert torch.equal(got[0], clean[0]) and torch.equal(got[1], clean[1])


@pytest.mark.parametrize("rows", ROWS)
def test_a_padded_batch_has_the_same_results(rows):
    """Tensors longer than the offsets say: the rows that there are equal the oracle's, split or not."""
    lens, spare = [6000], 5
    cache, ref, rng = build(rows, [6000 + rows], 1, 64, 16)
    q = queries(rng, rows + spare, 1, 64)
    for block in (1 << 20, 64):
        out = torch.full((rows + spare, 1, 64), float("nan"), dtype=torch.bfloat16, device="cuda")
        lse = torch.full((1, rows + spare), float("nan"), device="cuda")
        ba.cache_attention_fwd(cache, q.cuda(), i32([0, rows]), i32(lens), block, 1, out=out, lse=lse)
        assert torch.isnan(out[rows:]).all() and torch.isnan(lse[:, rows:]).all()
        check((out[:rows], lse[:, :rows]), C.attend(ref, f64(q[:rows]), [0, rows], lens, block, 1), 64)


@pytest.mark.parametrize("n", [[1, 1, 1, 1], [2, 1, 1, 1], [2, 2, 2, 2], [0, 0, 4, 0], [0, 5, 0, 0]])
@pytest.mark.parametrize("group", [1, 3])
def test_select_of_one_and_two_rows_a_sequence(n, group):
    """Around the border between the kernel for single events and the one for eight rows."""
    lens = [900, 16, 700, 333]
    cache, ref, rng = build(sum(n) + group, [a + b for a, b in zip(lens, n)], 2, 128, 16)
    q = queries(rng, sum(n), 2 * group, 128)
    mean = torch.from_numpy(rng.normal(size=(ref.k.shape[0], 2, 128))).float()
    got = ba.cache_select(cache, q.cuda(), i32(offsets(n)), i32(lens), mean.cuda(), 64, 1, 6)
    want = C.select(ref, f64(q), offsets(n), lens, f64(mean), 64, 1, 6)
    assert np.array_equal(got.cpu().numpy(), C.words(want))


@pytest.mark.parametrize("size", [16, 32, 128])
@pytest.mark.parametrize("rows", ROWS)
def test_pages_before_the_window_may_be_gone(rows, size):
    """A history whose pages before every row's window were given back: no call needs them, none reports them."""
    lens, block = [900], 48
    cache, ref, rng = build(rows + size, [900 + rows], 2, 64, size)
    gone = C.window_start(lens[0], block, 2) // size
    assert gone > 0 and C.window_start(lens[0], block, 2) % 64 >= 48
    cache.page_table[0, :gone] = -1
    ref.table[0, :gone] = -1
    q = queries(rng, rows, 2, 64)
    got = ba.cache_attention_fwd(cache, q.cuda(), i32([0, rows]), i32(lens), block, 2)
    assert ba.ba_device_status(cache.status) == ba.BA_OK
    check(got, C.attend(ref, f64(q), [0, rows], lens, block, 2), 64)
    cache.page_table[0, gone] = -1                       # one that is needed
    ba.cache_attention_fwd(cache, q.cuda(), i32([0, rows]), i32(lens), block, 2)
    assert ba.ba_device_status(cache.status) == ba.BA_ERR_INVALID_ARG


@pytest.mark.parametrize("selected", [False, True])
@pytest.mark.parametrize("rows", ROWS)
def test_rows_at_negative_positions_ask_for_nothing(rows, selected):
    """A row that sees nothing (a padded tree's) does not make its tile walk the history from the start: pages that
    the other rows do not need may be gone."""
    lens, block, n = [900, 900], 48, [rows, rows]
    cache, ref, rng = build(rows, [900 + rows] * 2, 2, 64, 16)
    gone = C.window_start(900, block, 2) // 16
    keep = [7] if selected else []
    drop = [c for c in range(gone) if c not in keep]
    cache.page_table[:, drop] = -1
    ref.table[:, drop] = -1
    q = queries(rng, 2 * rows, 2, 64)
    pos = [900 + t if t % 3 else -1 - t for t in range(rows)] + [-1] * rows
    mask = None
    if selected:
        bits = np.zeros((2 * rows, 2, ref.table.shape[1]), dtype=bool)
        bits[:, :, keep] = True
        mask = C.words(bits)
    got = ba.cache_attention_fwd(cache, q.cuda(), i32(offsets(n)), i32(lens), block, 2, positions=i32(pos),
                                 page_mask=None if mask is None else i32(mask))
    assert ba.ba_device_status(cache.status) == ba.BA_OK
    check(got, C.attend(ref, f64(q), offsets(n), lens, block, 2, pos, None, mask), 64)


@pytest.mark.parametrize("selected", [False, True])
@pytest.mark.parametrize("rows", ROWS)
def test_a_tree_without_positions(rows, selected):
    """tree_mask alone: row t is at position lens + t, and any bits count, those of later rows excepted."""
    lens, n = [70, 333], [rows, max(1, rows - 2)]
    cache, ref, rng = build(rows, [a + b for a, b in zip(lens, n)], 2, 128, 16)
    total = sum(n)
    q = queries(rng, total, 2, 128)
    tree = C.words(rng.random((total, 64)) < 0.5)
    mask = C.words(rng.random((total, 2, ref.table.shape[1])) < 0.2) if selected else None
    got = ba.cache_attention_fwd(cache, q.cuda(), i32(offsets(n)), i32(lens), 32, 2, tree_mask=i32(tree),
                                 page_mask=None if mask is None else i32(mask))
    check(got, C.attend(ref, f64(q), offsets(n), lens, 32, 2, None, tree, mask), 128)
    assert ba.ba_device_status(cache.status) == ba.BA_OK


@pytest.mark.parametrize("rows", ROWS)
def test_captured_with_the_bindings_buffers_on_a_stream_of_the_capture(rows):
    """Two branches of one graph, each a split call on an explicit stream with buffers from the binding."""
    cache, _, rng = build(rows, [4000 + rows], 1, 128, 64)
    q = [queries(rng, rows, 1, 128).cuda() for _ in "ab"]
    offs, lens = i32([0, rows]), i32([4000])
    want = [ba.cache_attention_fwd(cache, x, offs, lens, 1 << 20, 1) for x in q]
    side = [torch.cuda.Stream() for _ in q]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = []
        for s, x in zip(side, q):
            s.wait_stream(torch.cuda.current_stream())
            got.append(ba.cache_attention_fwd(cache, x, offs, lens, 1 << 20, 1, stream=s))
        for s in side:
            torch.cuda.current_stream().wait_stream(s)
    for _ in range(20):
        for out, lse in got:
            out.zero_(), lse.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for x, y in zip(got, want):
            assert torch.equal(x[0], y[0]) and torch.equal(x[1], y[1])
