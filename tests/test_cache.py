"""GPU parity of the history cache (ba_cache_*) against oracle/cache.py.

Writing is byte work and must match the oracle's codes; reading and page
selection must match exactly too. Attention is held to a bound that follows
from its arithmetic (attention_bound)."""
import numpy as np
import pytest
import torch

import block_sparse_attention_kunlun_b200 as ba
from oracle import cache as C
from parity_util import f64

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32).cuda()


def build(seed, lengths, kv_heads, D, size, extra_pages=3, spare=1):
    """A cache with random codes in shuffled pages; page table rows end in -1."""
    rng = np.random.default_rng(seed)
    need = [-(-int(n) // size) for n in lengths]
    pages = sum(need) + extra_pages
    ids = rng.permutation(pages)
    table = np.full((len(lengths), max(max(need), 1) + spare), -1, dtype=np.int32)
    at = 0
    for b, m in enumerate(need):
        table[b, :m] = ids[at:at + m]
        at += m
    shape = (pages, kv_heads, size, D)
    codes = []
    for _ in "kv":
        x = torch.from_numpy(rng.normal(size=shape))
        el, e = C.quantize(x.numpy())
        codes.append(torch.from_numpy(el).to(torch.float8_e4m3fn).view(torch.uint8))
        codes.append(torch.from_numpy((e + 127).astype(np.uint8)))
    k, ks, v, vs = codes
    cache = ba.HistoryCache(k.cuda(), v.cuda(), ks.cuda(), vs.cuda(), i32(table))
    return cache, C.Cache(k.numpy(), v.numpy(), ks.numpy(), vs.numpy(), table), rng


def offsets(n):
    return np.concatenate([[0], np.cumsum(n)]).astype(np.int32)


def queries(rng, rows, heads, D, gain=1.0):
    return torch.from_numpy(rng.normal(size=(rows, heads, D)) * gain).to(torch.bfloat16)


def attention_bound(ref, D):
    """Largest errors of out and lse. A float32 score over D products (cut, not rounded, in the tensor core's
    sum) is off by at most ds = (D + 8) 2^-23 reach, reach = sum |q k| / sqrt(D); 2^x, its argument and the sum
    of the probabilities add 2^-20; P is rounded to bf16 (2^-8) for the tensor core's P V; out is rounded to
    bf16 (2^-8 of its value). A change of all scores by ds changes out by at most (e^(2 ds) - 1) sum p |v|."""
    out, lse, spread, reach = ref
    ds = (D + 8) * 2.0 ** -23 * reach.T[..., None]
    tol_out = 2.0 ** -8 * np.abs(out) + (2.0 ** -8 + np.expm1(2 * ds) + 2.0 ** -19) * spread * (1 + 2.0 ** -8) + 1e-30
    tol_lse = ds[..., 0].T + 2.0 ** -19 + 2.0 ** -23 * np.abs(np.where(np.isfinite(lse), lse, 0.0))
    return tol_out, tol_lse


def check_attention(got, ref, D, more=0.0):
    out, lse = f64(got[0]), f64(got[1])
    tol_out, tol_lse = attention_bound(ref, D)
    tol_out = tol_out + more
    assert np.array_equal(np.isneginf(lse), np.isneginf(ref[1]))
    seen = np.isfinite(ref[1])
    assert np.all(np.abs(lse - ref[1])[seen] <= tol_lse[seen]), np.max((np.abs(lse - ref[1]) - tol_lse)[seen])
    bad = np.abs(out - ref[0]) > tol_out
    assert not bad.any(), (np.argwhere(bad)[:5], np.max(np.abs(out - ref[0]) / tol_out))


# ------------------------------------------------------------ write, read ---

@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("D,size,heads", [(64, 16, 1), (64, 128, 3), (128, 32, 5), (128, 64, 8)])
def test_write_matches_the_oracle_byte_for_byte(dtype, D, size, heads):
    n, starts = [0, 1, 37, 130, 2], [5, 15, 16, 3, 127]
    cache, _, rng = build(D + size, [a + b for a, b in zip(starts, n)], heads, D, size)
    rows = sum(n)
    x = [torch.from_numpy(rng.normal(size=(rows, heads, D)) * np.exp2(rng.integers(-30, 30, (rows, heads, 1)))).to(dtype)
         for _ in "kv"]
    x[0][0] = 0.0
    x[0][1, 0, :32] = 2.0 ** -130                        # subnormal in both types
    x[1][2, 0, 3] = 3.0e38
    x[1][3, 0, :4] = torch.tensor([448.0, 464.0, 480.0, -500.0])
    before = [t.clone() for t in (cache.k, cache.v, cache.k_scales, cache.v_scales)]
    offs = offsets(n)
    ba.cache_write(cache, x[0].cuda(), x[1].cuda(), i32(offs), i32(starts))
    assert ba.ba_device_status(cache.status) == ba.BA_OK
    table = cache.page_table.cpu().numpy()
    for t, el_pool, sc_pool, old_el, old_sc in ((x[0], cache.k, cache.k_scales, before[0], before[2]),
                                                (x[1], cache.v, cache.v_scales, before[1], before[3])):
        el, e = C.quantize(f64(t))
        want_el, want_sc = C.e4m3_values(old_el.cpu().numpy()), old_sc.cpu().numpy().astype(np.int64)
        for b in range(len(n)):
            for i in range(n[b]):
                p = starts[b] + i
                page, at = table[b, p // size], p % size
                want_el[page, :, at], want_sc[page, :, at] = el[offs[b] + i], e[offs[b] + i] + 127
        assert np.array_equal(C.e4m3_values(el_pool.cpu().numpy()), want_el)
        assert np.array_equal(sc_pool.cpu().numpy().astype(np.int64), want_sc)   # other slots as they were


def test_write_of_nan_and_infinity():
    cache, _, _ = build(3, [4], 1, 64, 16)
    x = torch.ones(2, 1, 64)
    x[0, 0, 5] = float("nan")
    x[1, 0, 40] = -float("inf")
    ba.cache_write(cache, x.cuda(), x.cuda(), i32([0, 2]), i32([1]))
    k, _ = ba.cache_read(cache, i32([0, 2]), i32([1]), 2, dtype=torch.float32)
    k = k.cpu()
    assert torch.isnan(k[0, 0, 5]) and torch.equal(torch.isnan(k).sum(), torch.tensor(1))
    assert k[1, 0, 40] == -448.0 * 2.0 ** 120 and k[1, 0, 41] == 0.0 and k[1, 0, 3] == 1.0 and k[0, 0, 6] == 1.0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("D,size,heads", [(64, 16, 3), (128, 128, 2)])
def test_read_is_exact(dtype, D, size, heads):
    n, starts = [40, 0, 1, 129], [3, 7, 0, 64]
    cache, ref, _ = build(7 + D, [a + b for a, b in zip(starts, n)], heads, D, size)
    offs = offsets(n)
    k, v = ba.cache_read(cache, i32(offs), i32(starts), sum(n), dtype=dtype)
    for got, pool in ((k, ref.k), (v, ref.v)):
        want = [pool[ref.slot(b, starts[b] + i)[0], :, ref.slot(b, starts[b] + i)[1]]
                for b in range(len(n)) for i in range(n[b])]
        assert got.dtype == dtype and np.array_equal(f64(got), np.stack(want))


def test_slots_outside_the_cache_are_skipped_and_reported():
    """Past max_pages, without a page, a page number past the pools, negative: zeros from a read, nothing
    written, the status word set (and kept until the caller clears it)."""
    cache, _, rng = build(11, [64, 64, 64, 64], 2, 64, 16, spare=0)
    table = cache.page_table
    table[1, 2], table[2, 1] = -7, cache.k.shape[0]
    n, starts = [5, 40, 30, 4], [62, 10, 10, -2]
    offs = offsets(n)
    before = [t.clone() for t in (cache.k, cache.v, cache.k_scales, cache.v_scales)]
    x = torch.from_numpy(rng.normal(size=(sum(n), 2, 64))).to(torch.bfloat16).cuda()
    ba.cache_write(cache, x, -x, i32(offs), i32(starts))
    assert ba.ba_device_status(cache.status) == ba.BA_ERR_INVALID_ARG
    k, v = ba.cache_read(cache, i32(offs), i32(starts), sum(n))
    ref = C.Cache(*(t.cpu().numpy() for t in (cache.k, cache.v, cache.k_scales, cache.v_scales, table)))
    written = set()
    for b in range(4):
        for i in range(n[b]):
            at = ref.slot(b, starts[b] + i)
            row = int(offs[b]) + i
            if at is None:
                assert not k[row].any() and not v[row].any()
            else:
                written.add(at)
                assert np.array_equal(f64(k[row]), ref.k[at[0], :, at[1]]) and torch.equal(k[row], -v[row])
    same = torch.ones(cache.k.shape[0], 16, dtype=torch.bool)
    for page, at in written:
        same[page, at] = False
    assert len(written) == 2 + (40 - 16) + (30 - 16) + 2
    for t, old in zip((cache.k, cache.v, cache.k_scales, cache.v_scales), before):
        assert torch.equal(t.cpu().transpose(1, 2)[same], old.cpu().transpose(1, 2)[same])
    cache.status.zero_()
    ba.cache_read(cache, i32([0, 1, 1, 1, 1]), i32([0, 0, 0, 0]), 1)
    assert ba.ba_device_status(cache.status) == ba.BA_OK


# ------------------------------------------------------ summaries, select ---

@pytest.mark.parametrize("D,size,heads", [(64, 16, 3), (64, 128, 1), (128, 16, 2), (128, 64, 8), (128, 128, 1)])
def test_summaries(D, size, heads):
    lengths = [size * 3, 5, size * 2 + 1, 0, size]
    cache, ref, rng = build(D + size, lengths, heads, D, size)
    starts, ends = [0, 0, size, 0, size - 1], lengths
    out = torch.full((ref.k.shape[0], heads, D), 7.0, device="cuda")
    ba.cache_summarize(cache, i32(starts), i32(ends), out)
    assert ba.ba_device_status(cache.status) == ba.BA_OK
    want = C.summarize(ref, starts, ends, np.full(out.shape, 7.0))
    mag = np.abs(ref.k).mean(axis=2)
    assert np.array_equal(want == 7.0, f64(out) == 7.0)
    # a float32 sum of `size` exact terms: size roundings of at most the sum of magnitudes
    assert np.all(np.abs(f64(out) - want) <= size * 2.0 ** -24 * np.maximum(mag, 1e-30))


def test_summaries_of_pages_without_a_number():
    cache, ref, _ = build(5, [64, 64], 2, 64, 16, spare=0)
    cache.page_table[0, 1] = -1
    out = torch.zeros((ref.k.shape[0], 2, 64), device="cuda")
    ba.cache_summarize(cache, i32([0, -5]), i32([64, 1000]), out)   # past max_pages: the pages that there are
    assert ba.ba_device_status(cache.status) == ba.BA_ERR_INVALID_ARG
    ref.table[0, 1] = -1
    want = C.summarize(ref, [0, 0], [64, 64], np.zeros(out.shape))
    assert np.array_equal(want.any(axis=(1, 2)), f64(out).any(axis=(1, 2)))


SELECT = [
    # D, size, kv heads, group, lens, rows, block, window, topk
    (64, 16, 2, 1, [0, 15, 16, 700, 333], [1, 1, 1, 1, 1], 64, 1, 8),
    (128, 64, 1, 4, [3000, 64, 129], [1, 1, 1], 1, 1, 3),
    (128, 32, 2, 2, [2000, 31, 900], [9, 3, 17], 128, 2, 5),
    (64, 128, 3, 1, [1500, 128], [8, 25], 100, 1, 64),
    (128, 16, 1, 3, [1040], [1], 16, 1, 1),
]


@pytest.mark.parametrize("D,size,kv,group,lens,n,block,window,topk", SELECT)
def test_select_matches_the_oracle(D, size, kv, group, lens, n, block, window, topk):
    cache, ref, rng = build(D + size + topk, [a + b for a, b in zip(lens, n)], kv, D, size)
    rows = sum(n)
    q = queries(rng, rows, kv * group, D)
    mean = torch.from_numpy(rng.normal(size=(ref.k.shape[0], kv, D))).float()
    mean[2] = mean[0]                                    # equal scores: the lower page wins
    if ref.k.shape[0] > 4:
        mean[4] = mean[0]
    got = ba.cache_select(cache, q.cuda(), i32(offsets(n)), i32(lens), mean.cuda(), block, window, topk)
    assert ba.ba_device_status(cache.status) == ba.BA_OK
    want = C.select(ref, f64(q), offsets(n), lens, f64(mean), block, window, topk)
    assert np.array_equal(got.cpu().numpy(), C.words(want))


def test_select_with_positions_ties_and_nan():
    cache, ref, rng = build(2, [400, 400], 2, 64, 16)
    n = [12, 1]
    q = queries(rng, 13, 2, 64)
    q[0] = 0.0                                           # every score 0: the first pages
    pos = [399 - 30 * i for i in range(12)] + [-3]       # past, near the start, negative
    mean = torch.from_numpy(rng.normal(size=(ref.k.shape[0], 2, 64))).float()
    mean[ref.table[0, 3]] = float("nan")                 # selected only when nothing else is left
    mean[ref.table[0, 5], 0, 7] = float("inf")
    for topk in (2, 6, 24, 100):
        got = ba.cache_select(cache, q.cuda(), i32(offsets(n)), i32([390, 390]), mean.cuda(), 32, 1, topk,
                              positions=i32(pos))
        with np.errstate(invalid="ignore"):
            want = C.select(ref, f64(q), offsets(n), [390, 390], f64(mean), 32, 1, topk, positions=pos)
        assert np.array_equal(got.cpu().numpy(), C.words(want)), topk


@pytest.mark.parametrize("D,size,pages,rows", [(64, 16, 40, 1), (128, 16, 300, 9), (64, 16, 1100, 3)])
def test_select_of_scores_that_float32_cannot_tell_apart(D, size, pages, rows):
    """Means equal but for last places: the order is that of the exact scores, ties to the lower page."""
    cache, ref, rng = build(pages, [pages * size + rows], 1, D, size)
    q = queries(rng, rows, 2, D)
    base = rng.normal(size=D)
    mean = torch.from_numpy(np.tile(base, (ref.k.shape[0], 1, 1))).float()
    for c in range(ref.k.shape[0]):
        d = int(rng.integers(0, D))
        mean[c, 0, d] = torch.nextafter(mean[c, 0, d], torch.tensor(float("inf") if c % 3 else float("-inf")))
    mean[5] = mean[1]
    for topk in (1, 7, pages // 2):
        got = ba.cache_select(cache, q.cuda(), i32([0, rows]), i32([pages * size]), mean.cuda(), size, 1, topk)
        want = C.select(ref, f64(q), [0, rows], [pages * size], f64(mean), size, 1, topk)
        assert np.array_equal(got.cpu().numpy(), C.words(want)), topk


def test_select_of_scores_past_float32():
    """Products that overflow float32 but not float64, and ones that underflow it."""
    cache, ref, rng = build(3, [700], 1, 64, 16)
    for scale_q, scale_m in ((2.0 ** 100, 2.0 ** 60), (2.0 ** -90, 2.0 ** -60), (2.0 ** -126, 1.0)):
        q = (queries(rng, 2, 1, 64).double() * scale_q).to(torch.bfloat16)
        mean = (torch.from_numpy(rng.normal(size=(ref.k.shape[0], 1, 64))) * scale_m).float()
        got = ba.cache_select(cache, q.cuda(), i32([0, 2]), i32([698]), mean.cuda(), 16, 1, 5)
        want = C.select(ref, f64(q), [0, 2], [698], f64(mean), 16, 1, 5)
        assert np.array_equal(got.cpu().numpy(), C.words(want)), scale_q


def test_select_skips_pages_without_a_number():
    cache, ref, rng = build(8, [300], 1, 64, 16)
    cache.page_table[0, 4] = -1
    ref.table[0, 4] = -1
    q = queries(rng, 1, 1, 64)
    mean = torch.from_numpy(rng.normal(size=(ref.k.shape[0], 1, 64))).float()
    got = ba.cache_select(cache, q.cuda(), i32([0, 1]), i32([299]), mean.cuda(), 16, 1, 100)
    want = C.select(ref, f64(q), [0, 1], [299], f64(mean), 16, 1, 100)
    assert not want[0, 0, 4] and np.array_equal(got.cpu().numpy(), C.words(want))
    assert ba.ba_device_status(cache.status) == ba.BA_ERR_INVALID_ARG


# -------------------------------------------------------------- attention ---

def tree_case(rng, lens, n, kind):
    """(tree words, positions) of random trees, candidates or random visibility."""
    words = max(1, -(-max(n) // 32))
    tree, pos = [], []
    for b in range(len(n)):
        sees = np.zeros((n[b], 32 * words), dtype=bool)
        for j in range(n[b]):
            if kind == "candidates":
                sees[j, j] = True
                pos.append(lens[b])
                continue
            parent = int(rng.integers(-1, j)) if j else -1
            if parent >= 0:
                sees[j] = sees[parent]
            sees[j, j] = True
            pos.append(lens[b] + int(sees[j].sum()) - 1)
            if kind == "ragged" and rng.random() < 0.3:
                sees[j] = rng.random(32 * words) < 0.5      # any bits, past the rows too
        tree.append(sees)
    return C.words(np.concatenate(tree)) if tree else np.zeros((0, words), dtype=np.int32), pos


ATTEND = [
    # D, size, kv, group, lens, rows, block, window, kind, selected
    (128, 64, 2, 1, [0, 1, 63, 64, 500, 777], [1] * 6, 256, 2, "chain", 0),
    (64, 16, 3, 1, [0, 15, 300], [1, 1, 1], 16, 1, "chain", 0),
    (128, 32, 1, 4, [1000, 31], [1, 1], 1 << 20, 1, "chain", 0),
    (128, 128, 2, 2, [129, 5, 600], [1, 0, 1], 1, 100, "chain", 0),
    (64, 64, 1, 3, [700, 2], [2, 1], 128, 3, "chain", 0),
    (128, 16, 2, 1, [40, 0, 200], [5, 33, 17], 64, 2, "tree", 0),
    (64, 32, 1, 8, [100, 257], [40, 1], 96, 1, "ragged", 0),
    (128, 64, 1, 2, [900, 64, 300], [20, 3, 65], 128, 1, "candidates", 4),
    (64, 16, 2, 1, [500, 48], [1, 1], 32, 1, "chain", 6),
    (128, 32, 1, 1, [333], [150], 64, 2, "chain", 0),
    (64, 128, 2, 4, [0], [70], 1 << 20, 1, "chain", 0),
    (128, 64, 1, 16, [260, 130], [9, 9], 64, 1, "tree", 2),
]


@pytest.mark.parametrize("D,size,kv,group,lens,n,block,window,kind,selected", ATTEND)
@pytest.mark.parametrize("gain", [1.0, 6.0], ids=["plain", "peaked"])
def test_attention_matches_the_oracle(D, size, kv, group, lens, n, block, window, kind, selected, gain):
    cache, ref, rng = build(D + size + len(n), [a + b for a, b in zip(lens, n)], kv, D, size)
    rows, offs = sum(n), offsets(n)
    q = queries(rng, rows, kv * group, D, gain)
    tree = pos = mask = None
    if kind != "chain":
        tree, pos = tree_case(rng, lens, n, kind)
    if selected:
        P = ref.table.shape[1]
        bits = np.zeros((rows, kv, P), dtype=bool)
        for r in range(rows):
            for h in range(kv):
                bits[r, h, rng.choice(P, min(selected, P), replace=False)] = True
        mask = C.words(bits)
    got = ba.cache_attention_fwd(cache, q.cuda(), i32(offs), i32(lens), block, window,
                                 positions=None if pos is None else i32(pos),
                                 tree_mask=None if tree is None else i32(tree),
                                 page_mask=None if mask is None else i32(mask))
    assert ba.ba_device_status(cache.status) == ba.BA_OK
    check_attention(got, C.attend(ref, f64(q), offs, lens, block, window, pos, tree, mask), D)


@pytest.mark.parametrize("rows,D", [(1, 128), (1, 64), (40, 128), (130, 64)])
def test_long_cache_split_over_blocks(rows, D):
    """Few rows over a long history: the slots are split and joined; whole history, window and selection."""
    lens, n = [9000, 4097], [rows, max(1, rows - 3)]
    cache, ref, rng = build(D + rows, [a + b for a, b in zip(lens, n)], 1, D, 128)
    offs = offsets(n)
    q = queries(rng, sum(n), 2, D)
    prob = ba.make_problem(q, i32(offs))
    assert ba.ba_cache_fwd_workspace_size(cache, prob, 1 << 20, 1) > 0
    bits = np.zeros((sum(n), 1, ref.table.shape[1]), dtype=bool)
    bits[:, :, [0, 7, 8, 31]] = True
    for block, window, mask in ((1 << 20, 1, None), (1024, 3, None), (64, 1, C.words(bits))):
        got = ba.cache_attention_fwd(cache, q.cuda(), i32(offs), i32(lens), block, window,
                                     page_mask=None if mask is None else i32(mask))
        again = ba.cache_attention_fwd(cache, q.cuda(), i32(offs), i32(lens), block, window,
                                       page_mask=None if mask is None else i32(mask))
        assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1])
        pick = [0, sum(n) - 1, n[0] - 1, n[0], n[0] // 2]
        for r in set(pick):   # the oracle row by row
            b = int(r >= n[0])
            t = r - int(offs[b])
            ref_r = C.attend(ref, f64(q[r:r + 1]), [0] * (b + 1) + [1] * (2 - b), lens, block, window,
                             positions=[lens[b] + t], mask=None if mask is None else mask[r:r + 1])
            if t:   # rows of a chain see the rows before them: as cached slots of a longer history
                longer = list(lens)
                longer[b] += t
                ref_r = C.attend(ref, f64(q[r:r + 1]), [0] * (b + 1) + [1] * (2 - b), longer, block, window,
                                 positions=[lens[b] + t], mask=None if mask is None else mask[r:r + 1])
            check_attention((got[0][r:r + 1], got[1][:, r:r + 1]), ref_r, D)


@pytest.mark.parametrize("rows", [1, 2, 3, 9])
def test_rows_that_see_nothing(rows):
    """No cached slot and no bit: out 0, lse -inf; negative positions; an empty history."""
    cache, ref, rng = build(rows, [50 + rows, rows], 2, 64, 16)
    n, lens = [rows, rows], [50, 0]
    q = queries(rng, 2 * rows, 4, 64)
    tree = np.zeros((2 * rows, 1), dtype=np.int32)
    tree[rows - 1] = 1 << (rows - 1)
    pos = [-1] * rows + list(range(rows))
    pos[rows - 1] = 50
    got = ba.cache_attention_fwd(cache, q.cuda(), i32(offsets(n)), i32(lens), 16, 1, positions=i32(pos),
                                 tree_mask=i32(tree))
    want = C.attend(ref, f64(q), offsets(n), lens, 16, 1, pos, tree)
    assert np.isneginf(want[1]).sum() == 4 * (2 * rows - 1)
    check_attention(got, want, 64)
    assert not got[0][torch.isneginf(got[1].t())].any()


def poison(cache, pages_slots, value):
    """Puts NaN codes (or the largest code under the largest scale) into slots (page, row) of k and v."""
    for page, at in pages_slots:
        for t, s in ((cache.k, cache.k_scales), (cache.v, cache.v_scales)):
            t[page, :, at] = 0x7F if value == "nan" else 0x7E
            if value != "nan":
                s[page, :, at] = 254


@pytest.mark.parametrize("value", ["nan", "huge"])
@pytest.mark.parametrize("D,kind,rows", [(128, "chain", 1), (128, "tree", 20), (64, "tree", 3), (64, "candidates", 50)])
def test_what_a_row_does_not_see_does_not_reach_it(value, D, kind, rows):
    """NaN and overflowing values in unseen slots (outside the window, on unselected pages, in other branches,
    behind the last row) leave the results bit-equal; a row that sees a NaN has NaN."""
    lens, n = [200, 90], [rows, rows]
    cache, ref, rng = build(D + rows, [a + b + 20 for a, b in zip(lens, n)], 1, D, 16)
    offs = offsets(n)
    q = queries(rng, 2 * rows, 2, D)
    tree = pos = None
    if kind != "chain":
        tree, pos = tree_case(rng, lens, n, kind)
    args = (q.cuda(), i32(offs), i32(lens), 32, 2)
    kw = dict(positions=None if pos is None else i32(pos), tree_mask=None if tree is None else i32(tree))
    clean = ba.cache_attention_fwd(cache, *args, **kw)
    # slots that no row sees: before every window, behind the last row
    hidden = [ref.slot(b, p) for b in range(2) for p in list(range(C.window_start(lens[b], 32, 2))) +
              list(range(lens[b] + n[b], lens[b] + n[b] + 20)) if ref.slot(b, p) is not None]
    poison(cache, hidden, value)
    got = ba.cache_attention_fwd(cache, *args, **kw)
    assert torch.equal(got[0], clean[0]) and torch.equal(got[1], clean[1])
    # the last row's slot: rows that see it become NaN, the others keep their bits
    poison(cache, [ref.slot(0, lens[0] + rows - 1)], value)
    got = ba.cache_attention_fwd(cache, *args, **kw)
    p = [lens[0] + t for t in range(rows)] if pos is None else pos[:rows]
    for t in range(2 * rows):
        sees = t < rows and lens[0] + rows - 1 in C.visible(ref, 0, 0, rows, t, lens[0], p, 32, 2,
                                                              None if tree is None else tree[:rows])
        if not sees:
            assert torch.equal(got[0][t], clean[0][t]) and torch.equal(got[1][:, t], clean[1][:, t]), t
        elif value == "nan":
            assert torch.isnan(got[0][t]).all() and torch.isnan(got[1][:, t]).all(), t


def test_nan_in_a_value_column_reaches_only_that_column():
    lens, n = [100], [12]
    cache, ref, rng = build(4, [112], 1, 128, 16)
    tree, pos = tree_case(rng, lens, n, "candidates")
    q = queries(rng, 12, 1, 128)
    args = (q.cuda(), i32([0, 12]), i32(lens), 32, 2)
    kw = dict(positions=i32(pos), tree_mask=i32(tree))
    clean = ba.cache_attention_fwd(cache, *args, **kw)
    page, at = ref.slot(0, 103)
    cache.v[page, 0, at, 77] = 0xFF
    got = ba.cache_attention_fwd(cache, *args, **kw)
    same = torch.ones_like(clean[0], dtype=torch.bool)
    same[3, 0, 77] = False
    assert torch.equal(got[0][same], clean[0][same]) and torch.equal(got[1], clean[1])
    assert torch.isnan(got[0][3, 0, 77])


def test_pages_without_a_number_are_unseen_and_reported():
    for rows in (1, 30):
        cache, ref, rng = build(6, [300 + rows], 2, 64, 16)
        cache.page_table[0, 17], cache.page_table[0, 18] = -1, 1 << 30
        ref.table[0, 17], ref.table[0, 18] = -1, 1 << 30
        q = queries(rng, rows, 2, 64)
        got = ba.cache_attention_fwd(cache, q.cuda(), i32([0, rows]), i32([300]), 64, 2)
        assert ba.ba_device_status(cache.status) == ba.BA_ERR_INVALID_ARG
        check_attention(got, C.attend(ref, f64(q), [0, rows], [300], 64, 2), 64)


def test_rows_past_the_cache_are_unseen_and_reported():
    cache, ref, rng = build(6, [60], 1, 64, 16, spare=0)       # 64 slots
    q = queries(rng, 10, 1, 64)
    got = ba.cache_attention_fwd(cache, q.cuda(), i32([0, 10]), i32([60]), 16, 2)
    assert ba.ba_device_status(cache.status) == ba.BA_ERR_INVALID_ARG
    check_attention(got, C.attend(ref, f64(q), [0, 10], [60], 16, 2), 64)


def test_rows_of_nobody_are_left_as_they_were():
    """Buffers with room behind the last row, and an empty batch."""
    cache, ref, rng = build(9, [41, 33], 2, 64, 16)
    q = queries(rng, 2, 2, 64)
    big = torch.full((6, 2, 64), 9.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((2, 2), 9.0, device="cuda")
    ba.cache_attention_fwd(cache, q.cuda(), i32([0, 1, 2]), i32([40, 32]), 16, 2, out=big[:2], lse=lse)
    assert torch.all(big[2:] == 9.0)
    check_attention((big[:2], lse), C.attend(ref, f64(q), [0, 1, 2], [40, 32], 16, 2), 64)
    none = torch.empty((0, 2, 64), dtype=torch.bfloat16, device="cuda")
    out, _ = ba.cache_attention_fwd(cache, none, i32([0, 0, 0]), i32([40, 32]), 16, 2)
    assert out.shape == (0, 2, 64)


def test_element_offsets_past_32_bits():
    """A pool of more than 2^32 element bytes; the pages in use are its last ones."""
    pages, size, heads, D = 70000, 128, 4, 128
    table = torch.full((1, 3), -1, dtype=torch.int32)
    table[0, :2] = torch.tensor([pages - 1, pages - 2])
    cache = ba.HistoryCache.empty(pages, size, heads, D, table.cuda())
    assert cache.k.numel() > 1 << 32
    rng = np.random.default_rng(1)
    x = [torch.from_numpy(rng.normal(size=(200, heads, D))).to(torch.bfloat16) for _ in "kv"]
    ba.cache_write(cache, x[0].cuda(), x[1].cuda(), i32([0, 200]), i32([0]))
    k, v = ba.cache_read(cache, i32([0, 200]), i32([0]), 200, dtype=torch.float32)
    for got, t in ((k, x[0]), (v, x[1])):
        el, e = C.quantize(f64(t))
        assert np.array_equal(f64(got), el * np.repeat(np.exp2(e), 32, axis=-1))
    q = queries(rng, 11, heads, D)
    last = [t[pages - 2:].cpu().numpy() for t in (cache.k, cache.v, cache.k_scales, cache.v_scales)]
    ref = C.Cache(*last, np.array([[1, 0, -1]]))
    for rows in (1, 11):
        got = ba.cache_attention_fwd(cache, q[:rows].cuda(), i32([0, rows]), i32([200 - rows]), 1 << 20, 1)
        check_attention(got, C.attend(ref, f64(q[:rows]), [0, rows], [200 - rows], 1 << 20, 1), D)
    mean = torch.zeros((pages, heads, D), device="cuda")
    ba.cache_summarize(cache, i32([0]), i32([200]), mean)
    want = ref.k[1].mean(axis=1)
    assert np.all(np.abs(f64(mean[pages - 1]) - want) <= size * 2.0 ** -24 * np.abs(ref.k[1]).mean(axis=1))
    assert not mean[:pages - 1].any()
    assert ba.ba_device_status(cache.status) == ba.BA_OK


# Sequences whose rows take several tiles of 8 or 16 rows, beside ones with a row or none.
MIDDLE = [
    # D, size, kv, group, lens, rows, block, window, kind, selected
    (128, 64, 1, 4, [900, 333], [3, 4], 256, 2, "chain", 0),
    (64, 16, 2, 3, [200, 50, 0], [5, 4, 3], 32, 1, "tree", 0),
    (128, 16, 1, 1, [300, 40, 40, 40], [30, 1, 1, 1], 64, 1, "tree", 3),
    (64, 128, 1, 2, [600, 100, 5], [20, 1, 1], 128, 1, "candidates", 2),
    (64, 32, 1, 1, [400, 9, 9], [17, 1, 0], 64, 1, "ragged", 4),
    (128, 32, 3, 1, [0], [12], 16, 3, "ragged", 0),
    (128, 128, 1, 2, [513, 128], [1, 6], 1 << 20, 1, "chain", 0),
    (128, 64, 2, 1, [64, 700], [33, 0], 96, 1, "past", 0),
    (64, 16, 1, 2, [90, 17, 256], [4, 2, 9], 32, 2, "past", 3),
    (128, 16, 1, 1, [90, 17, 256], [4, 2, 9], 32, 2, "past", 0),
    (64, 64, 2, 1, [500, 1, 70], [1, 1, 1], 64, 1, "past", 2),
]


@pytest.mark.parametrize("D,size,kv,group,lens,n,block,window,kind,selected", MIDDLE)
def test_attention_of_uneven_batches(D, size, kv, group, lens, n, block, window, kind, selected):
    if kind != "past":
        test_attention_matches_the_oracle(D, size, kv, group, lens, n, block, window, kind, selected, 2.0)
        return
    # positions in any order, before the history's end and before its start, without a tree
    cache, ref, rng = build(D + size + len(n), [a + b for a, b in zip(lens, n)], kv, D, size)
    rows, offs = sum(n), offsets(n)
    q = queries(rng, rows, kv * group, D)
    pos = [int(rng.integers(-2, lens[b] + n[b])) for b in range(len(n)) for _ in range(n[b])]
    mask = None
    if selected:
        mask = C.words(rng.random((rows, kv, ref.table.shape[1])) < selected / ref.table.shape[1])
    got = ba.cache_attention_fwd(cache, q.cuda(), i32(offs), i32(lens), block, window, positions=i32(pos),
                                 page_mask=None if mask is None else i32(mask))
    assert ba.ba_device_status(cache.status) == ba.BA_OK
    check_attention(got, C.attend(ref, f64(q), offs, lens, block, window, pos, None, mask), D)


@pytest.mark.parametrize("rows,D", [(5, 128), (5, 64), (7, 128), (7, 64)])
def test_long_cache_split_over_blocks_of_8_and_16_rows(rows, D):
    test_long_cache_split_over_blocks(rows, D)


ROWS = [1, 6, 12, 40]   # of one sequence: each of the attention's kernels


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("rows", ROWS)
def test_values_and_keys_of_any_scale(rows, D):
    """Scales over the whole range, past those the fast widening knows and below bf16's normal numbers."""
    cache, ref, rng = build(rows + D, [90 + rows], 2, D, 32)
    for t, low, high in ((cache.v_scales, 0, 200), (cache.k_scales, 90, 131)):
        old = t.cpu()
        some = torch.from_numpy(rng.random(tuple(old.shape)) < 0.3)
        old[some] = torch.from_numpy(rng.integers(low, high, tuple(old.shape)).astype(np.uint8))[some]
        t.copy_(old)
    ref = C.Cache(*(t.cpu().numpy() for t in (cache.k, cache.v, cache.k_scales, cache.v_scales, cache.page_table)))
    q = queries(rng, rows, 2, D)
    got = ba.cache_attention_fwd(cache, q.cuda(), i32([0, rows]), i32([90]), 1 << 20, 1)
    # Values reach 2^73 * 448 here while scores differ by hundreds, so what float32's range leaves out counts: a
    # probability below 2^-126 of its reference becomes 0, and so does a warp's or a split's weight. A reference is
    # at most 2^8 below the largest score, the final sum at least 1, so each of the three loses at most
    # 2^8 2^-126 |v| of a slot: 3 2^-118 sum |v| in all.
    seen = np.stack([ref.v[ref.slot(0, p)[0], :, ref.slot(0, p)[1]] for p in range(90 + rows)])
    check_attention(got, C.attend(ref, f64(q), [0, rows], [90], 1 << 20, 1), D,
                    more=3 * 2.0 ** -118 * np.abs(seen).sum(axis=0))


@pytest.mark.parametrize("rows", ROWS[1:])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_a_query_row_that_is_not_finite_reaches_no_other(rows, value):
    lens = [400]
    cache, ref, rng = build(rows, [400 + rows], 1, 128, 64)
    q = queries(rng, rows, 1, 128)
    mask = C.words(rng.random((rows, 1, ref.table.shape[1])) < 0.5)
    args = (i32([0, rows]), i32(lens), 64, 2)
    clean = ba.cache_attention_fwd(cache, q.cuda(), *args, page_mask=i32(mask))
    mean = torch.from_numpy(rng.normal(size=(ref.k.shape[0], 1, 128))).float().cuda()
    chosen = ba.cache_select(cache, q.cuda(), *args[:2], mean, 64, 1, 2)
    q[2, 0, 7] = value
    got = ba.cache_attention_fwd(cache, q.cuda(), *args, page_mask=i32(mask))
    rest = [t for t in range(rows) if t != 2]
    assert torch.equal(got[0][rest], clean[0][rest]) and torch.equal(got[1][:, rest], clean[1][:, rest])
    assert torch.isnan(got[0][2]).all()
    assert torch.equal(ba.cache_select(cache, q.cuda(), *args[:2], mean, 64, 1, 2)[rest], chosen[rest])


@pytest.mark.parametrize("rows", ROWS)
def test_sequences_that_share_pages(rows):
    """Two sequences on the same pages of a common beginning, with pages of their own after it."""
    cache, ref, rng = build(rows, [128 + rows, 96 + rows], 1, 128, 32)
    cache.page_table[1, :3] = cache.page_table[0, :3]
    ref.table[1, :3] = ref.table[0, :3]
    n, lens = [rows, rows], [128, 96]
    q = queries(rng, 2 * rows, 1, 128)
    mean = torch.zeros((ref.k.shape[0], 1, 128), device="cuda")
    ba.cache_summarize(cache, i32([0, 0]), i32(lens), mean)
    want = C.summarize(ref, [0, 0], lens, np.zeros(mean.shape))
    mag = np.maximum(np.abs(ref.k).mean(axis=2), 1e-30)
    assert np.all(np.abs(f64(mean) - want) <= 32 * 2.0 ** -24 * mag)
    got = ba.cache_attention_fwd(cache, q.cuda(), i32(offsets(n)), i32(lens), 64, 2)
    check_attention(got, C.attend(ref, f64(q), offsets(n), lens, 64, 2), 128)
    k, v = ba.cache_read(cache, i32([0, 96, 192]), i32([0, 0]), 192)
    assert torch.equal(k[:96], k[96:]) and torch.equal(v[:96], v[96:])
    assert ba.ba_device_status(cache.status) == ba.BA_OK


@pytest.mark.parametrize("rows", ROWS)
def test_rows_behind_the_last_sequence_of_a_padded_batch(rows):
    """Tensors longer than the offsets say: what belongs to the rest stays as it was, split or not."""
    lens, spare = [6000], 5
    cache, ref, rng = build(rows, [6000 + rows], 1, 64, 16, extra_pages=3, spare=2)
    offs = i32([0, rows])
    q = queries(rng, rows + spare, 1, 64).cuda()
    mean = torch.from_numpy(rng.normal(size=(ref.k.shape[0], 1, 64))).float().cuda()
    for block, split in ((1 << 20, True), (64, False)):
        assert (ba.ba_cache_fwd_workspace_size(cache, ba.make_problem(q, offs), block, 1) > 0) or not split
        out = torch.full_like(q, 9.0)
        lse = torch.full((1, rows + spare), 9.0, device="cuda")
        ba.cache_attention_fwd(cache, q, offs, i32(lens), block, 1, out=out, lse=lse)
        assert torch.all(out[rows:] == 9.0) and torch.all(lse[:, rows:] == 9.0)
        alone = ba.cache_attention_fwd(cache, q[:rows].contiguous(), offs, i32(lens), block, 1)
        assert torch.isfinite(alone[1]).all() and torch.allclose(alone[1], lse[:, :rows], atol=1e-4)
    mask = torch.full((rows + spare, 1, -(-ref.table.shape[1] // 32)), 9, dtype=torch.int32, device="cuda")
    ba.cache_select(cache, q, offs, i32(lens), mean, 64, 1, 3, page_mask=mask)
    assert torch.all(mask[rows:] == 9)
    want = C.select(ref, f64(q[:rows]), [0, rows], lens, f64(mean), 64, 1, 3)
    assert np.array_equal(mask[:rows].cpu().numpy(), C.words(want))
    k, v = (torch.full((rows + spare, 1, 64), 9.0, device="cuda") for _ in "kv")
    ba.cache_read(cache, offs, i32(lens), rows + spare, k=k, v=v)
    assert torch.all(k[rows:] == 9.0) and torch.all(v[rows:] == 9.0) and not torch.any(k[:rows] == 9.0)
    before = cache.k.clone()
    ba.cache_write(cache, k, v, offs, i32(lens))
    assert torch.equal(cache.k.view(torch.float8_e4m3fn).float(), before.view(torch.float8_e4m3fn).float())
    assert ba.ba_device_status(cache.status) == ba.BA_OK


@pytest.mark.parametrize("group,most", [(1, 1), (2, 4), (6, 4), (16, 4)], ids=["one", "eight", "sixteen", "many"])
def test_many_sequences_some_of_them_empty(group, most):
    """More sequences than two levels of the blocks' search cover, with and without rows and histories."""
    batch = 1100
    rng = np.random.default_rng(group)
    n = rng.integers(0, most + 1, batch)
    lens = rng.integers(0, 40, batch) * (rng.random(batch) < 0.8)
    cache, ref, rng = build(group, lens + n, 1, 64, 16, spare=0)
    rows, offs = int(n.sum()), offsets(n)
    q = queries(rng, rows, group, 64)
    got = ba.cache_attention_fwd(cache, q.cuda(), i32(offs), i32(lens), 16, 1)
    check_attention(got, C.attend(ref, f64(q), offs, lens, 16, 1), 64)
    mean = torch.from_numpy(rng.normal(size=(ref.k.shape[0], 1, 64))).float()
    mask = ba.cache_select(cache, q.cuda(), i32(offs), i32(lens), mean.cuda(), 16, 1, 1)
    assert np.array_equal(mask.cpu().numpy(), C.words(C.select(ref, f64(q), offs, lens, f64(mean), 16, 1, 1)))
    k, v = ba.cache_read(cache, i32(offs), i32(lens), rows)
    b, t = np.repeat(np.arange(batch), n), np.concatenate([np.arange(x) for x in n])
    p = lens[b] + t
    at = ref.table[b, p // 16], p % 16
    assert np.array_equal(f64(k)[:, 0], ref.k[at[0], 0, at[1]]) and np.array_equal(f64(v)[:, 0], ref.v[at[0], 0, at[1]])
    assert ba.ba_device_status(cache.status) == ba.BA_OK


@pytest.mark.parametrize("rows,pages", [(1, 16384), (9, 16384), (9, 2048)])
def test_select_of_the_most_pages(rows, pages):
    table = torch.arange(pages, dtype=torch.int32).flip(0).reshape(1, pages).contiguous().cuda()
    cache = ba.HistoryCache.empty(pages, 16, 1, 64, table)
    rng = np.random.default_rng(pages)
    q = queries(rng, rows, 2, 64)
    mean = torch.from_numpy(rng.normal(size=(pages, 1, 64))).float()
    mean[7] = mean[pages - 9]
    lens = [16 * pages - rows]
    ref = C.Cache(*(t[:, :, :1].cpu().numpy() for t in (cache.k, cache.v, cache.k_scales, cache.v_scales)), table.cpu())
    ref.size = 16
    for topk in (1, 40, pages // 2):
        got = ba.cache_select(cache, q.cuda(), i32([0, rows]), i32(lens), mean.cuda(), 64, 1, topk)
        want = C.select(ref, f64(q), [0, rows], lens, f64(mean), 64, 1, topk)
        assert np.array_equal(got.cpu().numpy(), C.words(want)), topk
    assert ba.ba_device_status(cache.status) == ba.BA_OK


def test_nan_in_a_value_column_of_many_rows():
    lens = [100]
    cache, ref, rng = build(4, [140], 1, 128, 16)
    tree, pos = tree_case(rng, lens, [40], "candidates")
    q = queries(rng, 40, 1, 128)
    args = (q.cuda(), i32([0, 40]), i32(lens), 32, 2)
    kw = dict(positions=i32(pos), tree_mask=i32(tree))
    clean = ba.cache_attention_fwd(cache, *args, **kw)
    page, at = ref.slot(0, 103)
    cache.v[page, 0, at, 77] = 0x7F
    got = ba.cache_attention_fwd(cache, *args, **kw)
    same = torch.ones_like(clean[0], dtype=torch.bool)
    same[3, 0, 77] = False
    assert torch.equal(got[0][same], clean[0][same]) and torch.equal(got[1], clean[1])
    assert torch.isnan(got[0][3, 0, 77])


def test_element_offsets_past_32_bits_of_bulk_copies():
    pages, size, heads, D = 70000, 128, 4, 128
    table = torch.tensor([[pages - 1, pages - 2]], dtype=torch.int32)
    cache = ba.HistoryCache.empty(pages, size, heads, D, table.cuda())
    rng = np.random.default_rng(2)
    x = [torch.from_numpy(rng.normal(size=(230, heads, D))).to(torch.bfloat16).cuda() for _ in "kv"]
    ba.cache_write(cache, x[0], x[1], i32([0, 230]), i32([0]))
    last = [t[pages - 2:].cpu().numpy() for t in (cache.k, cache.v, cache.k_scales, cache.v_scales)]
    ref = C.Cache(*last, np.array([[1, 0]]))
    q = queries(rng, 30, heads, D)
    got = ba.cache_attention_fwd(cache, q.cuda(), i32([0, 30]), i32([200]), 1 << 20, 1)
    check_attention(got, C.attend(ref, f64(q), [0, 30], [200], 1 << 20, 1), D)
    assert ba.ba_device_status(cache.status) == ba.BA_OK


# ------------------------------------------------------------- used together ---

def test_a_history_served_step_by_step():
    """Prompt written and attended in one call, events appended one by one, pages averaged as they fill,
    then drafted events: every step equals the oracle on the cache as it is, and the prompt's rows equal
    ba_fwd on the rows read back."""
    heads, D, size, block, window = 2, 128, 16, 32, 2
    lens = np.array([70, 33, 0])
    table = torch.arange(3 * 8, dtype=torch.int32).reshape(3, 8)[:, torch.randperm(8)].contiguous().cuda()
    cache = ba.HistoryCache.empty(24, size, heads, D, table)
    mean = torch.zeros((24, heads, D), device="cuda")
    rng = np.random.default_rng(12)

    def oracle_cache():
        return C.Cache(*(t.cpu().numpy() for t in (cache.k, cache.v, cache.k_scales, cache.v_scales, table)))

    offs = offsets(lens)
    k, v = (queries(rng, int(offs[-1]), heads, D).cuda() for _ in "kv")
    q = queries(rng, int(offs[-1]), heads, D)
    zero = i32([0, 0, 0])
    ba.cache_write(cache, k, v, i32(offs), zero)
    ba.cache_summarize(cache, zero, i32(lens), mean)
    out, lse = ba.cache_attention_fwd(cache, q.cuda(), i32(offs), zero, block, window)
    check_attention((out, lse), C.attend(oracle_cache(), f64(q), offs, [0, 0, 0], block, window), D)
    kr, vr = ba.cache_read(cache, i32(offs), zero, int(offs[-1]))
    dense, dense_lse = ba.block_attention_fwd(q.cuda(), kr, vr, i32(offs), block, window)
    # two roundings to bf16 and two bf16 P apart: twice the bound
    tol, tol_lse = attention_bound(C.attend(oracle_cache(), f64(q), offs, [0, 0, 0], block, window), D)
    assert np.all(np.abs(f64(out) - f64(dense)) <= 2 * tol)
    # the dense forward's lse is held to 2e-3 by its own parity tests
    assert np.all(np.abs(f64(lse) - f64(dense_lse)) <= 2e-3 + tol_lse)
    one = i32([0, 1, 2, 3])
    for step in range(20):
        ks, vs, qs = (queries(rng, 3, heads, D) for _ in "kvq")
        ba.cache_write(cache, ks.cuda(), vs.cuda(), one, i32(lens))
        ba.cache_summarize(cache, i32(lens), i32(lens + 1), mean)
        mask = ba.cache_select(cache, qs.cuda(), one, i32(lens), mean, block, window, 1)
        out, lse = ba.cache_attention_fwd(cache, qs.cuda(), one, i32(lens), block, window, page_mask=mask)
        if step % 5 == 4:
            ref = oracle_cache()
            want_mean = C.summarize(ref, [0, 0, 0], lens + 1, np.zeros(mean.shape))
            assert np.all(np.abs(f64(mean) - want_mean) <= size * 2.0 ** -24 * 4)
            chosen = C.select(ref, f64(qs), [0, 1, 2, 3], lens, f64(mean), block, window, 1)
            assert np.array_equal(mask.cpu().numpy(), C.words(chosen))
            check_attention((out, lse), C.attend(ref, f64(qs), [0, 1, 2, 3], lens, block, window,
                                                 mask=C.words(chosen)), D)
        lens = lens + 1
    n = [7, 12, 4]
    tree, pos = tree_case(rng, list(lens), n, "tree")
    offs = offsets(n)
    kd, vd, qd = (queries(rng, sum(n), heads, D) for _ in "kvq")
    ba.cache_write(cache, kd.cuda(), vd.cuda(), i32(offs), i32(lens))
    got = ba.cache_attention_fwd(cache, qd.cuda(), i32(offs), i32(lens), block, window, positions=i32(pos),
                                 tree_mask=i32(tree))
    check_attention(got, C.attend(oracle_cache(), f64(qd), offs, lens, block, window, pos, tree), D)
    assert ba.ba_device_status(cache.status) == ba.BA_OK


@pytest.mark.parametrize("rows", [1, 24])
def test_captured_into_a_graph_and_replayed_on_another_stream(rows):
    """One graph of write, summarize, select and attention, replayed while lengths and inputs change."""
    lens = torch.tensor([2000, 1500], dtype=torch.int32)
    cache, _, rng = build(rows, [2100, 1600], 2, 128, 16)
    n = [rows, rows]
    offs = i32(offsets(n))
    mean = torch.zeros((cache.k.shape[0], 2, 128), device="cuda")
    ba.cache_summarize(cache, i32([0, 0]), lens.cuda(), mean)
    q, k, v = (queries(rng, 2 * rows, h, 128).cuda() for h in (4, 2, 2))
    dl, de = lens.cuda(), (lens + rows).cuda()
    mask = torch.zeros((2 * rows, 2, -(-cache.page_table.shape[1] // 32)), dtype=torch.int32, device="cuda")
    out, lse = torch.empty_like(q), torch.empty((4, 2 * rows), device="cuda")
    ws = ba.workspace_for(ba.ba_cache_fwd_workspace_size(cache, ba.make_problem(q, offs), 64, 1), "cuda")

    def step():
        ba.cache_write(cache, k, v, offs, dl)
        ba.cache_summarize(cache, dl, de, mean)
        ba.cache_select(cache, q, offs, dl, mean, 64, 1, 4, page_mask=mask)
        ba.cache_attention_fwd(cache, q, offs, dl, 64, 1, page_mask=mask, out=out, lse=lse, workspace=ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(3):
        q.copy_(queries(rng, 2 * rows, 4, 128))
        k.copy_(queries(rng, 2 * rows, 2, 128))
        dl.add_(7)
        de.add_(7)
        graph.replay()
        a = [t.clone() for t in (mask, out, lse, cache.k, mean)]
        step()
        torch.cuda.synchronize()
        for x, y in zip(a, (mask, out, lse, cache.k, mean)):
            assert torch.equal(x, y)
    assert ba.ba_device_status(cache.status) == ba.BA_OK


def test_two_streams_at_once():
    """Two attentions over one cache at the same time, each with its own workspace, equal the calls one by one."""
    cache, _, rng = build(21, [5000, 4000], 2, 128, 64)
    args = []
    for rows in (1, 40):
        q = queries(rng, 2 * rows, 2, 128).cuda()
        args.append((q, i32([0, rows, 2 * rows]), i32([4900, 3900])))
    want = [ba.cache_attention_fwd(cache, *a, 1 << 20, 1) for a in args]
    streams = [torch.cuda.Stream() for _ in args]
    torch.cuda.synchronize()
    got = []
    for _ in range(3):
        got = []
        for s, a in zip(streams, args):
            with torch.cuda.stream(s):
                got.append(ba.cache_attention_fwd(cache, *a, 1 << 20, 1))
    torch.cuda.synchronize()
    for x, y in zip(got, want):
        assert torch.equal(x[0], y[0]) and torch.equal(x[1], y[1])
    # an explicit stream argument
    q, offs, lens = args[0]
    out, lse = torch.empty_like(q), torch.empty((2, 2), device="cuda")
    ws = ba.workspace_for(ba.ba_cache_fwd_workspace_size(cache, ba.make_problem(q, offs), 1 << 20, 1), "cuda")
    ba.cache_attention_fwd(cache, q, offs, lens, 1 << 20, 1, out=out, lse=lse, workspace=ws, stream=streams[0])
    streams[0].synchronize()
    assert torch.equal(out, want[0][0])


@pytest.mark.parametrize("rows", ROWS)
def test_two_graphs_share_a_workspace(rows):
    """Two captured calls over different caches and one workspace, replayed in turn on a stream of their own."""
    made = []
    for seed in (rows, rows + 50):
        cache, _, rng = build(seed, [4000 + rows], 1, 128, 64)
        q = queries(rng, rows, 1, 128).cuda()
        made.append((cache, q, i32([0, rows]), i32([4000])))
    want = [ba.cache_attention_fwd(*m, 1 << 20, 1) for m in made]
    need = max(ba.ba_cache_fwd_workspace_size(m[0], ba.make_problem(m[1], m[2]), 1 << 20, 1) for m in made)
    assert need > 0
    ws = ba.workspace_for(need, "cuda")
    outs = [(torch.empty_like(m[1]), torch.empty((1, rows), device="cuda")) for m in made]
    graphs = []
    torch.cuda.synchronize()
    for m, (out, lse) in zip(made, outs):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            ba.cache_attention_fwd(*m, 1 << 20, 1, out=out, lse=lse, workspace=ws)
        graphs.append(graph)
    side = torch.cuda.Stream()
    for _ in range(3):
        with torch.cuda.stream(side):
            for (out, lse), graph in zip(outs, graphs):
                out.zero_()
                graph.replay()
        side.synchronize()
        for (out, lse), w in zip(outs, want):
            assert torch.equal(out, w[0]) and torch.equal(lse, w[1])


def test_the_binding_refuses_what_does_not_fit():
    cache, _, rng = build(1, [40, 20], 2, 64, 16)
    q, offs, lens = queries(rng, 2, 4, 64).cuda(), i32([0, 1, 2]), i32([39, 19])
    ok = ba.cache_attention_fwd(cache, q, offs, lens, 16, 1)
    assert ok[0].shape == q.shape
    bad = [dict(q=q.float()), dict(q=q[:, :3].contiguous()), dict(q=q[..., :32].contiguous()), dict(q=q.cpu()),
           dict(q=q.transpose(0, 1)), dict(lens=lens.long()), dict(lens=lens[:1]), dict(offs=offs[:2])]
    for kw in bad:
        a = dict(q=q, offs=offs, lens=lens)
        a.update(kw)
        with pytest.raises(ValueError):
            ba.cache_attention_fwd(cache, a["q"], a["offs"], a["lens"], 16, 1)
        with pytest.raises(ValueError):
            ba.cache_select(cache, a["q"], a["offs"], a["lens"], torch.zeros((cache.k.shape[0], 2, 64), device="cuda"),
                            16, 1, 2)
    for kw in (dict(workspace=torch.empty(1 << 20, dtype=torch.uint8)), dict(tree_mask=i32([[], []])),
               dict(positions=i32([1])), dict(tree_mask=i32([1, 1])), dict(page_mask=i32([[1], [1]])),
               dict(out=q.float()), dict(lse=torch.zeros(2, 2, device="cuda"))):
        with pytest.raises(ValueError):
            ba.cache_attention_fwd(cache, q, offs, lens, 16, 1, **kw)
    x = torch.zeros((2, 2, 64), device="cuda")
    for k, v in ((x.half(), x.half()), (x, x.bfloat16()), (x[:, :1], x[:, :1]), (x, x[:1])):
        with pytest.raises(ValueError):
            ba.cache_write(cache, k, v, offs, lens)
    with pytest.raises(ValueError):
        ba.cache_read(cache, offs, lens, 2, k=x)
    with pytest.raises(ValueError):
        ba.cache_read(cache, offs, lens, 3, k=x, v=x)
    with pytest.raises(ValueError):
        ba.cache_summarize(cache, lens, lens, x)
    with pytest.raises(ba.BAError):
        ba.cache_attention_fwd(cache, q, offs, lens, 0, 1)
    with pytest.raises(ba.BAError):
        ba.cache_select(cache, q, offs, lens, torch.zeros((cache.k.shape[0], 2, 64), device="cuda"), 16, 1, 0)
