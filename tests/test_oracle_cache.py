"""Pins of oracle/cache.py against independent statements: codes against torch's
E4M3, attention of a chain against the dense oracle on the dequantised rows, a
tree against its paths run as chains, page selection against a plain sort."""
import numpy as np
import pytest
import torch

import oracle
from oracle import cache as C
from oracle import mx as MX


def filled(rng, batch, heads, D, size, lengths, shuffle=True):
    """A cache of quantised normal rows; returns (Cache, k rows, v rows dequantised per sequence, codes)."""
    need = [-(-int(n) // size) for n in lengths]
    pages = sum(need) + 2
    ids = rng.permutation(pages) if shuffle else np.arange(pages)
    table = np.full((batch, max(max(need), 1) + 1), -1, dtype=np.int32)
    at = 0
    for b in range(batch):
        table[b, :need[b]] = ids[at:at + need[b]]
        at += need[b]
    el = [rng.integers(0, 120, (pages, heads, size, D)).astype(np.uint8) for _ in "kv"]
    el = [e | (rng.integers(0, 2, e.shape).astype(np.uint8) << 7) for e in el]
    sc = [rng.integers(116, 121, (pages, heads, size, D // 32)).astype(np.uint8) for _ in "kv"]
    return C.Cache(el[0], el[1], sc[0], sc[1], table)


def rows_of(cache, b, n):
    at = [cache.slot(b, p) for p in range(n)]
    return np.stack([cache.k[p, :, r] for p, r in at]), np.stack([cache.v[p, :, r] for p, r in at])


def test_codes_match_torch():
    c = np.arange(256, dtype=np.uint8)
    ref = torch.from_numpy(c).view(torch.float8_e4m3fn).to(torch.float64).numpy()
    got = C.e4m3_values(c)
    assert np.array_equal(np.isnan(got), np.isnan(ref)) and np.array_equal(got[~np.isnan(got)], ref[~np.isnan(ref)])
    assert np.array_equal(np.signbit(got[[0, 128]]), [False, True])


def test_quantize_round_trip_is_the_mx_oracle():
    x = np.random.default_rng(1).normal(size=(5, 3, 64))
    el, e = C.quantize(x)
    assert np.array_equal(el * np.repeat(np.exp2(e), 32, axis=-1), MX.mx_round(x))


@pytest.mark.parametrize("block,window,size", [(8, 1, 16), (16, 2, 16), (5, 3, 32), (1, 7, 16), (1000, 1, 16)])
def test_a_chain_is_block_attention_of_the_whole_history(block, window, size):
    rng = np.random.default_rng(block)
    lens, n = [0, 13, 40], [3, 1, 9]
    total = [a + b for a, b in zip(lens, n)]
    cache = filled(rng, 3, 2, 64, size, total)
    offs = np.concatenate([[0], np.cumsum(n)])
    q = rng.normal(size=(int(offs[-1]), 2, 64))
    out, lse, _, _ = C.attend(cache, q, offs, lens, block, window)
    for b in range(3):
        k, v = rows_of(cache, b, total[b])
        full = np.concatenate([np.zeros((lens[b], 2, 64)), q[offs[b]:offs[b + 1]]])
        ro, rl = oracle.fwd(np.array([0, total[b]], dtype=np.int32), full, k, v, block, window)
        np.testing.assert_allclose(out[offs[b]:offs[b + 1]], ro[lens[b]:], rtol=0, atol=1e-12)
        np.testing.assert_allclose(lse[:, offs[b]:offs[b + 1]], rl[:, lens[b]:], rtol=0, atol=1e-12)


def test_a_tree_is_its_paths():
    rng = np.random.default_rng(3)
    n, length, block, window = 7, 11, 4, 2
    parent = [-1, 0, 0, 1, -1, 2, 5]
    path = []
    for j in range(n):
        path.append((path[parent[j]] if parent[j] >= 0 else []) + [j])
    cache = filled(rng, 1, 2, 64, 16, [length + n])
    tree = np.zeros((n, n), dtype=bool)
    for j in range(n):
        tree[j, path[j]] = True
    pos = np.array([length + len(p) - 1 for p in path])
    q = rng.normal(size=(n, 4, 64))
    out, lse, _, _ = C.attend(cache, q, [0, n], [length], block, window, positions=pos, tree=C.words(tree))
    k, v = rows_of(cache, 0, length + n)
    for j in range(n):
        at = list(range(length)) + [length + i for i in path[j]]
        kk, vv = np.repeat(k[at], 2, axis=1), np.repeat(v[at], 2, axis=1)
        full = np.zeros((len(at), 4, 64))
        full[-1] = q[j]
        ro, rl = oracle.fwd(np.array([0, len(at)], dtype=np.int32), full, kk, vv, block, window)
        np.testing.assert_allclose(out[j], ro[-1], rtol=0, atol=1e-12)
        np.testing.assert_allclose(lse[:, j], rl[:, -1], rtol=0, atol=1e-12)


def test_selected_pages_add_to_the_window():
    """All pages selected: full causal attention; none: the window alone."""
    rng = np.random.default_rng(4)
    cache = filled(rng, 1, 1, 64, 16, [70])
    q = rng.normal(size=(2, 1, 64))
    every = C.words(np.ones((2, 1, cache.table.shape[1]), dtype=bool))
    a = C.attend(cache, q, [0, 2], [68], 8, 1, mask=every)
    b = C.attend(cache, q, [0, 2], [68], 1000, 1)
    # rows of the chain before the window are not added by page bits: 68, 69 are in one block of 8
    np.testing.assert_allclose(a[0], b[0], rtol=0, atol=1e-13)
    none = C.attend(cache, q, [0, 2], [68], 8, 1, mask=np.zeros_like(every))
    plain = C.attend(cache, q, [0, 2], [68], 8, 1)
    assert np.array_equal(none[0], plain[0]) and np.array_equal(none[1], plain[1])


def test_rows_that_see_nothing():
    rng = np.random.default_rng(5)
    cache = filled(rng, 1, 1, 64, 16, [20])
    q = rng.normal(size=(2, 1, 64))
    out, lse, _, _ = C.attend(cache, q, [0, 2], [0], 8, 1, positions=[-1, 0], tree=np.zeros((2, 1), dtype=np.int32))
    assert not out.any() and np.all(lse == -np.inf)


def test_select_against_a_sort_and_ties():
    rng = np.random.default_rng(6)
    cache = filled(rng, 1, 2, 64, 16, [200])
    mean = np.zeros((cache.k.shape[0], 2, 64))
    C.summarize(cache, [0], [200], mean)
    for c in range(200 // 16):
        np.testing.assert_allclose(mean[cache.table[0, c]], cache.k[cache.table[0, c]].sum(axis=1) / 16)
    q = rng.normal(size=(1, 4, 64))
    got = C.select(cache, q, [0, 1], [200], mean, 32, 1, 3)
    for h in range(2):
        score = [(q[0, 2 * h] + q[0, 2 * h + 1]) @ mean[cache.table[0, c], h] for c in range(12)]  # 192 = ws
        assert set(np.flatnonzero(got[0, h])) == set(np.argsort(score)[-3:])
    flat = C.select(cache, np.zeros((1, 4, 64)), [0, 1], [200], mean, 32, 1, 3)
    assert np.array_equal(np.flatnonzero(flat[0, 0]), [0, 1, 2])
    # fewer candidates than topk: all of them; a page that is not full is none
    assert C.select(cache, q, [0, 1], [100], mean, 32, 1, 50)[0, 0].sum() == 6  # ws = 96
    assert not C.select(cache, q, [0, 1], [20], mean, 32, 1, 50).any()


def test_words():
    bits = np.zeros((1, 40), dtype=bool)
    bits[0, [0, 31, 32, 39]] = True
    w = C.words(bits)
    assert w.shape == (1, 2) and [C.bit(w[0], i) for i in (0, 1, 31, 32, 39, 38, 64)] == [True, False, True, True,
                                                                                       True, False, False]
