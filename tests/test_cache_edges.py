"""GPU tests of the history cache where its calls meet less usual arguments: positions past the cache's slots,
splits with selected pages, padded batches. Bounds are test_cache.py's; a NaN fails them here."""
import numpy as np
import pytest
import torch

import block_sparse_attention_kunlun_b200 as ba
from oracle import cache as C
from parity_util import f64
from test_cache import ROWS, attention_bound, build, i32, offsets, queries

pytestmark = pytest.mark.gpu


def check(got, ref, D):
    """Attention within its bounds, and finite wherever the oracle's is."""
    out, lse = f64(got[0]), f64(got[1])
    tol_out, tol_lse = attention_bound(ref, D)
    assert np.isfinite(ref[0]).all()
    assert np.array_equal(np.isneginf(lse), np.isneginf(ref[1]))
    seen = np.isfinite(ref[1])
    assert np.all(np.abs(lse[seen] - ref[1][seen]) <= tol_lse[seen])
    assert np.all(np.abs(out - ref[0]) <= tol_out), np.argwhere(~(np.abs(out - ref[0]) <= tol_out))[:5]


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
