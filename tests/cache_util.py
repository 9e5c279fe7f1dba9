"""The comparison of cache attention that NaN fails (no attention arithmetic here)."""
import numpy as np

from parity_util import f64
from test_cache import attention_bound


def check(got, ref, D, more=0.0):
    """out and lse within test_cache.py's bounds of the oracle's (which is finite, or -inf where a row sees nothing)."""
    out, lse = f64(got[0]), f64(got[1])
    tol_out, tol_lse = attention_bound(ref, D)
    assert np.isfinite(ref[0]).all()
    assert np.array_equal(np.isneginf(lse), np.isneginf(ref[1]))
    seen = np.isfinite(ref[1])
    assert np.all(np.abs(lse[seen] - ref[1][seen]) <= tol_lse[seen])
    bad = ~(np.abs(out - ref[0]) <= tol_out + more)
    assert not bad.any(), np.argwhere(bad)[:5]
