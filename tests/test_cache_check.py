"""The attention tests' own comparison, without a GPU: what it must not let pass."""
import numpy as np
import pytest

from cache_util import check


def sample():
    rng = np.random.default_rng(0)
    out, lse = rng.normal(size=(3, 2, 8)), rng.normal(size=(2, 3))
    out[1], lse[:, 1] = 0.0, -np.inf
    return out, lse, np.abs(out), np.ones((2, 3))


def test_equal_results_pass():
    ref = sample()
    check(ref[:2], ref, 8)


@pytest.mark.parametrize("value", [np.nan, np.inf, -np.inf, 9.0])
@pytest.mark.parametrize("where", ["out", "unseen out", "lse", "unseen lse"])
def test_wrong_results_fail(where, value):
    ref = sample()
    out, lse = ref[0].copy(), ref[1].copy()
    if where.endswith("out"):
        out[1 if "unseen" in where else 2, 1, 3] = value
    else:
        lse[0, 1 if "unseen" in where else 2] = value
    if where == "unseen lse" and value == -np.inf:
        return   # that is right
    with pytest.raises(AssertionError):
        check((out, lse), ref, 8)
