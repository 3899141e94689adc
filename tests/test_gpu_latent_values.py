"""Values of latent attention that are known without a reference: queries that are
not finite, values that are the same for every key."""
import numpy as np
import pytest
import torch

import paged_kv_cache_263_gb300 as pkv
from tests.gpu_util import require_gpu
from tests.test_gpu_latent import Paged, Prompt, check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    require_gpu()


# one unit a worker, units cut many times, several units a worker; both absorbed kernels
@pytest.mark.parametrize("heads,lens,rows", [
    (128, [40, 30], [1, 1]), (128, [3000, 70], [1, 1]), (96, [1500, 64, 200], [3, 1, 2]),
    (8, [40, 30], [1, 1]), (8, [6000, 70], [1, 1]), (16, [900, 64, 200], [3, 1, 2])])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_absorbed_queries_that_are_not_finite(heads, lens, rows, bad):
    """The product of such a query with finite keys of both signs is not finite for some
    key, so its row is NaN, however its context is cut; the other rows keep their bits."""
    w = Paged(heads, lens, rows, seed=heads)
    clean = w.run()
    assert np.isfinite(clean).all()
    for r, h in ((0, 0), (0, heads - 1), (w.q.shape[0] - 1, heads // 2)):
        w.q[r, h, 17] = bad
        got = w.run()
        assert np.isnan(got[r, h]).all()
        clean[r, h] = np.nan
        assert np.array_equal(got, clean, equal_nan=True)
    assert pkv.kv_last_device_status() == 0


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_expanded_queries_that_are_not_finite(bad):
    """(The other rows of a warp may move their references along, so their bits may change.)"""
    w = Prompt(3, [300, 5, 140], [700, 90, 140], seed=2)
    ref, tol = w.expected()
    for r, h in ((0, 0), (299, 1), (302, 2), (400, 1)):
        w.q[r, h, 100] = bad
        got = w.run()
        assert np.isnan(got[r, h]).all()
        ref[r, h] = np.nan
        check(got, ref, tol)
    assert pkv.kv_last_device_status() == 0
