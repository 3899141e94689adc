"""Absorbed latent attention at work: batches of several hundred key tiles, where
every worker runs its ring of stages and exchange slots many times over."""
import numpy as np
import pytest
import torch

import paged_kv_cache_263_gb300 as pkv
from tests.gpu_util import require_gpu
from tests.test_gpu_latent import Paged, check, f64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    require_gpu()


@pytest.mark.parametrize("heads,lens,rows", [
    (48, [500, 900, 1300, 130, 64, 700], [90, 70, 20, 90, 64, 5]), (128, [2000, 300, 1500], [9, 20, 1])])
def test_absorbed_masked_tiles_repeat_exactly(heads, lens, rows):
    """Chunks whose rows see different numbers of keys: the tiles at their ends are masked,
    and the exchange slots that carry them are used again at once."""
    w = Paged(heads, lens, rows, seed=heads)
    got = w.run()
    check(got, *w.expected())
    args, first = w.args(), w.out.clone().view(torch.int16)
    for _ in range(30):
        w.out.fill_(float("nan"))
        pkv.paged_latent_attention(**args)
        assert torch.equal(w.out.view(torch.int16), first)
    assert pkv.kv_last_device_status() == 0
