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


@pytest.mark.parametrize("heads", [8, 128])
@pytest.mark.parametrize("short", [0, 5])
def test_absorbed_longest_context(heads, short):
    """2^31 - 64 keys, all in two blocks: the first block's score 0 and hold 1 in dim 0,
    the last one's score 30 (to base 2) and hold 1 in dim 1.  Every number in the sums is
    exact, so only the quotient and its rounding to bf16 are off."""
    blocks = 2 ** 27 - 4
    L = 16 * blocks - short
    tables = torch.zeros(1, blocks, dtype=torch.int32, device="cuda")
    tables[0, -1] = 1
    cache = torch.zeros(2, 16, 576, dtype=torch.bfloat16, device="cuda")
    cache[0, :, 0], cache[1, :, 1], cache[1, :, 512] = 1.0, 1.0, 30.0
    if short:
        cache[1, 16 - short:] = float("nan")
    q = torch.zeros(1, heads, 576, dtype=torch.bfloat16, device="cuda")
    q[:, :, 512] = 1.0
    out = torch.full((1, heads, 512), float("nan"), dtype=torch.bfloat16, device="cuda")
    pkv.paged_latent_attention(out, q, cache, tables, torch.tensor([L], dtype=torch.int32, device="cuda"),
                               scale=float(np.log(2.0)))
    assert pkv.kv_last_device_status() == 0
    got, last = f64(out)[0], 2.0 ** 30 * (16 - short)
    exp = np.array([16.0 * (blocks - 1), last]) / (16.0 * (blocks - 1) + last)
    # (30 x scale x log2(e) in fp32 is 30 up to 2^-18, the exponential's weight up to as much)
    assert (np.abs(got[:, :2] - exp) <= exp * (2.0 ** -8 + 2.0 ** -16)).all(), (got[0, :2], exp)
    assert (got[:, 2:] == 0).all()
