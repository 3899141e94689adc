"""Limits of the latent operators that only sizes reach, without a GPU: the calls
below are refused before anything is launched, whatever the addresses."""
import pytest

from paged_kv_cache_263_gb300 import build as pkv_build
from tests.test_latent_args import ABS, INVALID, UNSUPPORTED, _call

MOST_BLOCKS = 2 ** 27 - 4       # the longest context's last tile of 64 keys ends at 2^31 - 64


@pytest.fixture(scope="module", autouse=True)
def built():
    pkv_build.build()


@pytest.mark.parametrize("blocks", [MOST_BLOCKS + 1, MOST_BLOCKS + 3])
def test_contexts_whose_last_tile_ends_past_32_bits(blocks):
    # (the scale is refused as well, later: nothing is launched either way)
    assert _call("paged_latent_attention", list(ABS), ABS, B=1, R=1, mb=blocks, scale=0.0) == UNSUPPORTED
    assert _call("paged_latent_attention", list(ABS), ABS, B=1, R=1, mb=MOST_BLOCKS, scale=0.0) == INVALID
