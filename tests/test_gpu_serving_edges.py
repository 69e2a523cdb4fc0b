"""GPU tests of the serving operators at their edges, against the same 64-bit
definitions (serving_reference.py) and with the same tolerances as
test_gpu_serving.py."""
import numpy as np
import pytest
import torch

from test_gpu_serving import check_decode, decode_state

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    from differential_attention_sm_b200 import binding
    binding.load()
    return binding


# ---- decode: windows that begin inside a stage ---------------------------------
@pytest.mark.parametrize("form", [1, 2])
@pytest.mark.parametrize("tile", [0, 1, 2, 3, 5, 7, 9, 33])
def test_window_before_the_first_tile_of_the_cache(B, form, tile):
    """One head and pages of one tile, taken in order from page 0 behind a
    window's first tile: what stands for the tiles before it is no neighbour of
    the cache's first tile."""
    n_tiles = tile + 9
    lens = [16 * n_tiles - 5]
    window = lens[0] - 16 * tile - 3
    cache, table, q, rng = decode_state(1, lens, 1, 16, form, seed=tile, spare=0,
                                        bad_tail=False)
    table[0, :n_tiles] = [n_tiles - tile + j for j in range(tile)] + list(range(n_tiles - tile))
    assert sorted(table[0, :n_tiles]) == list(range(n_tiles))
    check_decode(B, cache, table, lens, q, [0.4], form, window)
