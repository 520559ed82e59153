"""How calls of attention over the 8-bit pool are cut, seen in the workspaces that they ask for (no GPU: plans are a GB300's)."""
import os

import pytest


@pytest.fixture(scope="module")
def zp():
    from paged_kv_cache_obs_gb300 import build
    if not os.path.exists(build.LIB):
        build.build()
    from paged_kv_cache_obs_gb300 import zipage
    return zipage


def _size(zp, Hq, Hkv, B, new, blocks, T=None, window=0):
    p = dict(num_layers=1, num_q_heads=Hq, num_kv_heads=Hkv, head_dim=128, block_size=16, n_max=4, window=1, alpha=0.5, beta=0.5, decay=0.9,
             scale=0.125, protect_window=1, causal=1)
    return zp.zp_kv8_window_workspace_size(p, T or B * new, B, new, blocks, window, 0)


@pytest.mark.parametrize("blocks", [512, 1024, 4096, 8192, 65536])
def test_a_wide_table_is_no_reason_for_parts(zp, blocks):
    """Calls whose items fill the SMs several times are not split, however wide a serving loop's table is."""
    for B, new in ((4, 2048), (32, 256), (64, 128), (16, 1000)):
        assert _size(zp, 32, 8, B, new, blocks) == 256


def test_few_items_are_split(zp):
    for B, new, blocks in ((8, 64, 6250), (1, 300, 1000), (2, 64, 8192)):
        T = B * new
        assert _size(zp, 28, 4, B, new, blocks) > 256 + T * 28 * 132 * 4
    # and no further than is worth it: 512 items of up to 2048 tiles in 2 parts
    assert _size(zp, 32, 8, 64, 64, 16384) == 256 + 2 * 64 * 64 * 32 * 132 * 4
