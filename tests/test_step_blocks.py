"""Blocks and slots of a step (zp_step_slots): the largest step."""
import os

import pytest
import torch


@pytest.fixture(scope="module")
def zp():
    from paged_kv_cache_obs_gb300 import build
    if not os.path.exists(build.LIB):
        build.build()
    from paged_kv_cache_obs_gb300 import zipage
    return zipage


def _params(b=16):
    return dict(num_layers=1, num_q_heads=2, num_kv_heads=2, head_dim=64, block_size=b, n_max=4, window=1, alpha=0.5, beta=0.5, decay=0.9,
                scale=0.125, protect_window=1, causal=1)


@pytest.mark.gpu
def test_as_many_rows_as_there_are_numbers(zp):
    """2^31 - 1 rows of two requests: every row has its slot, and nothing else is written."""
    b, T, half = 32, 2 ** 31 - 1, 2 ** 30
    NB = T // b
    i32 = dict(dtype=torch.int32, device="cuda")
    free = torch.arange(NB + 1, **i32)
    free[NB] = 0                                       # the last block stands beside the first: there are no more ids
    tables, start, seq = torch.full((2, half // b), -1, **i32), torch.empty(3, **i32), torch.empty(2, **i32)
    buf, at, ws = torch.full((T + 1 + 2 * 4096,), 7, **i32), torch.zeros(1, **i32), zp.new_workspace(256)
    slots = buf[4096:4096 + T]
    zp.zp_step_slots(torch.zeros(2, **i32), torch.tensor([half, half - 1], **i32), free, tables, start, seq, slots, _params(b), ws,
                     num_blocks=NB, free_at=at)
    assert zp.zp_read_error(ws) == zp.ZP_OK and at.item() == NB + 1
    assert start.tolist() == [0, half, T] and seq.tolist() == [half, half - 1]
    assert torch.equal(tables.flatten(), free)
    for lo in range(0, NB * b, 1 << 28):
        hi = min(lo + (1 << 28), NB * b)
        assert torch.equal(slots[lo:hi], torch.arange(lo, hi, **i32))
    assert torch.equal(slots[NB * b:], torch.arange(T - NB * b, **i32))
    assert bool((buf[:4096] == 7).all()) and bool((buf[4096 + T:] == 7).all())
