"""Blocks and slots of a step (zp_step_slots): tables that hold more blocks than the tokens fill, and the largest step."""
import os

import numpy as np
import pytest
import torch

from oracle import serving_oracle as S


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


# ------------------------------------------------------------------ blocks of tokens that were taken back

def _i32(x):
    return torch.as_tensor(np.ascontiguousarray(x), dtype=torch.int32).cuda()


def test_held_blocks_are_checked(zp):
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)
    good = dict(cached=i32(3), new_tokens=i32(3), free_ids=i32(5), block_tables=i32(3, 2), token_start=i32(4), seq_lens=i32(3), slots=i32(9),
                params=_params(), workspace=torch.zeros(256, dtype=torch.uint8), num_blocks=4, held_blocks=i32(3))
    for held in (i32(2), i32(3, 1, 2), i32(6)[::2], torch.zeros(3, dtype=torch.int64)):
        with pytest.raises(ValueError, match="expected"):
            zp.zp_step_slots(**{**good, "held_blocks": held})
    with pytest.raises(ValueError, match="current CUDA device"):
        zp.zp_step_slots(**good)
    ws = torch.zeros(4096, dtype=torch.uint8)
    base = (ws.data_ptr() + 255) // 256 * 256
    call = lambda T: zp.lib.zp_step_slots_held(base, base, None, base, 2, base, 4, None, 8, base, 2, base, base, None, base, T,
                                               zp.make_params(_params()), base, 256, None)
    assert call(-1) == zp.ZP_ERR_INVALID_ARG


def test_oracle_of_held_blocks_by_hand():
    """18 of 33 tokens stay: the third block, which the others had begun, is used again before a free one."""
    t = np.array([[7, 5, 2, -1, -1]], dtype=np.int32)
    got = S.step_slots([18], [32], [9, 4], t, 16, 33, 10, held=[3])
    assert got[0].tolist() == [[7, 5, 2, 9, -1]] and got[5:] == (1, None, [4]) and got[2] == [50]
    assert got[4] == list(range(82, 96)) + list(range(32, 48)) + [9 * 16, 9 * 16 + 1, -1]


def _run(zp, b, T, NB, cached, new, free, tables, held, at, in_place):
    B, ws = len(cached), zp.new_workspace(256)
    d = dict(cached=_i32(cached), new_tokens=_i32(new), free_ids=_i32(free), block_tables=_i32(tables), held_blocks=_i32(held), free_at=_i32([at]))
    for name, n in (("token_start", B + 1), ("slots", T), ("positions", T)):
        d[name] = torch.full((n,), 77, dtype=torch.int32, device="cuda")
    d["seq_lens"] = d["cached"] if in_place else torch.full((B,), 77, dtype=torch.int32, device="cuda")
    zp.zp_step_slots(params=_params(b), workspace=ws, num_blocks=NB, **d)
    want = S.step_slots(cached, new, free, tables, b, T, NB, free_at=at, held=held)
    for name, x in zip(("block_tables", "token_start", "seq_lens", "positions", "slots", "free_at"), want):
        assert np.array_equal(d[name].cpu().numpy(), np.asarray(x, dtype=np.int32).reshape(d[name].shape)), name
    assert d["held_blocks"].tolist() == [int(x) for x in want[7]]
    assert zp.zp_read_error(ws) == {None: zp.ZP_OK, "table": zp.ZP_ERR_BAD_TABLE, "blocks": zp.ZP_ERR_NO_BLOCKS}[want[6]]
    return want


@pytest.mark.gpu
@pytest.mark.parametrize("B,b,max_len,max_new,extra,pad", [(1, 16, 40, 5, 2, 0), (7, 32, 100, 90, 3, 4), (64, 16, 500, 4, 1, 9), (1024, 16, 60, 20, 2, 0),
                                                           (1100, 32, 60, 20, 2, 3), (40, 16, 900, 700, 20, 1), (3000, 16, 30, 9, 1, 2)])
def test_held_blocks_match_oracle(zp, B, b, max_len, max_new, extra, pad):
    rng = np.random.default_rng(B)
    cached = rng.integers(0, max_len + 1, B)
    new = np.where(rng.random(B) < 0.2, 0, rng.integers(0, max_new + 1, B))
    held = -(-cached // b) + rng.integers(0, extra + 1, B)
    mb = int(max(held.max(), (-(-(cached + new) // b)).max())) + 1
    need = int(np.maximum(0, -(-(cached + new) // b) - held).sum())
    NB = int(held.sum()) + need + 3
    ids, tables = rng.permutation(NB), np.full((B, mb), -7, dtype=np.int32)
    tables[np.arange(mb)[None] < held[:, None]] = ids[:held.sum()]
    free, T = ids[held.sum():].astype(np.int32), int(new.sum()) + pad
    for in_place in (False, True):
        assert _run(zp, b, T, NB, cached, new, free, tables, held, 1, in_place)[6] is None
    if need:                                           # one free id less than it takes
        assert _run(zp, b, T, NB, cached, new, free[:need - 1], tables, held, 0, True)[6] == "blocks"
    # tables that cannot hold what is said
    held[0], held[B - 1] = (mb + 1, mb + 1) if B == 1 else (mb + 1, -(-int(cached[B - 1]) // b) - 1)
    assert _run(zp, b, T, NB, cached, new, free, tables, held, 0, False)[6] == "table"


@pytest.mark.gpu
@pytest.mark.parametrize("counted", [True, False])
def test_a_captured_loop_of_drafts_loses_no_blocks(zp, counted):
    """Drafts of 4 tokens of which some are taken back, also those that begin a block, in a pool with as many blocks as the longest
    caches take.  Uncounted, ids of blocks that they had begun are lost, and the pool runs out."""
    rng = np.random.default_rng(9)
    B, b, most, steps, T = 6, 16, 4, 60, 24
    keep = rng.integers(0, most + 1, (steps, B))
    top = -(-(keep.sum(0) + most) // b)
    mb, NB = int(top.max()), int(top.sum())
    d = dict(cached=_i32(np.zeros(B)), new_tokens=_i32(np.full(B, most)), free_ids=_i32(rng.permutation(NB)), free_at=_i32([0]), token_start=_i32(np.zeros(B + 1)),
             block_tables=_i32(np.full((B, mb), -1)), slots=_i32(np.zeros(T)), held_blocks=_i32(np.zeros(B)) if counted else None)
    back, ws, p = _i32(np.zeros(B)), zp.new_workspace(256), _params(b)
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        d["cached"].sub_(back)                         # what the step before did not accept
        zp.zp_step_slots(seq_lens=d["cached"], params=p, workspace=ws, num_blocks=NB, **d)
    L, where, err = np.zeros(B, dtype=int), [{} for _ in range(B)], 0
    for s in range(steps):
        back.copy_(_i32(most - keep[s - 1] if s else np.zeros(B)))
        graph.replay()
        err = zp.zp_read_error(ws)
        if err:
            break
        slots = d["slots"].view(B, most).tolist()
        for r in range(B):
            for i in range(most):
                where[r][int(L[r]) + i] = slots[r][i]
        L += keep[s]
        for r in range(B):                             # tokens that stay have slots of their own
            where[r] = {t: x for t, x in where[r].items() if t < L[r]}
        taken = [x for w in where for x in w.values()]
        assert len(set(taken)) == len(taken) == int(L.sum())
    if counted:
        assert err == zp.ZP_OK and d["held_blocks"].tolist() == [-(-int(n + k) // b) for n, k in zip(L - keep[-1], np.full(B, most))]
        assert d["free_at"].item() == sum(d["held_blocks"].tolist()) <= NB
    else:
        assert err == zp.ZP_ERR_NO_BLOCKS
