"""A step's blocks, slots and positions (zp_step_slots), cache writes by slot (zp_kv_append), and the two together."""
import ctypes
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


def _params(b=16, Hkv=2, d=64, layers=1, Hq=None):
    return dict(num_layers=layers, num_q_heads=Hq or Hkv, num_kv_heads=Hkv, head_dim=d, block_size=b, n_max=4, window=1, alpha=0.5,
                beta=0.5, decay=0.9, scale=0.125, protect_window=1, causal=1)


# ------------------------------------------------------------------ refusals (CPU) ------------

def test_slots_refuses(zp):
    ws = torch.zeros(4096, dtype=torch.uint8)
    base = (ws.data_ptr() + 255) // 256 * 256

    def call(cached=base, new=base, first=None, B=2, free=base, nf=4, at=None, nb=8, tables=base, mb=2, start=base, seq=base, pos=None,
             slots=base, T=4, params=zp.make_params(_params()), w=base, bytes=256):
        return zp.lib.zp_step_slots(cached, new, first, B, free, nf, at, nb, tables, mb, start, seq, pos, slots, T, params, w, bytes, None)

    for kw in (dict(params=None), dict(B=-1), dict(T=-1), dict(nf=-1), dict(nb=0), dict(mb=0), dict(w=None), dict(w=base + 64),
               dict(bytes=255), dict(start=None), dict(slots=None), dict(free=None), dict(cached=None), dict(new=None),
               dict(tables=None), dict(seq=None)):
        assert call(**kw) == zp.ZP_ERR_INVALID_ARG, kw
    for kw in (dict(params=zp.make_params(_params(b=8))), dict(B=65536), dict(nb=2 ** 31 // 16), dict(mb=(1 << 26) + 1)):
        assert call(**kw) == zp.ZP_ERR_UNSUPPORTED, kw


def test_append_refuses(zp):
    ws = torch.zeros(4096, dtype=torch.uint8)
    base = (ws.data_ptr() + 255) // 256 * 256
    good = zp.zp_rows(base, 128, 64)

    def call(pool=zp.zp_kv_pool(base, 4), layer=0, k=good, v=good, slots=base, T=2, params=zp.make_params(_params()), w=base, bytes=256):
        return zp.lib.zp_kv_append(pool, layer, k, v, slots, T, params, w, bytes, None)

    for kw in (dict(pool=None), dict(pool=zp.zp_kv_pool(None, 4)), dict(pool=zp.zp_kv_pool(base, 0)), dict(pool=zp.zp_kv_pool(base + 8, 4)),
               dict(layer=-1), dict(layer=1), dict(k=None), dict(v=None), dict(k=zp.zp_rows(None, 0, 0)), dict(v=zp.zp_rows(base + 1, 128, 64)),
               dict(slots=None), dict(T=-1), dict(params=None), dict(w=None), dict(w=base + 64), dict(bytes=128)):
        assert call(**kw) == zp.ZP_ERR_INVALID_ARG, kw
    for kw in (dict(params=zp.make_params(_params(d=96))), dict(params=zp.make_params(_params(b=8))), dict(pool=zp.zp_kv_pool(base, 2 ** 31 // 16))):
        assert call(**kw) == zp.ZP_ERR_UNSUPPORTED, kw
    assert call(T=0, k=None, v=None, slots=None) == zp.ZP_OK


def test_binding_refuses(zp):
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)
    ws, bf, pool = torch.zeros(256, dtype=torch.uint8), torch.zeros((4, 2, 64), dtype=torch.bfloat16), torch.zeros((1, 4, 2, 2, 16, 64), dtype=torch.bfloat16)
    good = dict(cached=i32(3), new_tokens=i32(3), free_ids=i32(5), block_tables=i32(3, 2), token_start=i32(4), seq_lens=i32(3), slots=i32(9),
                params=_params(), workspace=ws, num_blocks=4, positions=i32(9), first_pos=i32(3), free_at=i32(1))
    for kw in (dict(new_tokens=i32(2)), dict(block_tables=i32(2, 2)), dict(block_tables=i32(6)), dict(token_start=i32(3)), dict(seq_lens=i32(2)),
               dict(positions=i32(8)), dict(first_pos=i32(2)), dict(free_at=i32(0)), dict(cached=torch.zeros(3, dtype=torch.int64)),
               dict(slots=i32(18)[::2]), dict(free_ids=i32(5, 2))):
        with pytest.raises(ValueError, match="expected"):
            zp.zp_step_slots(**{**good, **kw})
    with pytest.raises(ValueError, match="current CUDA device"):
        zp.zp_step_slots(**good)
    with pytest.raises(TypeError):
        zp.zp_step_slots(**{**good, "num_blocks": "4"})
    for k, v, slots in ((bf[:3], bf, i32(4)), (bf, bf[:, :1], i32(4)), (bf, bf, i32(3)), (bf.float(), bf, i32(4)), (bf[..., ::2], bf, i32(4))):
        with pytest.raises(ValueError, match="expected"):
            zp.zp_kv_append(pool, 0, k, v, slots, _params(), ws)
    with pytest.raises(ValueError, match="current CUDA device"):
        zp.zp_kv_append(pool, 0, bf, bf, i32(4), _params(), ws)


def test_oracle_by_hand():
    """Blocks of 16: 15 cached and 2 new tokens fill the part-full block and begin one; nothing, then a fresh request."""
    t = np.array([[7, -1, -1], [3, -1, -1], [-1, -1, -1]], dtype=np.int32)
    got = S.step_slots([15, 4, 0], [2, 0, 17], [5, 2, 9], t, 16, 21, 10, first=[100, 0, 0])
    assert got[0].tolist() == [[7, 5, -1], [3, -1, -1], [2, 9, -1]] and got[1] == [0, 2, 2, 19] and got[2] == [17, 4, 17]
    assert got[3] == [100, 101] + list(range(17)) + [0, 0]
    assert got[4] == [7 * 16 + 15, 5 * 16] + list(range(32, 48)) + [9 * 16, -1, -1] and got[5:] == (3, None)


# ------------------------------------------------------------------ GPU -----------------------

def _dev(x):
    return torch.as_tensor(np.ascontiguousarray(x), dtype=torch.int32).cuda()


def _case(rng, B, b, max_len, max_new, zero=0.2):
    cached = rng.integers(0, max_len + 1, B)
    new = np.where(rng.random(B) < zero, 0, rng.integers(0, max_new + 1, B))
    mb = int(-(-(cached + new).max() // b)) + 1
    held = -(-cached // b)
    NB = int((-(-(cached + new) // b)).sum()) + 4
    ids = rng.permutation(NB)
    tables = np.full((B, mb), -7, dtype=np.int32)
    at = 0
    for r in range(B):
        tables[r, :held[r]] = ids[at:at + held[r]]
        at += held[r]
    return cached, new, tables, ids[at:].astype(np.int32), NB


def _run(zp, cached, new, free, tables, b, T, NB, first=None, free_at=None, in_place=False, ws=None, pos=True):
    B = len(cached)
    d = dict(cached=_dev(cached), new_tokens=_dev(new), free_ids=_dev(free), block_tables=_dev(tables),
             token_start=torch.full((B + 1,), 77, dtype=torch.int32, device="cuda"), slots=torch.full((T,), 77, dtype=torch.int32, device="cuda"),
             positions=torch.full((T,), 77, dtype=torch.int32, device="cuda") if pos else None,
             first_pos=None if first is None else _dev(first), free_at=None if free_at is None else _dev([free_at]))
    d["seq_lens"] = d["cached"] if in_place else torch.full((B,), 77, dtype=torch.int32, device="cuda")
    ws = zp.new_workspace(256) if ws is None else ws
    zp.zp_step_slots(params=_params(b), workspace=ws, num_blocks=NB, **d)
    return d, zp.zp_read_error(ws)


def _same(zp, d, err, want):
    tables, start, seq, positions, slots, at, error = want
    for name, x in (("block_tables", tables), ("token_start", start), ("seq_lens", seq), ("positions", positions), ("slots", slots)):
        if d[name] is not None:
            assert np.array_equal(d[name].cpu().numpy(), np.asarray(x, dtype=np.int32).reshape(d[name].shape)), name
    if d["free_at"] is not None:
        assert d["free_at"].item() == at
    assert err == {None: zp.ZP_OK, "table": zp.ZP_ERR_BAD_TABLE, "blocks": zp.ZP_ERR_NO_BLOCKS}[error]


@pytest.mark.gpu
@pytest.mark.parametrize("B,b,max_len,max_new,pad", [(1, 16, 0, 1, 0), (1, 32, 31, 0, 3), (1, 16, 100, 5000, 0), (3, 16, 40, 40, 5), (31, 32, 300, 9, 0),
                                                     (256, 16, 2047, 1, 0), (33, 16, 500, 700, 123), (1024, 16, 100, 3, 1), (1025, 32, 70, 20, 4),
                                                     (5000, 16, 50, 6, 900), (2, 32, 5, 40000, 17), (64, 16, 4000, 2000, 2)])
def test_slots_match_oracle(zp, B, b, max_len, max_new, pad):
    rng = np.random.default_rng(B * 7 + max_new)
    cached, new, tables, free, NB = _case(rng, B, b, max_len, max_new)
    if B == 1:
        new[:] = max_new
        cached, tables, free, NB = cached, tables, free, NB
        held = int(-(-cached[0] // b))
        used = int(-(-(cached[0] + max_new) // b))
        NB = used + 4
        ids = rng.permutation(NB)
        tables = np.full((1, used + 1), -7, dtype=np.int32)
        tables[0, :held] = ids[:held]
        free = ids[held:].astype(np.int32)
    T = int(new.sum()) + pad
    first = rng.integers(0, 10 ** 6, B)
    for in_place in (False, True):
        for at, f in ((None, None), (min(2, len(free)), first)):
            skip = np.concatenate([np.full(at or 0, -1, dtype=np.int32), free])
            want = S.step_slots(cached, new, skip, tables, b, T, NB, first=f, free_at=at or 0)
            assert want[6] is None
            d, err = _run(zp, cached, new, skip, tables, b, T, NB, first=f, free_at=at, in_place=in_place)
            _same(zp, d, err, want)


@pytest.mark.gpu
def test_no_requests_and_no_rows(zp):
    t = np.zeros((0, 3), dtype=np.int32)
    d, err = _run(zp, [], [], [4], t, 16, 5, 8, free_at=0)
    assert d["token_start"].tolist() == [0] and d["slots"].tolist() == [-1] * 5 and d["positions"].tolist() == [0] * 5 and err == zp.ZP_OK
    d, err = _run(zp, [3, 0], [0, 0], [], np.full((2, 1), 1), 16, 0, 8)
    assert d["token_start"].tolist() == [0, 0, 0] and d["seq_lens"].tolist() == [3, 0] and err == zp.ZP_OK
    d, err = _run(zp, [3], [2], [], np.full((1, 1), 1), 16, 2, 8, pos=False)
    assert d["slots"].tolist() == [19, 20] and err == zp.ZP_OK


@pytest.mark.gpu
@pytest.mark.parametrize("B", [40, 1100])
def test_a_step_that_does_not_fit_is_empty(zp, B):
    rng = np.random.default_rng(B)
    cached, new, tables, free, NB = _case(rng, B, 16, 60, 30)
    T = int(new.sum())
    need = int((-(-(cached + new) // 16) - -(-cached // 16)).sum())
    for rows, ids, at in ((T - 1, free, 0), (T, free[:need - 1], 0), (T, free[:need], 1), (T, free, len(free) + 1), (T, free, -1), (0, free, None)):
        want = S.step_slots(cached, new, ids, tables, 16, rows, NB, free_at=at or 0)
        assert want[6] is not None and sum(want[1]) == 0
        d, err = _run(zp, cached, new, ids, tables, 16, rows, NB, free_at=at)
        _same(zp, d, err, want)
    d, err = _run(zp, cached, new, free[:need], tables, 16, T, NB, free_at=0)   # it just fits
    _same(zp, d, err, S.step_slots(cached, new, free[:need], tables, 16, T, NB))


@pytest.mark.gpu
def test_bad_requests_take_part_without_tokens(zp):
    cached = np.array([5, -1, 20, 2 ** 31 - 1, 40, 48, 16, 3, 49])
    new = np.array([2, 3, -5, 1, 2 ** 31 - 1, 0, 2, 2 ** 30, 0])
    tables = np.arange(27, dtype=np.int32).reshape(9, 3)
    want = S.step_slots(cached, new, [30, 31], tables, 16, 6, 40)
    assert want[1] == [0, 2, 2, 2, 2, 2, 2, 4, 4, 4] and want[2] == [7, 0, 20, 0, 40, 48, 18, 3, 0] and want[6] == "table"
    d, err = _run(zp, cached, new, [30, 31], tables, 16, 6, 40)
    _same(zp, d, err, want)


@pytest.mark.gpu
def test_ids_outside_the_pool_give_no_slots(zp):
    tables = np.array([[40, -1], [-3, -1], [2, -1]], dtype=np.int32)
    free = [3, 41, -2]
    want = S.step_slots([3, 10, 16], [20, 2, 5], free, tables, 16, 30, 40)
    assert want[6] == "table" and want[4][:15] == [-1] * 13 + [48, 49]
    d, err = _run(zp, [3, 10, 16], [20, 2, 5], free, tables, 16, 30, 40)
    _same(zp, d, err, want)


@pytest.mark.gpu
def test_steps_follow_one_another_in_a_graph(zp):
    """A captured step whose lengths, tables and free ids live on the device, replayed: as the oracle's loop."""
    rng = np.random.default_rng(5)
    B, b, steps, T = 37, 16, 25, 160
    cached, mb = rng.integers(0, 40, B), 12
    held = -(-cached // b)
    NB = B * mb
    ids = rng.permutation(NB).astype(np.int32)
    tables = np.full((B, mb), -1, dtype=np.int32)
    for r in range(B):
        tables[r, :held[r]] = ids[held[:r].sum():held[:r + 1].sum()]
    free = ids[held.sum():]
    dev = dict(cached=_dev(cached), new_tokens=_dev(np.zeros(B)), free_ids=_dev(free), block_tables=_dev(tables), token_start=_dev(np.zeros(B + 1)),
               slots=_dev(np.zeros(T)), positions=_dev(np.zeros(T)), first_pos=None, free_at=_dev([0]))
    dev["seq_lens"] = dev["cached"]
    ws, p = zp.new_workspace(256), zp.make_params(_params(b))
    news = [rng.integers(0, 5, B) for _ in range(steps)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        zp.zp_step_slots(params=p, workspace=ws, num_blocks=NB, **dev)
    assert dev["cached"].cpu().numpy().tolist() == cached.tolist()   # captured, not run
    at = 0
    for new in news:
        dev["new_tokens"].copy_(_dev(new))
        graph.replay()
        want = S.step_slots(cached, new, free, tables, b, T, NB, free_at=at)
        assert want[6] is None
        _same(zp, dev, zp.ZP_OK, want)
        tables, cached, at = want[0], np.array(want[2]), want[5]
    assert zp.zp_read_error(ws) == zp.ZP_OK


def _append_case(g, T, Hkv, d, b, NB, layers, pad):
    slots = torch.randperm(NB * b, generator=g)[:T].to(torch.int32)
    slots[torch.randperm(T, generator=g)[:pad]] = -1
    pool = torch.randn((layers, NB, 2, Hkv, b, d), generator=g).to(torch.bfloat16)
    return slots, pool


def _append_want(pool, layer, k, v, slots, b):
    want = pool.clone()
    for t, s in enumerate(slots.tolist()):
        if 0 <= s < pool.shape[1] * b:
            want[layer, s // b, 0, :, s % b] = k[t]
            want[layer, s // b, 1, :, s % b] = v[t]
    return want


@pytest.mark.gpu
@pytest.mark.parametrize("T,Hkv,d,b", [(1, 1, 64, 16), (1, 8, 128, 16), (7, 3, 64, 32), (100, 4, 128, 32), (257, 8, 128, 16), (1000, 2, 64, 16), (5, 5, 128, 16)])
@pytest.mark.parametrize("form", ["contiguous", "fused", "odd", "head-major", "broadcast"])
def test_append_is_bit_exact(zp, T, Hkv, d, b, form):
    g = torch.Generator().manual_seed(T * 10 + Hkv)
    layers, NB = 2, -(-T // b) + 5
    slots, pool = _append_case(g, T, Hkv, d, b, NB, layers, T // 5)
    if form == "contiguous":
        k, v = (torch.randn((T, Hkv, d), generator=g).to(torch.bfloat16) for _ in range(2))
        dk, dv = k.cuda(), v.cuda()
    elif form == "fused":
        x = torch.randn((T, 4 * Hkv, d), generator=g).to(torch.bfloat16)
        dk, dv = x.cuda()[:, Hkv:2 * Hkv], x.cuda()[:, 3 * Hkv:]
    elif form == "odd":
        x = torch.randn(2 * T * Hkv * d + 3, generator=g).to(torch.bfloat16).cuda()
        dk, dv = x[1:1 + T * Hkv * d].view(T, Hkv, d), x[3 + T * Hkv * d:].view(T, Hkv, d)
    elif form == "head-major":
        x = torch.randn((2, Hkv, T, d), generator=g).to(torch.bfloat16).cuda()
        dk, dv = x[0].transpose(0, 1), x[1].transpose(0, 1)
    else:
        x = torch.randn((2, 1, 1, d), generator=g).to(torch.bfloat16).cuda()
        dk, dv = x[0].expand(T, Hkv, d), x[1].expand(T, Hkv, d)
    # every bit pattern passes: NaN and infinities as they are
    if form == "contiguous":
        dk[0, 0, :4] = torch.tensor([0x7FC1, 0x7F80, 0xFF80, 0xFFFF], dtype=torch.int32).to(torch.uint16).view(torch.bfloat16).cuda()
    want = _append_want(pool, 1, dk.cpu(), dv.cpu(), slots, b)
    got, ws = pool.cuda(), zp.new_workspace(256)
    zp.zp_kv_append(got, 1, dk, dv, slots.cuda(), _params(b, Hkv, d, layers), ws)
    assert torch.equal(got.cpu().view(torch.int16), want.view(torch.int16)) and zp.zp_read_error(ws) == zp.ZP_OK


@pytest.mark.gpu
def test_append_skips_slots_outside_the_pool(zp):
    g = torch.Generator().manual_seed(1)
    slots, pool = _append_case(g, 20, 2, 64, 16, 4, 1, 0)
    slots[3], slots[7], slots[11], slots[12] = 64, 2 ** 31 - 1, -2 ** 31, -1
    k, v = (torch.randn((20, 2, 64), generator=g).to(torch.bfloat16) for _ in range(2))
    got, ws = pool.cuda(), zp.new_workspace(256)
    zp.zp_kv_append(got, 0, k.cuda(), v.cuda(), slots.cuda(), _params(16, 2, 64), ws)
    assert torch.equal(got.cpu(), _append_want(pool, 0, k, v, slots, 16)) and zp.zp_read_error(ws) == zp.ZP_ERR_BAD_TABLE
    zp.zp_kv_append(got, 0, k[:0].cuda(), v[:0].cuda(), slots[:0].cuda(), _params(16, 2, 64), ws)   # no rows
    assert zp.zp_read_error(ws) == zp.ZP_OK


@pytest.mark.gpu
def test_append_past_32_bit_offsets(zp):
    """A pool of 4.5 G values: the last block's rows land there and nowhere else."""
    Hkv, d, b, NB = 8, 128, 32, 70000
    pool = torch.zeros((1, NB, 2, Hkv, b, d), dtype=torch.bfloat16, device="cuda")
    k, v = (torch.randn((3, Hkv, d), device="cuda").to(torch.bfloat16) for _ in range(2))
    slots = torch.tensor([NB * b - 1, 5, (NB - 2) * b], dtype=torch.int32).cuda()
    ws = zp.new_workspace(256)
    zp.zp_kv_append(pool, 0, k, v, slots, _params(b, Hkv, d), ws)
    assert zp.zp_read_error(ws) == zp.ZP_OK
    for t, s in enumerate(slots.tolist()):
        assert torch.equal(pool[0, s // b, 0, :, s % b], k[t]) and torch.equal(pool[0, s // b, 1, :, s % b], v[t])
        pool[0, s // b, :, :, s % b] = 0
    assert not bool(torch.any(pool.view(torch.int64)))


@pytest.mark.gpu
def test_slots_place_what_append_writes(zp):
    """Three steps of a ragged batch: the cache read back through the tables is every request's tokens in order."""
    rng = np.random.default_rng(11)
    g = torch.Generator(device="cuda").manual_seed(3)
    B, b, Hkv, d, mb, T = 21, 16, 2, 64, 10, 700
    NB = B * mb
    pool = torch.full((1, NB, 2, Hkv, b, d), 9.0, dtype=torch.bfloat16, device="cuda")
    cached, tables, at = _dev(np.zeros(B)), torch.full((B, mb), -1, dtype=torch.int32, device="cuda"), _dev([0])
    free, start, slots = _dev(rng.permutation(NB)), _dev(np.zeros(B + 1)), _dev(np.zeros(T))
    ws, p = zp.new_workspace(256), zp.make_params(_params(b, Hkv, d))
    kept = [[] for _ in range(B)]
    for hi in (60, 1, 30):
        new = rng.integers(0, hi + 1, B)
        zp.zp_step_slots(cached, _dev(new), free, tables, start, cached, slots, p, ws, num_blocks=NB, free_at=at)
        k, v = (torch.randn((T, Hkv, d), generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
        zp.zp_kv_append(pool, 0, k, v, slots, p, ws)
        lo = 0
        for r in range(B):
            kept[r].append(torch.stack((k[lo:lo + new[r]], v[lo:lo + new[r]])))
            lo += new[r]
    assert zp.zp_read_error(ws) == zp.ZP_OK
    used = 0
    for r in range(B):
        want = torch.cat(kept[r], dim=1)                       # [2, L, H, d]
        L = want.shape[1]
        assert cached[r].item() == L
        ids = tables[r, :-(-L // b)].long()
        used += len(ids)
        got = pool[0, ids].transpose(0, 1).transpose(2, 3).flatten(1, 2)[:, :L]
        assert torch.equal(got, want)
    assert at.item() == used and bool((pool[0, free[used:].long()] == 9.0).all())


@pytest.mark.gpu
def test_on_another_stream(zp):
    """Calls go to the stream that is current, in its order."""
    B, b, NB = 200, 16, 400
    cached, new = np.full(B, 15), np.full(B, 2)
    tables = np.concatenate([np.arange(B)[:, None], np.full((B, 1), -1)], axis=1)
    want = S.step_slots(cached, new, np.arange(200, 400), tables, b, 400, NB)
    side = torch.cuda.Stream()
    big = torch.zeros(1 << 28, device="cuda")
    with torch.cuda.stream(side):
        big.add_(1.0)                         # the lengths come behind it
        d = dict(cached=_dev(cached), new_tokens=torch.zeros(B, dtype=torch.int32, device="cuda"))
        d["new_tokens"] += _dev(new)
        out = dict(block_tables=_dev(tables), token_start=_dev(np.zeros(B + 1)), seq_lens=_dev(np.zeros(B)), slots=_dev(np.zeros(400)),
                   positions=_dev(np.zeros(400)), free_at=None)
        ws = zp.new_workspace(256)
        zp.zp_step_slots(d["cached"], d["new_tokens"], _dev(np.arange(200, 400)), out["block_tables"], out["token_start"], out["seq_lens"],
                         out["slots"], _params(b), ws, num_blocks=NB, positions=out["positions"])
    side.synchronize()
    _same(zp, out, zp.zp_read_error(ws, stream=side), want)
