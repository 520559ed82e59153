"""The operators around the cache as a serving loop runs them together: rotary positions, quantising
the new token, decode attention over the 8-bit cache, and, when a request reaches its cap, reading its
blocks back, the compression pass and packing what it kept; and chunked prefill over the bf16 pool,
whose cache then moves to the 8-bit one."""
import math

import numpy as np
import pytest
import torch

from oracle import parity
from oracle import serving_oracle as S
from paged_kv_cache_obs_gb300 import synth

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def zp():
    import os
    from paged_kv_cache_obs_gb300 import build
    if not os.path.exists(build.LIB):
        build.build()
    from paged_kv_cache_obs_gb300 import zipage
    return zipage


LAYERS, HQ, HKV, D, B, N_MAX, W = 2, 8, 2, 64, 16, 6, 8
THETA = 1e4


def _params(max_blocks=N_MAX):
    return dict(num_layers=LAYERS, num_q_heads=HQ, num_kv_heads=HKV, head_dim=D, block_size=B, n_max=max_blocks, window=W,
                alpha=0.5, beta=0.5, decay=0.9, scale=1.0 / math.sqrt(D), protect_window=1, causal=1)


def _i32(x):
    return torch.as_tensor(np.ascontiguousarray(x), dtype=torch.int32).cuda()


def _check_rows(got, q, k, v, scale, visible, rel):
    """Rows got [G, d] of one kv head against fp64; `rel`: rounding of the weights."""
    for g in range(q.shape[0]):
        want, mass = S.attention_row(q[g], k, v, scale, visible)
        err = np.abs(got[g] - want)
        assert (err <= 2.0 ** -8 * np.abs(want) + (rel + 2.0 ** -14) * mass + 1e-30).all(), float(err.max())


def test_decode_steps_on_an_8_bit_cache(zp):
    # four requests, one of them idle in every other step, 40 steps; a window on one layer
    rng = np.random.default_rng(0)
    g = torch.Generator(device="cuda").manual_seed(0)
    R, steps, max_blocks = 4, 40, 5
    NB = R * max_blocks + 2
    tables = rng.permutation(NB)[:R * max_blocks].reshape(R, max_blocks).astype(np.int32)
    codes = np.zeros((LAYERS, NB, 2, HKV, B, D), dtype=np.uint8)
    scales = np.zeros((LAYERS, NB, 2, HKV))
    d_codes, d_scales, d_tables = torch.from_numpy(codes).cuda(), torch.zeros((LAYERS, NB, 2, HKV), device="cuda"), _i32(tables)
    p = _params(max_blocks)
    rope = zp.zp_rope_init(D, D, THETA)
    freqs, size = S.rope_frequencies(D, THETA)
    ws = zp.new_workspace(zp.zp_kv8_decode_workspace_size(p, R, max_blocks))
    lens = [0, 7, 16, 33]
    # prompts enter the cache as one ragged append per layer
    T = sum(lens)
    pos = np.concatenate([np.arange(n) for n in lens])
    start = [0] + np.cumsum(lens).tolist()
    for layer in range(LAYERS):
        qkv = torch.randn((T, HQ + 2 * HKV, D), generator=g, device="cuda").to(torch.bfloat16)
        k = qkv[:, HQ:HQ + HKV]
        zp.zp_rope_apply(rope, None, k, _i32(pos))           # in place, inside the projection
        zp.zp_kv8_append(d_codes, d_scales, layer, k, qkv[:, HQ + HKV:], _i32(start), _i32([0] * R), d_tables, p, ws)
        S.append(codes, scales, layer, k.double().cpu().numpy(), qkv[:, HQ + HKV:].double().cpu().numpy(), start, [0] * R, tables, B)
    for step in range(steps):
        new = [1, 1, 1, step % 2]
        start = [0] + np.cumsum(new).tolist()
        on = [r for r in range(R) if new[r]]
        positions = _i32([lens[r] for r in on])
        seq = [lens[r] + 1 if new[r] else 0 for r in range(R)]
        for layer in range(LAYERS):
            window, sinks = (0, 0) if layer == 0 else (20, 4)
            qkv = torch.randn((len(on), HQ + 2 * HKV, D), generator=g, device="cuda").to(torch.bfloat16)
            x = qkv.double().cpu().numpy()
            zp.zp_rope_apply(rope, qkv[:, :HQ], qkv[:, HQ:HQ + HKV], positions)
            y = qkv.double().cpu().numpy()
            want = S.rope(x[:, :HQ + HKV], np.array([lens[r] for r in on]), freqs, size, False)
            assert (np.abs(y[:, :HQ + HKV] - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -19 * np.abs(x).max()).all()
            zp.zp_kv8_append(d_codes, d_scales, layer, qkv[:, HQ:HQ + HKV], qkv[:, HQ + HKV:], _i32(start), _i32(lens), d_tables, p, ws)
            S.append(codes, scales, layer, y[:, HQ:HQ + HKV], y[:, HQ + HKV:], start, lens, tables, B)
            # the batch keeps its size; an idle request is a padded row of length 0
            q = torch.zeros((R, HQ, D), dtype=torch.bfloat16, device="cuda")
            q[on] = qkv[:, :HQ]
            out = torch.full_like(q, 7.0)
            zp.zp_kv8_decode_attn(d_codes, d_scales, layer, q, d_tables, _i32(seq), out, p, ws, window=window, sinks=sinks)
            if step % 8 == 7 or step == 0:
                got, qd = out.double().cpu().numpy(), q.double().cpu().numpy()
                for r in range(R):
                    if not new[r]:
                        assert (got[r] == 0).all()
                        continue
                    L = seq[r]
                    nb = -(-L // B)
                    kv = S.e4m3_decode(codes[layer, tables[r, :nb]]) * scales[layer, tables[r, :nb]][..., None, None]
                    vis = S.window_visible(L - 1, L, window, sinks)
                    for h in range(HKV):
                        kk, vv = (kv[:, i, h].reshape(-1, D)[:L] for i in (0, 1))
                        _check_rows(got[r, 4 * h:4 * h + 4], qd[r, 4 * h:4 * h + 4], kk, vv, p["scale"], vis, 2.0 ** -11)
        lens = [n + a for n, a in zip(lens, new)]
    assert np.array_equal(d_codes.cpu().numpy() & 0x7F, codes & 0x7F) and np.array_equal(d_scales.double().cpu().numpy(), scales)
    assert zp.zp_read_error(ws) == 0


def test_compression_of_a_request_held_in_8_bits(zp):
    # at its cap a request is read back into a bf16 staging pool, compressed there, and what it kept
    # is packed again; the next token then decodes over the compacted 8-bit cache
    rng = np.random.default_rng(1)
    g = torch.Generator(device="cuda").manual_seed(1)
    L, k_keep = N_MAX * B, (N_MAX - 1) * B
    NB = 20
    table = rng.permutation(NB)[:N_MAX].astype(np.int32)
    p = _params()
    ws = zp.new_workspace(max(256, zp.zp_kv8_decode_workspace_size(p, 1, N_MAX)))
    d_codes = torch.zeros((LAYERS, NB, 2, HKV, B, D), dtype=torch.float8_e4m3fn, device="cuda")
    d_scales = torch.zeros((LAYERS, NB, 2, HKV), device="cuda")
    for layer in range(LAYERS):
        kv = torch.randn((L, 2 * HKV, D), generator=g, device="cuda").to(torch.bfloat16)
        zp.zp_kv8_append(d_codes, d_scales, layer, kv[:, :HKV], kv[:, HKV:], _i32([0, L]), _i32([0]), _i32(table[None]), p, ws)
    ids, stage = _i32(table), _i32(np.arange(N_MAX))
    pool = torch.zeros((LAYERS, N_MAX, 2, HKV, B, D), dtype=torch.bfloat16, device="cuda")
    zp.zp_kv8_unpack_blocks(d_codes, d_scales, ids, pool, stage, p, ws)
    exact = d_codes[:, table.tolist()].double() * d_scales[:, table.tolist()].double()[..., None, None]
    assert torch.equal(pool.double(), exact)                 # power-of-two scales: nothing is rounded
    # the compression pass, as on any bf16 pool
    pool_in = synth.bf16_bits(pool)
    obs_q = torch.randn((1, LAYERS, W, HQ, D), generator=g, device="cuda").to(torch.bfloat16)
    gs = torch.rand((1, LAYERS, HKV, L), generator=g, device="cuda")
    gs_in = gs.cpu().numpy()
    tab = np.arange(N_MAX, dtype=np.int32)[None]
    dbg = {n: torch.zeros((1, LAYERS, HKV, L), dtype=t, device="cuda")
           for n, t in (("attn", torch.float32), ("redund", torch.float32), ("score", torch.float32), ("keep", torch.int32))}
    cws = zp.new_workspace(zp.zp_compress_workspace_size(p, 1))
    zp.zp_compress(pool, _i32(tab), _i32([L]), _i32([0]), _i32(tab), obs_q, gs, p, cws, debug=dbg)
    assert zp.zp_read_error(cws) == 0
    parity.check_units([(0, layer, h) for layer in range(LAYERS) for h in range(HKV)], pool_in, synth.bf16_bits(obs_q), gs_in,
                       tab, tab, np.array([L]), np.array([0]), p, {n: v.cpu().numpy() for n, v in dbg.items()}, gs.cpu().numpy(),
                       synth.bf16_bits(pool), full_pool=True)
    zp.zp_kv8_pack_blocks(pool, stage[:N_MAX - 1], d_codes, d_scales, ids[:N_MAX - 1], p, ws)
    # the values came from E4M3 at their old blocks' scales; in their new blocks they are rounded to
    # the new scale's grid, which a value of a larger scale's block keeps
    x = pool[:, :N_MAX - 1].double()
    y = d_codes[:, table[:-1].tolist()].double() * d_scales[:, table[:-1].tolist()].double()[..., None, None]
    tol = torch.maximum(x.abs() * 2.0 ** -4, d_scales[:, table[:-1].tolist()].double()[..., None, None] * 2.0 ** -10)
    assert ((x - y).abs() <= tol).all() and float((x == y).double().mean()) > 0.9
    # decode over it
    q = torch.randn((1, HQ, D), generator=g, device="cuda").to(torch.bfloat16)
    for layer in range(LAYERS):
        out = torch.zeros_like(q)
        zp.zp_kv8_decode_attn(d_codes, d_scales, layer, q, _i32(table[None]), _i32([k_keep]), out, p, ws)
        got, qd, kv = out.double().cpu().numpy(), q.double().cpu().numpy(), y[layer].cpu().numpy()
        for h in range(HKV):
            kk, vv = (kv[:, i, h].reshape(-1, D) for i in (0, 1))
            _check_rows(got[0, 4 * h:4 * h + 4], qd[0, 4 * h:4 * h + 4], kk, vv, p["scale"], np.ones(k_keep, dtype=bool), 2.0 ** -11)
    assert zp.zp_read_error(ws) == 0


def test_chunked_prefill_then_8_bit_decode(zp):
    # a prompt in three chunks over the bf16 pool (its rows written by the user's own code), then its
    # blocks, the last one part full, move to the 8-bit pool and one token is decoded
    rng = np.random.default_rng(2)
    g = torch.Generator(device="cuda").manual_seed(2)
    chunks, window, sinks = [70, 1, 52], 48, 3
    L = sum(chunks)
    nb = -(-(L + 1) // B)
    p = _params(nb)
    table = rng.permutation(nb + 3)[:nb].astype(np.int32)
    pool = torch.randn((LAYERS, nb + 3, 2, HKV, B, D), generator=g, device="cuda").to(torch.bfloat16)
    kvs = pool[:, table.tolist()].double().cpu().numpy()      # [layers, blocks, 2, H, B, D]
    done = 0
    for n in chunks:
        q = torch.randn((n, HQ, D), generator=g, device="cuda").to(torch.bfloat16)
        for layer in range(LAYERS):
            out = torch.zeros_like(q)
            ws = zp.new_workspace(zp.zp_paged_window_workspace_size(p, n, 1, n, nb, window, sinks))
            zp.zp_paged_window_attn(pool, layer, q, _i32([0, n]), _i32(table[None]), _i32([done + n]), out, p, ws, window, sinks, n)
            assert zp.zp_read_error(ws) == 0
            got, qd = out.double().cpu().numpy(), q.double().cpu().numpy()
            for h in range(HKV):
                kk, vv = (kvs[layer, :, i, h].reshape(-1, D)[:done + n] for i in (0, 1))
                for i in range(0, n, 7):
                    _check_rows(got[i, 4 * h:4 * h + 4], qd[i, 4 * h:4 * h + 4], kk, vv, p["scale"],
                                S.window_visible(done + i, done + n, window, sinks), 2.0 ** -8)
        done += n
    used = -(-L // B)
    fill = [B] * (used - 1) + [L - (used - 1) * B]
    codes = torch.zeros(pool.shape, dtype=torch.uint8, device="cuda")
    scales = torch.zeros(pool.shape[:4], device="cuda")
    ws = zp.new_workspace(zp.zp_kv8_decode_workspace_size(p, 1, nb))
    ids = _i32(table[:used])
    zp.zp_kv8_pack_blocks(pool, ids, codes, scales, ids, p, ws, fill=_i32(fill))
    kv = torch.randn((1, 2 * HKV, D), generator=g, device="cuda").to(torch.bfloat16)
    q = torch.randn((1, HQ, D), generator=g, device="cuda").to(torch.bfloat16)
    for layer in range(LAYERS):
        zp.zp_kv8_append(codes, scales, layer, kv[:, :HKV], kv[:, HKV:], _i32([0, 1]), _i32([L]), _i32(table[None]), p, ws)
        out = torch.zeros_like(q)
        zp.zp_kv8_decode_attn(codes, scales, layer, q, _i32(table[None]), _i32([L + 1]), out, p, ws, window=window, sinks=sinks)
        c = codes[layer, table.tolist()].cpu().numpy()
        values = S.e4m3_decode(c) * scales[layer, table.tolist()].double().cpu().numpy()[..., None, None]
        # what the cache holds is the prompt's rows and the new token's, to half a step of E4M3
        flat = values.transpose(1, 2, 0, 3, 4).reshape(2, HKV, -1, D)[:, :, :L + 1]
        want = np.concatenate([kvs[layer].transpose(1, 2, 0, 3, 4).reshape(2, HKV, -1, D)[:, :, :L],
                               kv.double().cpu().numpy().reshape(2, HKV, 1, D)], axis=2)
        # (twice rounded where the last block's scale grew)
        s = scales[layer, table.tolist()].double().cpu().numpy().max()
        assert (np.abs(flat - want) <= np.maximum(np.abs(want) * (2.0 ** -4 + 2.0 ** -4), s * 2.0 ** -9)).all()
        got, qd = out.double().cpu().numpy(), q.double().cpu().numpy()
        for h in range(HKV):
            _check_rows(got[0, 4 * h:4 * h + 4], qd[0, 4 * h:4 * h + 4], flat[0, h], flat[1, h], p["scale"],
                        S.window_visible(L, L + 1, window, sinks), 2.0 ** -11)
    assert zp.zp_read_error(ws) == 0


def test_pools_past_32_bit_offsets(zp):
    # the same requests in the first blocks of small pools and in the last blocks of pools of 4.6 GB (8-bit) and
    # 9.2 GB (bf16), whose offsets pass 2^32; every result is the same bits
    g = torch.Generator(device="cuda").manual_seed(3)
    Hq, Hkv, d, b, lens, small, big = 32, 8, 128, 16, [300, 17, 40], 40, 70000
    used = [-(-n // b) for n in lens]
    max_blocks, R, T = max(used), len(lens), sum(lens)
    table = np.zeros((R, max_blocks), dtype=np.int32)
    ids = np.random.default_rng(3).permutation(small)[:sum(used)]
    at = 0
    for r, n in enumerate(used):
        table[r, :n] = ids[at:at + n]
        at += n
    p = zp.make_params(dict(num_layers=2, num_q_heads=Hq, num_kv_heads=Hkv, head_dim=d, block_size=b, n_max=4, window=1, alpha=0.5,
                            beta=0.5, decay=0.9, scale=d ** -0.5, protect_window=1, causal=1))
    kv = torch.randn((T, 2 * Hkv, d), generator=g, device="cuda").to(torch.bfloat16)
    q = torch.randn((T, Hq, d), generator=g, device="cuda").to(torch.bfloat16)
    start = _i32(np.concatenate([[0], np.cumsum(lens)]))
    results = []
    for NB, shift in ((small, 0), (big, big - small)):
        ws = zp.new_workspace(max(zp.zp_kv8_decode_workspace_size(p, R, max_blocks),
                                  zp.zp_paged_window_workspace_size(p, T, R, max(lens), max_blocks, 100, 4),
                                  zp.zp_paged_window_workspace_size(p, R, R, 1, max_blocks, 100, 4)))
        tables, blocks = _i32(table + shift), _i32(ids + shift)
        codes = torch.zeros((2, NB, 2, Hkv, b, d), dtype=torch.uint8, device="cuda")
        scales = torch.zeros((2, NB, 2, Hkv), device="cuda")
        zp.zp_kv8_append(codes, scales, 1, kv[:, :Hkv], kv[:, Hkv:], start, _i32([0] * R), tables, p, ws)
        out8 = torch.zeros((R, Hq, d), dtype=torch.bfloat16, device="cuda")
        zp.zp_kv8_decode_attn(codes, scales, 1, q[:R], tables, _i32(lens), out8, p, ws)
        pool = torch.zeros((2, NB, 2, Hkv, b, d), dtype=torch.bfloat16, device="cuda")
        zp.zp_kv8_unpack_blocks(codes, scales, blocks, pool, blocks, p, ws)
        many, few = torch.zeros_like(q), torch.zeros((R, Hq, d), dtype=torch.bfloat16, device="cuda")
        zp.zp_paged_window_attn(pool, 1, q, start, tables, _i32(lens), many, p, ws, 100, 4, max(lens))
        zp.zp_paged_window_attn(pool, 1, q[:R], _i32([0, 1, 2, 3]), tables, _i32(lens), few, p, ws, 100, 4, 1)
        codes.zero_()
        scales.zero_()
        zp.zp_kv8_pack_blocks(pool, blocks, codes, scales, blocks, p, ws)
        assert zp.zp_read_error(ws) == 0
        keep = (ids + shift).tolist()
        results.append((out8, many, few, codes[:, keep].clone(), scales[:, keep].clone(), pool[:, keep].clone()))
        del codes, pool
        torch.cuda.empty_cache()
    assert all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(*results))
    assert float(results[0][1].abs().max()) > 0 and float(results[0][3].float().abs().max()) > 0


def _chain(zp, steps, sync, graph=False):
    """Operators whose inputs are the outputs of the ones before, torch's own kernels between some of them."""
    g = torch.Generator(device="cuda").manual_seed(4)
    p, R = zp.make_params(_params()), 3
    q = torch.randn((R, HQ, D), generator=g, device="cuda").to(torch.bfloat16)
    kv = torch.randn((R, 2 * HKV, D), generator=g, device="cuda").to(torch.bfloat16)
    codes = torch.zeros((LAYERS, 24, 2, HKV, B, D), dtype=torch.uint8, device="cuda")
    scales = torch.zeros((LAYERS, 24, 2, HKV), device="cuda")
    pool = torch.zeros((LAYERS, 24, 2, HKV, B, D), dtype=torch.bfloat16, device="cuda")
    tables, start, lens = _i32(np.arange(18).reshape(R, N_MAX)), _i32([0, 1, 2, 3]), _i32([0, 5, 30])
    many, more = (torch.zeros((3 * R, HQ, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    ids, rope = _i32(np.arange(18)), zp.zp_rope_init(D, D, THETA)
    ws = zp.new_workspace(max(zp.zp_kv8_decode_workspace_size(p, R, N_MAX), zp.zp_paged_window_workspace_size(p, 3 * R, R, 5, N_MAX, 40, 2)))
    out8, out16 = torch.zeros_like(q), torch.zeros_like(q)
    done = torch.cuda.synchronize if sync else (lambda: None)

    def step():
        zp.zp_rope_apply(rope, q, kv[:, :HKV], lens)
        done()
        zp.zp_kv8_append(codes, scales, 1, kv[:, :HKV], kv[:, HKV:], start, lens, tables, p, ws)
        done()
        lens.add_(1)
        done()
        zp.zp_kv8_decode_attn(codes, scales, 1, q, tables, lens, out8, p, ws)
        done()
        zp.zp_rope_apply(rope, out8, kv[:, HKV:], lens)
        done()
        zp.zp_kv8_unpack_blocks(codes, scales, ids, pool, ids, p, ws)
        done()
        zp.zp_paged_window_attn(pool, 1, out8, start, tables, lens, out16, p, ws, 40, 2, 1)
        done()
        many[:R] = out16
        zp.zp_paged_window_attn(pool, 1, many, start, tables, lens, more, p, ws, 40, 2, 5)
        done()
        zp.zp_kv8_pack_blocks(pool, ids, codes, scales, ids, p, ws)
        done()
        kv.copy_(more[:R, :2 * HKV])
        q.copy_(out16)
        done()
    if graph:
        step()
        c = torch.cuda.CUDAGraph()
        with torch.cuda.graph(c):
            for _ in range(5):
                step()
        for _ in range(steps // 5):
            c.replay()
    else:
        for _ in range(steps):
            step()
    assert zp.zp_read_error(ws) == 0
    return [x.clone() for x in (q, kv, codes, scales, pool, more, out8, out16, lens)]


def test_calls_follow_one_another_in_order(zp):
    # kernels come in before the ones ahead of them are complete; what they compute is what calls with a
    # synchronisation after each compute, on a stream and in a captured graph
    want = _chain(zp, 51, True)
    for _ in range(3):
        assert all(torch.equal(x, y) for x, y in zip(want, _chain(zp, 51, False)))
    assert all(torch.equal(x, y) for x, y in zip(want, _chain(zp, 51, False, graph=True)))
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = _chain(zp, 51, False)
    side.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(want, got))


@pytest.mark.parametrize("captured", [False, True])
def test_calls_wait_for_other_streams_and_for_copies(zp, captured):
    # a call behind an event of another stream, whose work takes long, and behind a copy, right after a call of
    # the same operator
    g = torch.Generator(device="cuda").manual_seed(5)
    T = 64
    fresh, other = (torch.randn((T, HQ, D), generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    x, copied = torch.zeros_like(fresh), torch.zeros_like(fresh)
    out, out2, scrap = torch.zeros_like(fresh), torch.zeros_like(fresh), torch.zeros_like(fresh)
    pos = _i32(np.arange(T))
    rope = zp.zp_rope_init(D, D, THETA)
    want = torch.zeros_like(fresh)
    zp.zp_rope_apply(rope, fresh, None, pos, q_out=want)
    main, side = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()

    def work():
        side.wait_stream(main)
        with torch.cuda.stream(side):
            torch.cuda._sleep(2_000_000)           # about a millisecond
            x.copy_(fresh)
        zp.zp_rope_apply(rope, other, None, pos, q_out=scrap)
        main.wait_stream(side)
        zp.zp_rope_apply(rope, x, None, pos, q_out=out)
        copied.copy_(fresh)
        zp.zp_rope_apply(rope, copied, None, pos, q_out=out2)

    with torch.cuda.stream(main):
        if captured:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=main):
                work()
        for _ in range(5):
            for t in (x, copied, out, out2):
                t.zero_()
            graph.replay() if captured else work()
            main.synchronize()
            assert torch.equal(out, want) and torch.equal(out2, want)
