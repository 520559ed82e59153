"""Decode attention over the 8-bit pool (zp_kv8_decode_attn) and attention with a sliding window and
first tokens that stay visible over the bf16 pool (zp_paged_window_attn), against fp64."""
import ctypes
import math
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


def _rows(zp, t):
    return zp.zp_rows(t.data_ptr(), t.stride(0), t.stride(1))


def _params(Hq, Hkv, d, b, layers=1, scale=None):
    return dict(num_layers=layers, num_q_heads=Hq, num_kv_heads=Hkv, head_dim=d, block_size=b, n_max=4, window=1, alpha=0.5,
                beta=0.5, decay=0.9, scale=scale or 1.0 / math.sqrt(d), protect_window=1, causal=1)


# ------------------------------------------------------------------ refusals (CPU) ------------

def _refusals(zp, call, base, x, p):
    bad, uns = zp.ZP_ERR_INVALID_ARG, zp.ZP_ERR_UNSUPPORTED
    params = lambda **kw: zp.make_params({**p, **kw})
    for kw in (dict(pool=None), dict(layer=-1), dict(layer=1), dict(q=None), dict(out=None), dict(tables=None), dict(seq=None),
               dict(B=-1), dict(mb=0), dict(window=-1), dict(sinks=-1), dict(params=None), dict(ws=None), dict(ws=base + 64),
               dict(nb=255), dict(q=zp.zp_rows(x.data_ptr() + 1, 128, 64)), dict(out=zp.zp_rows(None, 0, 0)),
               dict(params=params(scale=0.0)), dict(params=params(scale=-1.0)), dict(params=params(scale=math.inf)),
               dict(params=params(scale=math.nan)), dict(params=params(scale=3.4e38)), dict(params=params(num_q_heads=3)), dict(params=params(num_kv_heads=0))):
        assert call(**kw) == bad, kw
    for kw in (dict(params=params(head_dim=96)), dict(params=params(block_size=8)), dict(params=params(num_q_heads=34)),
               dict(mb=1 << 28), dict(B=65536, nb=1 << 40)):
        assert call(**kw) == uns, kw


def _host(zp):
    ws = torch.zeros(1 << 16, dtype=torch.uint8)
    base = (ws.data_ptr() + 255) // 256 * 256
    x = torch.zeros((2, 2, 64), dtype=torch.bfloat16)
    return ws, base, x, _params(2, 2, 64, 16)


def test_kv8_decode_refuses(zp):
    ws, base, x, p = _host(zp)
    rows = _rows(zp, x)

    def call(pool=zp.zp_kv8_pool(base, base, 4), layer=0, q=rows, tables=base, seq=base, B=2, mb=2, window=0, sinks=0, out=rows,
             params=zp.make_params(p), ws=base, nb=1 << 40):
        return zp.lib.zp_kv8_decode_attn(pool, layer, q, tables, seq, B, mb, window, sinks, out, params, ws, nb, None)

    _refusals(zp, call, base, x, p)
    bad = zp.ZP_ERR_INVALID_ARG
    for pool in (zp.zp_kv8_pool(None, base, 4), zp.zp_kv8_pool(base, None, 4), zp.zp_kv8_pool(base, base, 0),
                 zp.zp_kv8_pool(base + 8, base, 4), zp.zp_kv8_pool(base, base + 1, 4)):
        assert call(pool=pool) == bad
    assert call(B=0, q=None, out=None, tables=None, seq=None) == zp.ZP_OK
    assert call(mb=4096, B=1, nb=zp.zp_kv8_decode_workspace_size(p, 1, 4096) - 1) == bad


def test_window_refuses(zp):
    ws, base, x, p = _host(zp)
    rows = _rows(zp, x)

    def call(pool=zp.zp_kv_pool(base, 4), layer=0, q=rows, start=base, T=2, max_q=1, tables=base, seq=base, B=2, mb=2, window=4,
             sinks=1, out=rows, params=zp.make_params(p), ws=base, nb=1 << 40):
        return zp.lib.zp_paged_window_attn(pool, layer, q, start, T, max_q, tables, seq, B, mb, window, sinks, out, params, ws, nb, None)

    _refusals(zp, call, base, x, p)
    bad = zp.ZP_ERR_INVALID_ARG
    for kw in (dict(start=None), dict(T=-1), dict(max_q=0), dict(pool=zp.zp_kv_pool(None, 4)), dict(pool=zp.zp_kv_pool(base + 8, 4)),
               dict(pool=zp.zp_kv_pool(base, 0))):
        assert call(**kw) == bad, kw
    assert call(pool=zp.zp_kv_pool(base, 1 << 31)) == zp.ZP_ERR_UNSUPPORTED
    assert call(B=0, q=None, out=None, tables=None, seq=None, start=None) == zp.ZP_OK
    assert call(T=0) == zp.ZP_OK and call(T=0, q=zp.zp_rows(None, 0, 0), out=zp.zp_rows(None, 0, 0)) == zp.ZP_OK


def test_workspace_sizes(zp):
    p = _params(32, 8, 128, 16)
    # a batch that is not split, or whose splits are one cluster, needs the header alone; few long
    # requests need parts, never fewer for longer caches, and a window never more than none
    assert zp.zp_kv8_decode_workspace_size(p, 256, 8192) == 256 and zp.zp_kv8_decode_workspace_size(p, 1, 1) == 256
    sizes = [zp.zp_kv8_decode_workspace_size(p, 1, mb) for mb in range(1, 3000, 7)]
    assert sizes == sorted(sizes) and 256 < sizes[-1] < 16 << 20
    for w in (1, 100, 5000, 10 ** 6):
        assert zp.zp_paged_window_workspace_size(p, 2, 1, 2, 4096, w, 9) <= zp.zp_paged_window_workspace_size(p, 2, 1, 2, 4096, 0, 0)
    assert zp.zp_kv8_decode_workspace_size(p, -1, 4) == 0 and zp.zp_paged_window_workspace_size(p, 4, 1, 0, 4, 1, 1) == 0
    # heads that no kernel takes
    assert zp.zp_kv8_decode_workspace_size(_params(400, 2, 128, 16), 1, 4) == 0
    assert zp.zp_paged_window_workspace_size(_params(400, 2, 128, 16), 4, 1, 4, 4, 1, 1) == 0
    # any bound on the new tokens; a workspace for many rows is enough for fewer
    most = 2 ** 31 - 1
    assert zp.zp_paged_window_workspace_size(p, most, 65535, most, 1 << 26, 0, 0) == 256
    for mq in (17, 64, 2048, most):
        sizes = [zp.zp_paged_window_workspace_size(p, T, 1, mq, 4096, 0, 0) for T in (0, 1, 17, 64, 500, 2048, 60000)]
        assert sizes == sorted(sizes)


# ------------------------------------------------------------------ inputs and checks ---------

def _tables(rng, lens, b, extra=3):
    used = [-(-int(x) // b) for x in lens]
    NB = sum(used) + extra
    perm = rng.permutation(NB)
    tables = np.full((len(lens), max(1, max(used))), -1, dtype=np.int32)   # entries past the sequence are not read
    at = 0
    for r, n in enumerate(used):
        tables[r, :n] = perm[at:at + n]
        at += n
    return tables, NB


def _tolerance(want, mass, rel):
    """bf16 rounding of the output 2^-8; weights off by `rel` (P's rounding) and 2^-14 (logits and
    sums in fp32: |logit| <= 64 here, 128 products, ex2) against the weighted magnitudes."""
    return 2.0 ** -8 * np.abs(want) + (rel + 2.0 ** -14) * mass + 1e-30


def _kv8_case(zp, Hq, Hkv, d, b, lens, window=0, sinks=0, seed=0, scale_exp=(-8, -4), layer=1, q_gain=2.0, hidden_nan=True,
              q_off=0, expect=0, tables_edit=None, seq_edit=None):
    rng = np.random.default_rng(seed)
    G, B = Hq // Hkv, len(lens)
    tables, NB = _tables(rng, lens, b)
    codes = S.e4m3_encode(np.clip(rng.standard_normal((2, NB, 2, Hkv, b, d)) * 64, -448, 448))
    scales = (2.0 ** rng.integers(*scale_exp, (2, NB, 2, Hkv)) * (1 + rng.random((2, NB, 2, Hkv)))).astype(np.float32)
    # every token that a request does not see holds NaN
    if hidden_nan:
        for r, L in enumerate(lens):
            vis = S.window_visible(L - 1, L, window, sinks)
            for t in range(tables.shape[1] * b):
                if t // b < -(-L // b) and not (t < L and vis[t]):
                    codes[layer, tables[r, t // b], :, :, t % b] = 0x7F
    q = torch.from_numpy(rng.standard_normal((B, Hq, d)) * q_gain).to(torch.bfloat16)
    buf = torch.zeros(B * Hq * d + 8, dtype=torch.bfloat16)
    buf[q_off:q_off + q.numel()] = q.flatten()
    dq = buf.cuda()[q_off:q_off + q.numel()].view(B, Hq, d)
    obuf = torch.full((B * Hq * d + 8,), 7.0, dtype=torch.bfloat16, device="cuda")
    out = obuf[q_off:q_off + q.numel()].view(B, Hq, d)
    p = _params(Hq, Hkv, d, b, 2)
    ws = zp.new_workspace(zp.zp_kv8_decode_workspace_size(p, B, tables.shape[1]))
    dev_tables = tables.copy() if tables_edit is None else tables_edit(tables.copy())
    seq = list(lens) if seq_edit is None else seq_edit(list(lens))
    args = (torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda(), layer, dq, torch.from_numpy(dev_tables).cuda(),
            torch.tensor(seq, dtype=torch.int32).cuda(), out, p, ws)
    for _ in range(2):  # twice: the workspace is left as the next call expects it
        zp.zp_kv8_decode_attn(*args, window=window, sinks=sinks)
    assert zp.zp_read_error(ws) == expect
    got, qd = out.double().cpu().numpy(), q.double().numpy()
    rest = obuf.cpu()
    assert bool((rest[:q_off] == 7).all()) and bool((rest[q_off + q.numel():] == 7).all())
    kv = S.e4m3_decode(codes[layer]) * scales[layer].astype(np.float64)[..., None, None]
    for r, L in enumerate(lens):
        if (seq[r] != L) or (dev_tables[r] != tables[r]).any():
            assert (got[r] == 7).all()      # skipped
            continue
        vis = S.window_visible(L - 1, L, window, sinks)
        for h in range(Hkv):
            n = -(-L // b)
            k, v = (kv[tables[r, :n], i, h].reshape(-1, d)[:L] for i in (0, 1))
            for gi in range(G):
                want, mass = S.attention_row(qd[r, h * G + gi], k, v, p["scale"], vis)
                err = np.abs(got[r, h * G + gi] - want)
                assert (err <= _tolerance(want, mass, 2.0 ** -11)).all(), (r, h, gi, float(err.max()))
    return args


SHAPES = [(32, 8, 128, 16), (28, 4, 128, 32), (8, 8, 64, 16), (16, 2, 64, 32), (8, 4, 128, 16), (3, 1, 128, 32), (16, 1, 128, 16),
          (10, 1, 64, 32), (11, 1, 64, 16)]


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,Hkv,d,b", SHAPES)
def test_kv8_decode_lengths(zp, Hq, Hkv, d, b):
    _kv8_case(zp, Hq, Hkv, d, b, [1, 0, b - 1, b, b + 1, 255, 256, 257, 700], seed=Hq)


@pytest.mark.gpu
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (7, 3), (16, 16), (17, 0), (100, 4), (64, 40), (300, 1000), (5000, 2), (33, 64)])
def test_kv8_decode_windows(zp, window, sinks):
    _kv8_case(zp, 8, 2, 128, 16, [1, 2, 16, 17, 40, 300, 513, 0, 1100], window, sinks, seed=window)
    _kv8_case(zp, 7, 1, 64, 32, [5, 64, 65, 777], window, sinks, seed=sinks, layer=0)


@pytest.mark.gpu
def test_kv8_decode_many_splits(zp):
    _kv8_case(zp, 8, 2, 128, 16, [9000, 1, 4097], seed=1)
    _kv8_case(zp, 14, 2, 64, 32, [5000, 130], window=4000, sinks=7, seed=2)


@pytest.mark.gpu
@pytest.mark.parametrize("lo,hi", [(-60, -50), (40, 50), (-30, 20)])
def test_kv8_decode_scales_of_any_size(zp, lo, hi):
    # K and V scales far from 1 and from one another; logits are brought back by the query's size
    _kv8_case(zp, 8, 2, 128, 16, [300, 33], seed=3, scale_exp=(lo, hi), q_gain=2.0 ** -(hi + 6))


@pytest.mark.gpu
def test_kv8_decode_unaligned_rows_and_large_batch(zp):
    _kv8_case(zp, 8, 2, 64, 16, [1, 50, 300], seed=4, q_off=1)
    rng = np.random.default_rng(5)
    _kv8_case(zp, 4, 2, 64, 16, [int(x) for x in rng.integers(0, 200, 300)], seed=5, hidden_nan=False)


@pytest.mark.gpu
@pytest.mark.parametrize("B,top", [(305, 40), (1024, 9), (1025, 9), (512, 1)])
def test_batches_of_several_waves(zp, B, top):
    # long requests are taken first, up to 1024 of them: every request once, whatever their lengths
    rng = np.random.default_rng(B)
    lens = [int(x) for x in rng.integers(0, top, B)]
    lens[B // 2] = 200

    def seq(x):
        x[0], x[B - 1], x[B // 3] = 2 ** 31 - 1, -2 ** 31, 10 ** 6
        return x
    _kv8_case(zp, 2, 2, 64, 16, lens, seed=B, seq_edit=seq, expect=zp.ZP_ERR_BAD_TABLE, hidden_nan=False)
    _window_case(zp, 2, 2, 64, 16, lens, [1 + r % 3 for r in range(B)], 0, 0, seed=B, rel=SPLIT)
    if B < 400:
        _window_case(zp, 8, 2, 128, 16, lens, [1 + r % 3 for r in range(B)], 0, 0, seed=B, rel=SPLIT)


@pytest.mark.gpu
def test_kv8_decode_skips_bad_rows_and_reports(zp):
    def edit(t):
        t[1, 2] = 10 ** 6
        return t

    for lens in ([100, 90, 40], [100, 3000, 40]):   # one split and several
        _kv8_case(zp, 8, 2, 128, 16, lens, seed=6, tables_edit=edit, expect=zp.ZP_ERR_BAD_TABLE)
        for bad in (-1, 10 ** 6):
            def seq(x, bad=bad):
                x[1] = bad
                return x
            _kv8_case(zp, 8, 2, 128, 16, lens, seed=7, seq_edit=seq, expect=zp.ZP_ERR_BAD_TABLE)


@pytest.mark.gpu
def test_kv8_decode_entries_outside_the_window_are_not_read(zp):
    def edit(t):
        t[0, 2:10] = -5      # between the first tokens and the window
        return t
    rng = np.random.default_rng(8)
    lens = [400]
    tables, NB = _tables(rng, lens, 16)
    # the same outputs with and without the hidden entries
    outs = []
    for t in (tables, edit(tables.copy())):
        g = torch.Generator(device="cuda").manual_seed(1)
        codes = (torch.randn((1, NB, 2, 1, 16, 128), generator=g, device="cuda") * 64).clamp(-448, 448).to(torch.float8_e4m3fn)
        scales = torch.full((1, NB, 2, 1), 2.0 ** -6, device="cuda")
        q = torch.randn((1, 4, 128), generator=g, device="cuda").to(torch.bfloat16)
        out = torch.zeros_like(q)
        p = _params(4, 1, 128, 16)
        ws = zp.new_workspace(zp.zp_kv8_decode_workspace_size(p, 1, t.shape[1]))
        zp.zp_kv8_decode_attn(codes, scales, 0, q, torch.from_numpy(t).cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), out, p, ws,
                              window=200, sinks=20)
        assert zp.zp_read_error(ws) == 0
        outs.append(out)
    assert torch.equal(*outs)


@pytest.mark.gpu
def test_kv8_decode_nan_in_a_seen_key_or_value_shows(zp):
    for kv, where in ((0, "all"), (1, "dim")):
        codes = torch.full((1, 4, 2, 1, 16, 64), 0x38, dtype=torch.uint8, device="cuda")   # 1.0
        scales = torch.ones((1, 4, 2, 1), device="cuda")
        codes[0, 1, kv, 0, 5, 3] = 0x7F
        q = torch.ones((1, 2, 64), dtype=torch.bfloat16, device="cuda")
        out = torch.zeros_like(q)
        p = _params(2, 1, 64, 16)
        ws = zp.new_workspace(zp.zp_kv8_decode_workspace_size(p, 1, 4))
        zp.zp_kv8_decode_attn(codes, scales, 0, q, torch.arange(4, dtype=torch.int32, device="cuda")[None],
                              torch.tensor([60], dtype=torch.int32, device="cuda"), out, p, ws)
        nan = torch.isnan(out)
        assert bool(nan.all()) if where == "all" else (bool(nan[..., 3].all()) and int(nan.sum()) == 2)


# ------------------------------------------------------------------ windowed attention --------

def _window_case(zp, Hq, Hkv, d, b, cached, new, window, sinks, seed=0, max_q=None, off=0, gain=2.0, expect=0, poison=None,
                 hidden_nan=False, skip=(), start_edit=None, seq_edit=None, tables_edit=None, rel=2.0 ** -8):
    """poison(kv, tables): puts special values into the bf16 pool (fp64 array of layer 1)."""
    rng = np.random.default_rng(seed)
    G, B = Hq // Hkv, len(new)
    lens = [c + n for c, n in zip(cached, new)]
    tables, NB = _tables(rng, lens, b)
    x = rng.standard_normal((NB, 2, Hkv, b, d))
    if hidden_nan:
        for r in range(B):
            seen = np.zeros(lens[r], dtype=bool)
            for i in range(new[r]):
                seen |= S.window_visible(cached[r] + i, lens[r], window, sinks)
            for t in range(-(-lens[r] // b) * b):
                if not (t < lens[r] and seen[t]):
                    x[tables[r, t // b], :, :, t % b] = rng.choice([np.nan, np.inf, -np.inf])
    if poison:
        poison(x, tables)
    pool = torch.zeros((2, NB, 2, Hkv, b, d), dtype=torch.bfloat16)
    pool[1] = torch.from_numpy(x).to(torch.bfloat16)
    kv = pool[1].double().numpy()
    T = sum(new)
    start = [0] + np.cumsum(new).tolist()
    q = torch.from_numpy(rng.standard_normal((T, Hq, d)) * gain).to(torch.bfloat16)
    n = q.numel()
    buf = torch.zeros(n + 8, dtype=torch.bfloat16)
    buf[off:off + n] = q.flatten()
    dq = buf.cuda()[off:off + n].view(T, Hq, d)
    obuf = torch.full((n + 8,), 7.0, dtype=torch.bfloat16, device="cuda")
    out = obuf[off:off + n].view(T, Hq, d)
    p = _params(Hq, Hkv, d, b, 2)
    mq = max_q or max(1, max(new))
    ws = zp.new_workspace(zp.zp_paged_window_workspace_size(p, T, B, mq, tables.shape[1], window, sinks))
    i32 = lambda v: torch.tensor(v, dtype=torch.int32).cuda()
    args = (pool.cuda(), 1, dq, i32(start if start_edit is None else start_edit(list(start))),
            torch.from_numpy(tables.copy() if tables_edit is None else tables_edit(tables.copy())).cuda(),
            i32(lens if seq_edit is None else seq_edit(list(lens))), out, p, ws, window, sinks, mq)
    for _ in range(2):
        zp.zp_paged_window_attn(*args)
    assert zp.zp_read_error(ws) == expect
    got, qd = out.double().cpu().numpy(), q.double().numpy()
    rest = obuf.cpu()
    assert bool((rest[:off] == 7).all()) and bool((rest[off + n:] == 7).all())
    worst = 0.0
    for r in range(B):
        rows = got[start[r]:start[r + 1]]
        if r in skip:
            assert (rows == 7).all()
            continue
        nb = -(-lens[r] // b)
        for h in range(Hkv):
            k, v = (kv[tables[r, :nb], i, h].reshape(-1, d)[:lens[r]] for i in (0, 1))
            for i in range(new[r]):
                vis = S.window_visible(cached[r] + i, lens[r], window, sinks)
                for gi in range(G):
                    with np.errstate(invalid="ignore"):
                        want, mass = S.attention_row(qd[start[r] + i, h * G + gi], k, v, p["scale"], vis)
                    y = rows[i, h * G + gi]
                    fin = np.isfinite(want)
                    assert np.array_equal(fin, np.isfinite(y)), (r, h, i, gi)
                    tol = _tolerance(want[fin], mass[fin], rel)
                    err = np.abs(y[fin] - want[fin])
                    assert (err <= tol).all(), (r, h, i, gi, float(err.max()))
                    worst = max(worst, float((err / tol).max(initial=0)))
    return args


# P is a bf16 pair (2^-16) in the split form, bf16 (2^-8) in the tiled form
SPLIT, TILED = 2.0 ** -16, 2.0 ** -8


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,Hkv,d,b", SHAPES)
def test_window_single_tokens(zp, Hq, Hkv, d, b):
    _window_case(zp, Hq, Hkv, d, b, [0, 1, b - 1, b, 254, 700, 1999], [1] * 7, 100, 5, seed=Hq, hidden_nan=True, rel=SPLIT)


@pytest.mark.gpu
@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (2, 1), (16, 17), (100, 0), (64, 64), (5000, 3)])
def test_window_few_tokens(zp, window, sinks):
    # several queries per request in the split form, ragged, some requests idle
    _window_case(zp, 8, 2, 128, 16, [0, 5, 0, 300, 31, 63], [3, 1, 0, 2, 4, 4], window, sinks, seed=window, hidden_nan=True, rel=SPLIT)
    _window_case(zp, 4, 1, 64, 32, [200, 0, 30], [4, 2, 3], window, sinks, seed=sinks, hidden_nan=True, rel=SPLIT)


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,Hkv,d,b", [(32, 8, 128, 16), (28, 4, 128, 32), (8, 8, 64, 16), (16, 2, 64, 32), (16, 1, 128, 16), (3, 1, 64, 16)])
def test_window_chunks(zp, Hq, Hkv, d, b):
    _window_case(zp, Hq, Hkv, d, b, [0, 17, 130, 5], [40, 33, 1, 0], 50, 5, seed=Hq, hidden_nan=True, rel=TILED)


@pytest.mark.gpu
@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (1, 1), (16, 17), (100, 0), (128, 128), (129, 300), (70, 33), (5000, 3)])
def test_window_chunks_of_several_tiles(zp, window, sinks):
    _window_case(zp, 4, 2, 128, 16, [0, 333], [150, 129], window, sinks, seed=window, hidden_nan=True, rel=TILED)
    _window_case(zp, 2, 2, 64, 32, [100, 0], [300, 257], window, sinks, seed=sinks, hidden_nan=True, rel=TILED)


@pytest.mark.gpu
def test_window_long_prompt(zp):
    _window_case(zp, 2, 1, 128, 16, [0], [1500], 700, 4, seed=1, rel=TILED)
    _window_case(zp, 7, 1, 64, 32, [2500], [40], 0, 0, seed=2, rel=TILED)


@pytest.mark.gpu
def test_window_unaligned_rows(zp):
    _window_case(zp, 4, 2, 128, 16, [10], [70], 30, 2, seed=3, off=1, rel=TILED)
    _window_case(zp, 4, 2, 64, 16, [10, 3], [2, 1], 30, 2, seed=3, off=3, rel=SPLIT)


@pytest.mark.gpu
@pytest.mark.parametrize("new", [3, 70])
@pytest.mark.parametrize("value", [math.inf, -math.inf, math.nan])
def test_window_values_reach_only_the_rows_that_see_them(zp, new, value):
    # one bad value in V (and one in K) at positions that later rows see and earlier ones do not,
    # and one that leaves the window of the later rows
    def poison(x, tables):
        L = 200 + new
        for t, kv, dim in ((L - 2, 1, 7), (190 + 5, 1, 60)):
            x[tables[0, t // 16], kv, 0, t % 16, dim] = value
    _window_case(zp, 4, 2, 64, 16, [200], [new], 6, 2, seed=4, poison=poison, rel=TILED if new > 4 else SPLIT)


@pytest.mark.gpu
@pytest.mark.parametrize("new", [2, 60])
def test_window_skips_bad_rows_and_reports(zp, new):
    kw = dict(window=40, sinks=2, seed=5, expect=zp.ZP_ERR_BAD_TABLE, skip=(1,), rel=TILED)
    cached, n = [30, 60, 9], [new, new, new]

    def put(i, v):
        def f(x):
            x[i] = v
            return x
        return f

    def table(t):
        t[1, (60 + new - 1) // 16] = -1
        return t
    _window_case(zp, 4, 2, 64, 16, cached, n, seq_edit=put(1, new - 1), **kw)
    _window_case(zp, 4, 2, 64, 16, cached, n, seq_edit=put(1, 10 ** 6), **kw)
    _window_case(zp, 4, 2, 64, 16, cached, n, tables_edit=table, **kw)
    kw["skip"] = (2,)
    _window_case(zp, 4, 2, 64, 16, cached, n, start_edit=put(3, 3 * new + 1), **kw)
    # a request above max_q
    kw["skip"] = (0,)
    _window_case(zp, 4, 2, 64, 16, cached, [new + 1, new, new], max_q=new, **kw)


@pytest.mark.gpu
def test_window_padded_rows_are_left_alone(zp):
    # rows of q behind the last request
    p = _params(4, 2, 64, 16)
    for n in (1, 50):
        pool = torch.randn((1, 8, 2, 2, 16, 64), device="cuda").to(torch.bfloat16)
        q = torch.randn((n + 9, 4, 64), device="cuda").to(torch.bfloat16)
        out = torch.full_like(q, 7.0)
        ws = zp.new_workspace(zp.zp_paged_window_workspace_size(p, n + 9, 1, n, 8, 9, 0))
        i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")
        zp.zp_paged_window_attn(pool, 0, q, i32(0, n), torch.arange(8, dtype=torch.int32, device="cuda")[None], i32(100), out, p, ws,
                                9, 0, n)
        assert zp.zp_read_error(ws) == 0
        assert bool((out[n:] == 7).all()) and not bool((out[:n] == 7).any())


@pytest.mark.gpu
@pytest.mark.parametrize("max_q", [200, 2 ** 31 - 1])
def test_window_takes_a_loose_bound_on_the_new_tokens(zp, max_q):
    _window_case(zp, 4, 2, 64, 16, [300, 5, 0], [3, 1, 20], 100, 4, seed=14, max_q=max_q, rel=TILED)
    _window_case(zp, 4, 2, 128, 16, [3000], [70], 0, 0, seed=15, max_q=max_q, rel=TILED)


@pytest.mark.gpu
def test_window_values_in_split_items(zp):
    # a few rows over a long cache share their tiles between CTAs; one of the last values is not
    # finite and only the last rows see it
    def poison(x, tables):
        x[tables[0, 3059 // 16], 1, 0, 3059 % 16, 11] = math.nan
    _window_case(zp, 4, 2, 64, 16, [3000], [70], 0, 0, seed=16, poison=poison, rel=TILED)


@pytest.mark.gpu
def test_window_long_items_before_short_ones(zp):
    # Every CTA takes one item of two query tiles, whose rows are computed plainly (slowly, and the
    # second tile's longer than the first's) because a value that only the last of them sees is not
    # finite, and then nine items of one tile, which the second group of warps has no part in.
    heavy, light = 76, 76 * 9

    def poison(x, tables):
        for r in range(heavy):
            x[tables[r, 63 // 16], 1, :, 63 % 16, 5] = math.inf
    _window_case(zp, 8, 2, 64, 16, [0] * (heavy + light), [64] * heavy + [6] * light, 0, 0, seed=17, poison=poison, rel=TILED)


@pytest.mark.gpu
def test_both_forms_agree(zp):
    # the same rows through the split form (max_q 4) and the tiled one (an upper bound of 40)
    outs = []
    for mq in (4, 40):
        args = _window_case(zp, 4, 2, 128, 16, [50, 700], [4, 3], 128, 9, seed=6, max_q=mq, rel=TILED)
        outs.append(args[6].double())
    assert (outs[0] - outs[1]).abs().max() <= 2.0 ** -5


# ------------------------------------------------------------------ streams, graphs -----------

@pytest.mark.gpu
def test_results_repeat_and_streams_and_graphs_share_nothing(zp):
    rng = np.random.default_rng(9)
    lens = [5000, 300, 2222]
    kv8 = _kv8_case(zp, 8, 2, 128, 16, lens, seed=10, hidden_nan=False)
    win = _window_case(zp, 8, 2, 128, 16, [3000, 100], [1, 1], 2500, 4, seed=11, rel=SPLIT)
    tile = _window_case(zp, 4, 2, 128, 16, [300], [90], 200, 4, seed=12, rel=TILED)
    calls = [(zp.zp_kv8_decode_attn, kv8, 6), (zp.zp_paged_window_attn, win, 6), (zp.zp_paged_window_attn, tile, 6)]
    for fn, args, at in calls:
        want = args[at].clone()
        # two streams at once, a workspace each
        streams = [torch.cuda.Stream() for _ in range(2)]
        outs = []
        torch.cuda.synchronize()
        for s in streams:
            a = list(args)
            a[at] = torch.zeros_like(want)
            a[8] = torch.zeros_like(args[8])
            torch.cuda.synchronize()
            outs.append(a)
        for _ in range(20):
            for s, a in zip(streams, outs):
                fn(*a, stream=s)
        torch.cuda.synchronize()
        assert all(torch.equal(a[at], want) for a in outs)
        # two graphs with one workspace, replayed in turn
        graphs = []
        for a in outs:
            a[8] = outs[0][8]
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                fn(*a)
            graphs.append(g)
        for a in outs:
            a[at].zero_()
        for _ in range(5):
            for g in graphs:
                g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a[at], want) for a in outs)
        assert zp.zp_read_error(outs[0][8]) == 0
