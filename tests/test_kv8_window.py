"""Attention of a chunk of new tokens over the 8-bit pool (zp_kv8_window_attn): against 64 bits, and against the same call
over the unpacked pool."""
import math
import os

import numpy as np
import pytest
import torch

import test_cache_attention as A
from oracle import serving_oracle as S

# How far weights are held: f16, half a step is 2^-11 of the value.  In the form for many rows values of scales that are not powers
# of two are rounded too, the block's scale over the tile's and its product with the code: 2^-11 each, so p (1 + e1) v (1 + e2) (1 + e3)
# is off by 3 * 2^-11 and terms of 2^-22.
FEW, MANY = 2.0 ** -11, 3 * 2.0 ** -11


@pytest.fixture(scope="module")
def zp():
    from paged_kv_cache_obs_gb300 import build
    if not os.path.exists(build.LIB):
        build.build()
    from paged_kv_cache_obs_gb300 import zipage
    return zipage


def _i32(x):
    return torch.as_tensor(np.ascontiguousarray(x), dtype=torch.int32).cuda()


# ------------------------------------------------------------------ refusals (CPU) ------------

def test_refuses(zp):
    ws, base, x, p = A._host(zp)
    rows = A._rows(zp, x)

    def call(pool=zp.zp_kv8_pool(base, base, 4), layer=0, q=rows, start=base, T=2, max_q=1, tables=base, seq=base, B=2, mb=2, window=4,
             sinks=1, out=rows, params=zp.make_params(p), ws=base, nb=1 << 40):
        return zp.lib.zp_kv8_window_attn(pool, layer, q, start, T, max_q, tables, seq, B, mb, window, sinks, out, params, ws, nb, None)

    A._refusals(zp, call, base, x, p)
    for kw in (dict(start=None), dict(T=-1), dict(max_q=0), dict(pool=zp.zp_kv8_pool(None, base, 4)), dict(pool=zp.zp_kv8_pool(base, None, 4)),
               dict(pool=zp.zp_kv8_pool(base + 8, base, 4)), dict(pool=zp.zp_kv8_pool(base, base + 1, 4)), dict(pool=zp.zp_kv8_pool(base, base, 0)),
               dict(out=zp.zp_rows(base, 0, 64))):
        assert call(**kw) == zp.ZP_ERR_INVALID_ARG, kw
    assert call(pool=zp.zp_kv8_pool(base, base, 1 << 31)) == zp.ZP_ERR_UNSUPPORTED
    assert call(B=0, q=None, out=None, tables=None, seq=None, start=None) == zp.ZP_OK
    assert call(T=0, q=zp.zp_rows(None, 0, 0), out=zp.zp_rows(None, 0, 0)) == zp.ZP_OK
    for mq in (2, 40):
        need = zp.zp_kv8_window_workspace_size(p, 2, 1, mq, 4096, 0, 0)
        assert need % 256 == 0 and call(mb=4096, B=1, window=0, max_q=mq, nb=need - 1) == (zp.ZP_ERR_INVALID_ARG)


def test_binding_refuses(zp):
    p = A._params(2, 2, 64, 16)
    bf, ws = torch.zeros((4, 2, 64), dtype=torch.bfloat16), torch.zeros(256, dtype=torch.uint8)
    codes, scales = torch.zeros((1, 4, 2, 2, 16, 64), dtype=torch.uint8), torch.zeros((1, 4, 2, 2))
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)
    good = dict(codes=codes, scales=scales, layer=0, q=bf, q_start=i32(3), block_tables=i32(2, 6), seq_lens=i32(2), out=bf.clone(), params=p,
                workspace=ws, window=0, sinks=0, max_q=2)
    for kw in (dict(codes=codes.view(torch.float8_e5m2)), dict(scales=scales.double()), dict(scales=scales[:, :3]), dict(q=bf[:3]), dict(out=bf[:, :1]),
               dict(q_start=i32(2)), dict(block_tables=i32(1, 6)), dict(seq_lens=i32(2, 2)), dict(max_q=1 << 31)):
        with pytest.raises(ValueError, match="expected"):
            zp.zp_kv8_window_attn(**{**good, **kw})
    with pytest.raises(ValueError, match="current CUDA device"):
        zp.zp_kv8_window_attn(**good)


# ------------------------------------------------------------------ GPU -----------------------

def _pool(rng, NB, layers, Hkv, b, d, scale_exp=(-8, -4), plain=False):
    codes = S.e4m3_encode(np.clip(rng.standard_normal((layers, NB, 2, Hkv, b, d)) * 64, -448, 448))
    scales = 2.0 ** rng.integers(*scale_exp, (layers, NB, 2, Hkv)) * (1.0 if plain else 1 + rng.random((layers, NB, 2, Hkv)))
    return codes, scales.astype(np.float32)


def _exact_pool(codes, scales):
    """What is attended to, in 64 bits."""
    return codes.view(torch.float8_e4m3fn).double() * scales.double()[..., None, None]


def _case(zp, Hq, Hkv, d, b, cached, new, window=0, sinks=0, seed=0, max_q=None, off=0, expect=0, hidden_nan=True, skip=(), start_edit=None,
          seq_edit=None, tables_edit=None, pad=0, scale_exp=(-8, -4), gain=2.0, ws_bytes=None, plain=False, check=True):
    """Ragged requests over layer 1 of two; tokens that none of a request's rows sees hold NaN."""
    rng = np.random.default_rng(seed)
    G, B = Hq // Hkv, len(new)
    lens = [c + n for c, n in zip(cached, new)]
    tables, NB = A._tables(rng, lens, b)
    codes, scales = _pool(rng, NB, 2, Hkv, b, d, scale_exp, plain)
    if hidden_nan:
        for r in range(B):
            seen = np.zeros(-(-lens[r] // b) * b, dtype=bool)
            for i in range(new[r]):
                seen[:lens[r]] |= S.window_visible(cached[r] + i, lens[r], window, sinks)
            for t in np.nonzero(~seen)[0]:
                codes[1, tables[r, t // b], :, :, t % b] = 0x7F
    T = sum(new) + pad
    start = [0] + np.cumsum(new).tolist()
    q = torch.from_numpy(rng.standard_normal((T, Hq, d)) * gain).to(torch.bfloat16)
    q[sum(new):] = math.nan
    n = q.numel()
    buf = torch.zeros(n + 8, dtype=torch.bfloat16)
    buf[off:off + n] = q.flatten()
    dq = buf.cuda()[off:off + n].view(T, Hq, d)
    obuf = torch.full((n + 8,), 7.0, dtype=torch.bfloat16, device="cuda")
    out = obuf[off:off + n].view(T, Hq, d)
    p = A._params(Hq, Hkv, d, b, 2)
    mq = max_q or max(1, max(new))
    ws = zp.new_workspace(zp.zp_kv8_window_workspace_size(p, T, B, mq, tables.shape[1], window, sinks) if ws_bytes is None else ws_bytes)
    args = (torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda(), 1, dq, _i32(start if start_edit is None else start_edit(list(start))),
            torch.from_numpy(tables.copy() if tables_edit is None else tables_edit(tables.copy())).cuda(),
            _i32(lens if seq_edit is None else seq_edit(list(lens))), out, p, ws, window, sinks, mq)
    for _ in range(2):
        zp.zp_kv8_window_attn(*args)
    assert zp.zp_read_error(ws) == expect
    rest = obuf.clone()
    rest[off:off + sum(new) * Hq * d] = 7.0
    assert bool((rest == 7).all())                          # nothing around the requests' rows
    rel = FEW if G * mq <= 16 else MANY
    pool = _exact_pool(args[0][1], args[1][1])
    for r in range(B):
        rows = slice(start[r], start[r + 1])
        if r in skip:
            assert bool((out[rows] == 7).all())
        elif new[r] and check:
            _check(pool, torch.from_numpy(tables[r]).cuda(), dq[rows], out[rows], lens[r], window, sinks, p, rel, r)
    return args


def _exact_rows(pool, table, q, L, window, sinks, p):
    """Outputs and weighted magnitudes [n, Hq, d] in 64 bits of one request's rows q over pool [blocks, 2, H, b, d]."""
    n, Hq, d = q.shape
    Hkv, b = p["num_kv_heads"], p["block_size"]
    pos, t = torch.arange(L - n, L, device="cuda")[:, None], torch.arange(L, device="cuda")
    see = (t <= pos) & ((t > pos - window) | (t < sinks) | (window == 0))
    some = see.any(0)
    kv = pool[table[:-(-L // b)].long()]
    want, mass = (torch.empty((n, Hq, d), dtype=torch.float64, device="cuda") for _ in range(2))
    for h in range(Hq):
        k, v = (torch.where(some[:, None], kv[:, i, h // (Hq // Hkv)].reshape(-1, d)[:L], 0.0) for i in (0, 1))
        w = torch.softmax((p["scale"] * (q[:, h].double() @ k.T)).masked_fill(~see, -math.inf), -1)
        want[:, h], mass[:, h] = w @ v, w @ v.abs()
    return want, mass


def _check(pool, table, q, got, L, window, sinks, p, rel, where):
    want, mass = _exact_rows(pool, table, q, L, window, sinks, p)
    err = (got.double() - want).abs()
    # As in test_cache_attention; and weights below 2^-18 of the largest are held to 2^-29 of it (f16's last bit is 2^-24, half
    # of it 2^-25, and the largest weight stands at 2^4 or above), each times a value of up to the largest.
    most = pool[table[:-(-L // p["block_size"])].long(), 1].abs().nan_to_num(0.0).max()
    tol = 2.0 ** -8 * want.abs() + (rel + 2.0 ** -14) * mass + (rel == MANY) * 2.0 ** -29 * L * most + 1e-30
    assert bool((err <= tol).all()), (where, float((err / tol).max()))


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,Hkv,d,b", A.SHAPES)
def test_single_tokens(zp, Hq, Hkv, d, b):
    _case(zp, Hq, Hkv, d, b, [0, 1, b - 1, b, 254, 700, 1999], [1] * 7, 100, 5, seed=Hq)
    _case(zp, Hq, Hkv, d, b, [0, 300], [1, 1], seed=Hq + 1)


@pytest.mark.gpu
@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (2, 1), (16, 17), (100, 0), (64, 64), (5000, 3)])
def test_few_tokens(zp, window, sinks):
    _case(zp, 8, 2, 128, 16, [0, 5, 0, 300, 31, 63], [3, 1, 0, 2, 4, 4], window, sinks, seed=window)
    _case(zp, 4, 1, 64, 32, [200, 0, 30], [4, 2, 3], window, sinks, seed=sinks, pad=2)
    _case(zp, 2, 2, 64, 16, [200, 0, 30, 9], [16, 2, 3, 11], window, sinks, seed=sinks)
    _case(zp, 7, 1, 128, 32, [500, 1], [2, 2], window, sinks, seed=sinks, off=1)


@pytest.mark.gpu
def test_few_tokens_of_long_caches(zp):
    _case(zp, 8, 2, 128, 16, [9000, 1, 4097], [3, 4, 4], seed=1)
    _case(zp, 14, 2, 64, 32, [5000, 130], [2, 1], window=4000, sinks=7, seed=2)


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,Hkv,d,b", [(32, 8, 128, 16), (28, 4, 128, 32), (8, 8, 64, 16), (16, 2, 64, 32), (16, 1, 128, 16), (3, 1, 64, 16), (1, 1, 128, 32)])
def test_chunks(zp, Hq, Hkv, d, b):
    _case(zp, Hq, Hkv, d, b, [0, 17, 130, 5], [40, 33, 1, 0], 50, 5, seed=Hq, pad=3)
    _case(zp, Hq, Hkv, d, b, [0, 260, 31], [300, 17, 129], seed=Hq)


@pytest.mark.gpu
@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (1, 1), (16, 17), (100, 0), (128, 128), (129, 300), (70, 33), (5000, 3)])
def test_chunks_of_several_tiles(zp, window, sinks):
    _case(zp, 4, 2, 128, 16, [0, 333], [150, 129], window, sinks, seed=window)
    _case(zp, 2, 2, 64, 32, [100, 0], [300, 257], window, sinks, seed=sinks)


@pytest.mark.gpu
def test_long_chunks_and_caches(zp):
    _case(zp, 2, 1, 128, 16, [0], [1500], 700, 4, seed=1)
    _case(zp, 7, 1, 64, 32, [2500], [40], seed=2)
    _case(zp, 4, 1, 128, 32, [6000, 10], [17, 64], seed=3, off=1)


@pytest.mark.gpu
@pytest.mark.parametrize("new", [4, 80])
@pytest.mark.parametrize("lo,hi", [(-60, -50), (40, 50), (-12, 2), (-100, -90)])
def test_scales_of_any_size(zp, new, lo, hi):
    _case(zp, 8, 2, 128, 16, [300, 33], [new, new], seed=3, scale_exp=(lo, hi), gain=min(2.0 ** -(hi + 6), 2.0 ** 90))
    _case(zp, 8, 2, 64, 32, [300, 33], [new, new], seed=3, scale_exp=(lo, hi), gain=min(2.0 ** -(hi + 6), 2.0 ** 90), plain=True)


@pytest.mark.gpu
@pytest.mark.parametrize("d,b", [(128, 16), (128, 32), (64, 16), (64, 32)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (150, 20)])
def test_every_code(zp, d, b, window, sinks):
    """All codes that are numbers, under scales as the library writes them; and over blocks of a pool that the library
    packed, the values of the pool."""
    rng = np.random.default_rng(d + b)
    Hq, Hkv, new, cached = 4, 2, [200, 37, 64], [0, 300, 700]
    lens = [c + n for c, n in zip(cached, new)]
    tables, NB = A._tables(rng, lens, b)
    p = A._params(Hq, Hkv, d, b)
    T, mb = sum(new), tables.shape[1]
    q = torch.from_numpy(rng.standard_normal((T, Hq, d)) / 4).to(torch.bfloat16).cuda()
    start, seq, dt = _i32(np.concatenate([[0], np.cumsum(new)])), _i32(lens), torch.from_numpy(np.where(tables < 0, 0, tables).astype(np.int32)).cuda()
    ws = zp.new_workspace(max(zp.zp_kv8_window_workspace_size(p, T, 3, 200, mb, window, sinks), 256))

    def attend(c, s):
        out = torch.full_like(q, 7.0)
        zp.zp_kv8_window_attn(c, s, 0, q, start, dt, seq, out, p, ws, window, sinks, 200)
        assert zp.zp_read_error(ws) == 0
        for r, L in enumerate(lens):
            rows = slice(start[r].item(), start[r + 1].item())
            _check(_exact_pool(c[0], s[0]), dt[r], q[rows], out[rows], L, window, sinks, p, MANY, r)
        return out
    codes = rng.integers(0, 0x7F, (1, NB, 2, Hkv, b, d)) + 0x80 * rng.integers(0, 2, (1, NB, 2, Hkv, b, d))
    scales = 2.0 ** rng.integers(-8, -4, (1, NB, 2, Hkv))
    attend(torch.from_numpy(codes.astype(np.uint8)).cuda(), torch.from_numpy(scales.astype(np.float32)).cuda())
    # packed from bf16 blocks of very different sizes, one of zeros: the same as from the bf16 pool read back
    ids = torch.arange(NB, dtype=torch.int32, device="cuda")
    pool = (torch.randn((1, NB, 2, Hkv, b, d), device="cuda") * 2.0 ** torch.randint(-6, 3, (1, NB, 2, Hkv, 1, 1), device="cuda")).to(torch.bfloat16)
    pool[0, int(tables[2][1])] = 0
    c, s = torch.zeros(pool.shape, dtype=torch.uint8, device="cuda"), torch.zeros((1, NB, 2, Hkv), device="cuda")
    zp.zp_kv8_pack_blocks(pool, ids, c, s, ids, p, ws)
    got = attend(c, s)
    zp.zp_kv8_unpack_blocks(c, s, ids, pool, ids, p, ws)
    want = torch.full_like(q, 7.0)
    wws = zp.new_workspace(zp.zp_paged_window_workspace_size(p, T, 3, 200, mb, window, sinks))
    zp.zp_paged_window_attn(pool, 0, q, start, dt, seq, want, p, wws, window, sinks, 200)
    for r, L in enumerate(lens):                                # both are near the exact rows
        rows = slice(start[r].item(), start[r + 1].item())
        exact, mass = _exact_rows(_exact_pool(c[0], s[0]), dt[r], q[rows], L, window, sinks, p)
        tol = 2.0 ** -8 * (2 * exact.abs() + mass) + (MANY + 2.0 ** -13) * mass + 2.0 ** -29 * L * pool.float().abs().max() + 1e-30
        assert bool(((got[rows].double() - want[rows].double()).abs() <= tol).all())


@pytest.mark.gpu
@pytest.mark.parametrize("d,b", [(128, 16), (64, 32)])
@pytest.mark.parametrize("new", [4, 70])
def test_keys_with_scales_of_every_kind(zp, d, b, new):
    """Scales of 0 and below, of many bits, subnormal: logits are code * scale as they are."""
    rng = np.random.default_rng(new)
    Hq, Hkv, L = 4, 2, 900 + new
    tables, NB = A._tables(rng, [L], b)
    codes, scales = _pool(rng, NB, 1, Hkv, b, d)
    scales[0, :, 0] = rng.choice(np.array([0.0, -0.0, -2.0 ** -6, 2.0 ** -6, -0.01, 0.013, 2.0 ** -140, 1e-30, 3e-3], dtype=np.float32), (NB, Hkv))
    q = torch.from_numpy(rng.standard_normal((new, Hq, d)) * 2).to(torch.bfloat16).cuda()
    p, rel = A._params(Hq, Hkv, d, b), FEW if 2 * new <= 16 else MANY
    c, s, dt = torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda(), torch.from_numpy(tables).cuda()
    for window, sinks in ((0, 0), (333, 20)):
        out = torch.full_like(q, 7.0)
        ws = zp.new_workspace(zp.zp_kv8_window_workspace_size(p, new, 1, new, tables.shape[1], window, sinks))
        zp.zp_kv8_window_attn(c, s, 0, q, _i32([0, new]), dt, _i32([L]), out, p, ws, window, sinks, new)
        assert zp.zp_read_error(ws) == 0
        _check(_exact_pool(c[0], s[0]), dt[0], q, out, L, window, sinks, p, rel, window)


@pytest.mark.gpu
@pytest.mark.parametrize("d,b", [(128, 32), (64, 16)])
@pytest.mark.parametrize("new", [4, 70])
def test_values_with_scales_of_every_kind(zp, d, b, new):
    """Scales of 0 and below, of many bits, 2^90 apart from one 128 tokens to the next, and up to 2^15 apart within."""
    rng = np.random.default_rng(new)
    Hq, Hkv, L = 4, 2, 900 + new
    tables, NB = A._tables(rng, [L], b)
    codes, scales = _pool(rng, NB, 1, Hkv, b, d)
    per = 128 // b
    q = torch.from_numpy(rng.standard_normal((new, Hq, d)) * 2).to(torch.bfloat16).cuda()
    p, rel = A._params(Hq, Hkv, d, b), FEW if 2 * new <= 16 else MANY
    c, dt = torch.from_numpy(codes).cuda(), torch.from_numpy(tables).cuda()
    for spread in (0, 12, 45):
        for i in range(-(-L // b)):
            far = 2.0 ** (spread * ((i // per) % 3 - 1)) if spread else 1.0
            scales[0, tables[0, i], 1] = rng.choice(np.array([0.0, -2.0 ** -6, 2.0 ** -6, 2.0 ** -7, -0.01, 0.013, 0.9, 2.0 ** -15, 3e-3], dtype=np.float64)) * far
        s = torch.from_numpy(scales).cuda()
        out = torch.full_like(q, 7.0)
        ws = zp.new_workspace(zp.zp_kv8_window_workspace_size(p, new, 1, new, tables.shape[1], 0, 0))
        zp.zp_kv8_window_attn(c, s, 0, q, _i32([0, new]), dt, _i32([L]), out, p, ws, 0, 0, new)
        assert zp.zp_read_error(ws) == 0
        _check(_exact_pool(c[0], s[0]), dt[0], q, out, L, 0, 0, p, rel, spread)


@pytest.mark.gpu
@pytest.mark.parametrize("ratio", [30.0, 2.0 ** 14, 2.0 ** 40, 2.0 ** 90])
@pytest.mark.parametrize("d", [64, 128])
def test_values_behind_a_block_of_a_larger_scale(zp, d, ratio):
    """Blocks of weight 0 with a V scale `ratio` times the others' come first, then one token takes most of the weight with a
    value of 0, and the result is the sum of 4000 equal weights of e^-9 of it."""
    p = A._params(1, 1, d, 16, scale=0.125)
    NB, new = 8 + 8 + 256, 20
    L = NB * 16
    codes = np.zeros((1, NB, 2, 1, 16, d), dtype=np.uint8)
    enc = lambda v: S.e4m3_encode(np.array(float(v)))
    codes[0, :, 0, 0, :, 0] = enc(-9)
    codes[0, :, 1, 0] = enc(1.5)
    codes[0, :8, 0, 0, :, 0] = enc(-88)
    codes[0, 8, 0, 0, 0, 0] = 0
    codes[0, 8, 1, 0, 0] = 0
    scales = np.ones((1, NB, 2, 1), dtype=np.float32)
    scales[0, :, 1] = 2.0 ** -6
    scales[0, :8, 1] = 2.0 ** -6 * ratio
    q = torch.zeros((new, 1, d), dtype=torch.bfloat16, device="cuda")
    q[:, 0, 0] = 8.0
    out = torch.zeros_like(q)
    tables = np.arange(NB, dtype=np.int32)[None]
    ws = zp.new_workspace(256)
    c, s = torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda()
    zp.zp_kv8_window_attn(c, s, 0, q, _i32([0, new]), _i32(tables), _i32([L]), out, p, ws, 0, 0, new)
    assert zp.zp_read_error(ws) == 0
    _check(_exact_pool(c[0], s[0]), torch.arange(NB, device="cuda"), q, out, L, 0, 0, p, MANY, ratio)


@pytest.mark.gpu
@pytest.mark.parametrize("gain", [2.0 ** 10, 2.0 ** 16, 2.0 ** 24])
def test_queries_with_one_large_value(zp, gain):
    """A value of the query `gain` times the others, where the keys are 0: the logits are the others'."""
    rng = np.random.default_rng(5)
    Hq, d, b, new, L = 4, 128, 16, 60, 300
    tables, NB = A._tables(rng, [L], b)
    codes, scales = _pool(rng, NB, 1, 1, b, d)
    codes[0, :, 0, :, :, 77] = 0
    q = torch.from_numpy(rng.standard_normal((new, Hq, d)) * 2).to(torch.bfloat16).cuda()
    q[:, :, 77] = gain
    p = A._params(Hq, 1, d, b)
    out = torch.full_like(q, 7.0)
    ws = zp.new_workspace(zp.zp_kv8_window_workspace_size(p, new, 1, new, tables.shape[1], 0, 0))
    c, s, dt = torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda(), torch.from_numpy(tables).cuda()
    zp.zp_kv8_window_attn(c, s, 0, q, _i32([0, new]), dt, _i32([L]), out, p, ws, 0, 0, new)
    assert zp.zp_read_error(ws) == 0
    _check(_exact_pool(c[0], s[0]), dt[0], q, out, L, 0, 0, p, MANY, gain)


@pytest.mark.gpu
@pytest.mark.parametrize("new", [3, 4, 70])
@pytest.mark.parametrize("d,b,Hq", [(64, 16, 4), (128, 32, 4), (64, 32, 8), (128, 16, 8)])
def test_nan_reaches_only_the_rows_that_see_it(zp, new, d, b, Hq):
    """Codes that are NaN, in V at tokens that later rows see and earlier ones do not or that leave the window, and in K
    of a token that the last row alone sees."""
    rng = np.random.default_rng(new)
    Hkv, window, sinks, L = 2, 6, 2, 200 + new
    tables, NB = A._tables(rng, [L], b)
    codes, scales = _pool(rng, NB, 1, Hkv, b, d)
    at = lambda t: (0, tables[0, t // b])
    for t, dim in ((L - 2, 7), (195, 60), (1, 33)):
        codes[at(t) + (1, 0, t % b, dim)] = 0x7F if dim != 60 else 0xFF
    codes[at(L - 1) + (0, 1, (L - 1) % b, 5)] = 0x7F                     # K of the second kv head
    q = torch.from_numpy(rng.standard_normal((new, Hq, d)) * 2).to(torch.bfloat16).cuda()
    p = A._params(Hq, Hkv, d, b)
    out = torch.full_like(q, 7.0)
    ws = zp.new_workspace(zp.zp_kv8_window_workspace_size(p, new, 1, new, tables.shape[1], window, sinks))
    c, s, dt = torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda(), torch.from_numpy(tables).cuda()
    zp.zp_kv8_window_attn(c, s, 0, q, _i32([0, new]), dt, _i32([L]), out, p, ws, window, sinks, new)
    assert zp.zp_read_error(ws) == 0
    G, nan = Hq // Hkv, torch.isnan(out).cpu()
    want = torch.zeros_like(nan)
    for i in range(new):
        vis = S.window_visible(200 + i, L, window, sinks)
        for t, dim in ((L - 2, 7), (195, 60), (1, 33)):
            if vis[t]:
                want[i, :G, dim] = True
    want[new - 1, G:] = True
    assert torch.equal(nan, want)
    clean = np.where((codes & 0x7F) == 0x7F, 0, codes)
    rel = FEW if G * new <= 16 else MANY
    pool = _exact_pool(torch.from_numpy(clean).cuda()[0], s[0])
    exact, mass = _exact_rows(pool, dt[0], q, L, window, sinks, p)
    fine = ~want.cuda()
    tol = 2.0 ** -8 * exact.abs() + (rel + 2.0 ** -14) * mass + 2.0 ** -29 * L * pool[:, 1].abs().max() + 1e-30      # as in _check
    assert bool(((out.double() - exact).abs() <= tol)[fine].all())


@pytest.mark.gpu
@pytest.mark.parametrize("new", [2, 60])
def test_skips_bad_rows_and_reports(zp, new):
    kw = dict(window=40, sinks=2, seed=5, expect=zp.ZP_ERR_BAD_TABLE, skip=(1,))
    cached, n = [30, 60, 9], [new, new, new]

    def put(i, v):
        def edit(x):
            x[i] = v
            return x
        return edit
    for bad in (-1, new - 1, 10 ** 6, 2 ** 31 - 1):
        _case(zp, 4, 2, 64, 16, cached, n, seq_edit=put(1, bad), **kw)
    for bad in (10 ** 6, -1):
        _case(zp, 4, 2, 64, 16, cached, n, tables_edit=put((1, (60 + new - 1) // 16), bad), **kw)
    _case(zp, 4, 2, 64, 16, cached, [new, new + 5, new], max_q=new + 4, **kw)
    _case(zp, 4, 2, 64, 16, [30, 60], [new, new], start_edit=put(2, 2 ** 31 - 1), **kw)


@pytest.mark.gpu
@pytest.mark.parametrize("new", [2, 40])
def test_entries_that_no_row_sees_are_not_read(zp, new):
    """Between the first tokens and the window a table may hold anything."""
    outs = []
    for hidden in (None, -5):
        def edit(t):
            if hidden is not None:
                t[0, 2:10] = hidden
            return t
        outs.append(_case(zp, 4, 1, 128, 16, [400], [new], 200, 20, seed=8, tables_edit=edit, check=hidden is None)[7])
    assert torch.equal(*outs)


@pytest.mark.gpu
@pytest.mark.parametrize("new,window", [(2, 0), (2, 3000), (70, 0), (300, 0)])
def test_workspaces_of_other_batches(zp, new, window):
    args = _case(zp, 4, 1, 64, 16, [9000], [new], window, 4, seed=new)
    own = args[9].numel()
    assert own > 256
    pool = _exact_pool(args[0][1], args[1][1])
    for n in (256, own // 512 * 256, own, own + 256):
        buf = torch.zeros(n + 512, dtype=torch.uint8, device="cuda")
        buf[n:] = 0xA5
        out = torch.full_like(args[7], 7.0)
        for _ in range(2):
            zp.zp_kv8_window_attn(*args[:7], out, args[8], buf[:n], *args[10:])
        torch.cuda.synchronize()
        assert bool((buf[n:] == 0xA5).all()) and int(buf[:4].view(torch.int32)) == 0
        _check(pool, args[5][0], args[3], out, 9000 + new, window, 4, args[8], FEW if 4 * new <= 16 else MANY, n)
    with pytest.raises(zp.ZipageError):
        zp.zp_kv8_window_attn(*args[:9], torch.zeros(own - 1, dtype=torch.uint8, device="cuda"), *args[10:])


@pytest.mark.gpu
@pytest.mark.parametrize("new", [3, 200])
def test_a_wait_that_runs_out_is_reported(zp, new):
    args = _case(zp, 4, 2, 128, 16, [700, 40, 300], [new] * 3, seed=11)
    zp.zp_test_kv8_window_stalled(*args[:7], torch.zeros_like(args[7]), *args[8:], 1000000)
    assert zp.zp_read_error(args[9]) == zp.ZP_ERR_TIMEOUT
    again = torch.zeros_like(args[7])
    zp.zp_kv8_window_attn(*args[:7], again, *args[8:])
    assert zp.zp_read_error(args[9]) == zp.ZP_OK and torch.equal(again, args[7])
    for ns in (0, -1, 10 ** 9 + 1):
        with pytest.raises(zp.ZipageError):
            zp.zp_test_kv8_window_stalled(*args, ns)


@pytest.mark.gpu
@pytest.mark.parametrize("new", [4, 50])
def test_offsets_past_32_bits(zp, new):
    """A pool of 4.6 G codes whose last blocks are a request's."""
    Hkv, d, b, NB = 8, 128, 32, 70000
    p = A._params(16, Hkv, d, b)
    codes = torch.zeros((1, NB, 2, Hkv, b, d), dtype=torch.uint8, device="cuda")
    scales = torch.zeros((1, NB, 2, Hkv), device="cuda")
    ids = [NB - 1, 3, NB - 2, NB - 7]
    g = torch.Generator(device="cuda").manual_seed(1)
    for i in ids:
        codes[0, i] = (torch.randn((2, Hkv, b, d), generator=g, device="cuda") * 64).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        scales[0, i] = 2.0 ** -6
    q = torch.randn((new, 16, d), generator=g, device="cuda").to(torch.bfloat16)
    out, L = torch.zeros_like(q), 120
    ws = zp.new_workspace(zp.zp_kv8_window_workspace_size(p, new, 1, new, 4, 0, 0))
    zp.zp_kv8_window_attn(codes, scales, 0, q, _i32([0, new]), _i32([ids]), _i32([L]), out, p, ws, 0, 0, new)
    assert zp.zp_read_error(ws) == 0
    pool = codes[0, ids].view(torch.float8_e4m3fn).double() * scales[0, ids].double()[..., None, None]
    _check(pool, torch.arange(4, device="cuda"), q, out, L, 0, 0, p, FEW if new == 4 else MANY, new)


@pytest.mark.gpu
@pytest.mark.parametrize("new", [3, 60])
def test_captured_and_replayed(zp, new):
    args = _case(zp, 4, 2, 64, 16, [300, 20], [new, new], 0, 0, seed=12, pad=4)
    want = args[7].clone()
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        zp.zp_kv8_window_attn(*args)
    args[7].fill_(7.0)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(args[7], want)
    args[6].copy_(_i32([200 + new, 10 + new]))           # shorter caches: the same captured call
    graph.replay()
    pool = _exact_pool(args[0][1], args[1][1])
    for r, L in enumerate((200 + new, 10 + new)):
        rows = slice(r * new, (r + 1) * new)
        _check(pool, args[5][r], args[3][rows], args[7][rows], L, 0, 0, args[8], FEW if 2 * new <= 16 else MANY, r)
    assert zp.zp_read_error(args[9]) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,Hkv,d,b", [(16, 8, 128, 16), (28, 4, 64, 32)])
def test_many_requests_of_one_query_tile(zp, Hq, Hkv, d, b):
    """CTAs take several items one after another of which one softmax group has no part; here and there one has two tiles."""
    rng = np.random.default_rng(d)
    tile = 128 // (Hq // Hkv)
    for two in (0.0, 0.3):
        new = [int(rng.integers(1, tile + 1)) + (tile if rng.random() < two else 0) for _ in range(120)]
        _case(zp, Hq, Hkv, d, b, rng.integers(0, 300, 120).tolist(), new, seed=b)


@pytest.mark.gpu
@pytest.mark.parametrize("G,d,b", [(4, 64, 16), (7, 128, 32)])
def test_split_requests_of_one_query_tile(zp, G, d, b):
    """100 items of up to 46 tiles are cut into 3 parts, of which CTAs take two or more; those of short caches have no tiles."""
    rng = np.random.default_rng(G)
    tile = 128 // G
    cached = [int(rng.integers(4000, 5800)) if r % 3 else int(rng.integers(0, 200)) for r in range(50)]
    args = _case(zp, 2 * G, 2, d, b, cached, [int(rng.integers(17, tile + 1)) for _ in cached[:-1]] + [17], seed=G)
    assert args[9].numel() > 256 + 2 * args[3].numel() * 4


@pytest.mark.gpu
def test_bad_blocks_between_parts_without_tiles(zp):
    """A wide table cuts requests of one tile into parts that mostly have none: the warps that bring tiles run far ahead, and what
    they note of bad blocks stays with its request."""
    B, new, wide = 153, 20, 50000
    bad = tuple(r for r in range(B) if r % 3)

    def edit(t):
        w = np.zeros((B, wide), dtype=np.int32)
        w[:, :t.shape[1]] = t
        for r in bad:
            w[r, 1] = -1 if r % 2 else 10 ** 6
        return w
    _case(zp, 4, 1, 64, 16, [12] * B, [new] * B, seed=3, tables_edit=edit, expect=zp.ZP_ERR_BAD_TABLE, skip=bad, ws_bytes=32 * B * new * 4 * 68 * 4 + 256)


@pytest.mark.gpu
def test_random_calls(zp):
    rng = np.random.default_rng(21)
    for i in range(60):
        Hkv, G = int(rng.integers(1, 4)), int(rng.integers(1, 17))
        B, top = int(rng.integers(1, 6)), int(rng.choice([4, 30, 300]))
        new = [int(x) for x in rng.integers(0, top + 1, B)]
        cached = [int(x) for x in rng.integers(0, rng.choice([3, 100, 900]), B)]
        _case(zp, G * Hkv, Hkv, int(rng.choice([64, 128])), int(rng.choice([16, 32])), cached, new, int(rng.choice([0, rng.integers(1, 700)])),
              int(rng.choice([0, rng.integers(1, 200)])), seed=i, off=int(rng.choice([0, 1])), pad=int(rng.integers(0, 20)),
              max_q=max(max(new), 1) + int(rng.integers(0, 50)), plain=bool(rng.random() < 0.5))
