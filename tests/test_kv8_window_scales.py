"""Scales of the 8-bit pool in zp_kv8_window_attn: values of 0, scales far from one another, factors of the logits that leave fp32;
against 64 bits, for scales that are powers of two, to the bits that weights are held to."""
import os

import numpy as np
import pytest
import torch

import test_cache_attention as A
from oracle import serving_oracle as S

F16 = 2.0 ** -11        # half a step of the weights, relative to them


@pytest.fixture(scope="module")
def zp():
    from paged_kv_cache_obs_gb300 import build
    if not os.path.exists(build.LIB):
        build.build()
    from paged_kv_cache_obs_gb300 import zipage
    return zipage


def _i32(x):
    return torch.as_tensor(np.ascontiguousarray(x), dtype=torch.int32).cuda()


def _codes(rng, shape):
    return S.e4m3_encode(np.clip(rng.standard_normal(shape) * 64, -448, 448))


def _attend(zp, codes, scales, q, new, lens, tables, p, window=0, sinks=0):
    """Outputs of one call over layer 0 (a second call gives the same bits)."""
    T, B, mq = q.shape[0], len(lens), max(new)
    ws = zp.new_workspace(zp.zp_kv8_window_workspace_size(p, T, B, mq, tables.shape[1], window, sinks))
    start = _i32(np.concatenate([[0], np.cumsum(new)]))
    outs = [torch.full_like(q, 7.0) for _ in range(2)]
    for out in outs:
        zp.zp_kv8_window_attn(codes, scales, 0, q, start, tables, _i32(lens), out, p, ws, window, sinks, mq)
    assert zp.zp_read_error(ws) == 0 and torch.equal(outs[0].view(torch.int16), outs[1].view(torch.int16))
    return outs[0]


def _walked(scale, i0, n, L, window, sinks, G, b):
    """For queries i0 .. of an item and the V scales of a request's blocks: the largest of the 128 tokens that are walked together with
    each token, as a power of two at or above it (2^-104 at least), [L]."""
    first = max(0, L - n + i0 - window + 1) if window else 0
    last = min(n, i0 + 2 * (128 // G)) - 1 + L - n
    lo = first // b
    listed = list(range(min(-(-min(sinks, L) // b), lo))) + list(range(lo, last // b + 1))
    out = np.full(-(-L // b), 2.0 ** -104)
    for i in range(0, len(listed), 128 // b):
        part = listed[i:i + 128 // b]
        out[part] = max(2.0 ** -104, 2.0 ** np.ceil(np.log2(max(float(abs(scale[part]).max()), 2.0 ** -104))))
    return torch.from_numpy(np.repeat(out, b)[:L].copy()).cuda()


def _check(codes, scales, table, q, got, L, window, sinks, p, where, tiled=True):
    """One request's rows against 64 bits: the output's rounding; weights to half a step of f16, and what fp32 sums add; and what is below
    f16's range.  Few rows: weights end at 2^-29 of the row's largest.  Tiled: weights times the largest V scale S_t of the 128 tokens
    walked together, W_t, end at 2^-29 of the row's largest W, each off by as much of its value over S_t; and f16 holds scale / S_t and
    its product with a code, which end at 2^-25 each: a value of a scale below 2^-15 S_t is off by 2^-25 S_t (|code| + 1)."""
    n, Hq, d = q.shape
    Hkv, b = p["num_kv_heads"], p["block_size"]
    G = Hq // Hkv
    pos, t = torch.arange(L - n, L, device="cuda")[:, None], torch.arange(L, device="cuda")
    see = (t <= pos) & ((t > pos - window) | (t < sinks) | (window == 0))
    ids = table[:-(-L // b)].long()
    worst = 0.0
    for h in range(Hkv):
        k, v = ((codes[ids, i, h].view(torch.float8_e4m3fn).double() * scales[ids, i, h].double()[:, None, None]).reshape(-1, d)[:L] for i in (0, 1))
        v_scale = scales[ids, 1, h].cpu().numpy().astype(np.float64)
        for g in range(h * G, (h + 1) * G):
            w = torch.softmax((p["scale"] * (q[:, g].double() @ k.T)).masked_fill(~see, -torch.inf), -1)
            want, mass = w @ v, w @ v.abs()
            tol = 2.0 ** -8 * want.abs() + (F16 + 2.0 ** -14) * mass + 1e-38
            if not tiled:
                tol += 2.0 ** -29 * w.amax(-1, keepdim=True) * (see.double() @ v.abs())
            step = 2 * (128 // G)
            for i0 in range(0, n if tiled else 0, step):
                rows = slice(i0, i0 + step)
                top = _walked(v_scale, i0, n, L, window, sinks, G, b)[:, None]
                tol[rows] += 2.0 ** -29 * (w[rows] * top.T).amax(-1, keepdim=True) * (see[rows].double() @ (v.abs() / top))
                scale = torch.from_numpy(np.repeat(np.abs(v_scale), b)[:L]).cuda()[:, None]
                code = torch.where(scale > 0, v.abs() / scale, 0.0)
                tol[rows] += 2.0 ** -25 * (w[rows] @ ((scale < 2.0 ** -15 * top) * top * (code + (code > 0))))
            err = (got[:, g].double() - want).abs()
            assert bool((err <= tol).all()), (where, h, g, float((err / tol).max()))
            worst = max(worst, float((err / tol).max()))
    return worst


# ------------------------------------------------------------------ values of 0 ---------------

@pytest.mark.gpu
@pytest.mark.parametrize("exp", [-8, -30, -60])
@pytest.mark.parametrize("d,b,zeros", [(128, 16, 128), (64, 32, 256), (64, 16, 128), (128, 32, 300)])
def test_values_of_zero_first(zp, d, b, zeros, exp):
    """Tokens whose values are 0 (scale 0, as the library writes it) come first, then values of 2^exp."""
    rng = np.random.default_rng(zeros)
    Hq, Hkv, new, L = 4, 2, 70, 700
    tables, NB = A._tables(rng, [L], b)
    codes = _codes(rng, (1, NB, 2, Hkv, b, d))
    scales = 2.0 ** rng.integers(-8, -4, (1, NB, 2, Hkv))
    scales[0, :, 1] = 2.0 ** exp
    scales[0, tables[0, :zeros // b], 1] = 0
    codes[0, tables[0, :zeros // b], 1] = 0
    q = torch.from_numpy(rng.standard_normal((new, Hq, d)) * 2).to(torch.bfloat16).cuda()
    p = A._params(Hq, Hkv, d, b)
    c, s, dt = torch.from_numpy(codes).cuda(), torch.from_numpy(scales.astype(np.float32)).cuda(), torch.from_numpy(tables).cuda()
    for window, sinks in ((0, 0), (500, 20)):
        got = _attend(zp, c, s, q, [new], [L], dt, p, window, sinks)
        _check(c[0], s[0], dt[0], q, got, L, window, sinks, p, (exp, window))


@pytest.mark.gpu
@pytest.mark.parametrize("exp", [-8, -30, -60])
def test_values_of_zero_first_behind_a_request_of_large_ones(zp, exp):
    """CTAs take a request with scales of 2^20 and then one that begins with values of 0: its rows are those of a call by itself."""
    rng = np.random.default_rng(7)
    B, d, b, new, L = 330, 64, 16, 20, 300
    per = -(-L // b)
    codes = torch.from_numpy(_codes(rng, (1, B * per, 2, 1, b, d))).cuda()
    scales = torch.full((1, B * per, 2, 1), 2.0 ** -6, device="cuda")
    tables = torch.from_numpy(rng.permutation(B * per).reshape(B, per).astype(np.int32)).cuda()
    last = list(range(B // 2, B))
    scales[0, tables[:B // 2].long().flatten(), 1] = 2.0 ** 20
    scales[0, tables[last].long().flatten(), 1] = 2.0 ** exp
    scales[0, tables[last, :8].long().flatten(), 1] = 0.0
    q = torch.from_numpy(rng.standard_normal((B * new, 2, d)) * 2).to(torch.bfloat16).cuda()
    p = A._params(2, 1, d, b)
    got = _attend(zp, codes, scales, q, [new] * B, [L] * B, tables, p)
    for r in [0, 5] + last[::9] + [B - 1]:
        rows = slice(r * new, (r + 1) * new)
        _check(codes[0], scales[0], tables[r], q[rows], got[rows], L, 0, 0, p, r)
        alone = _attend(zp, codes, scales, q[rows].contiguous(), [new], [L], tables[r:r + 1], p)
        assert torch.equal(alone, got[rows])


@pytest.mark.gpu
@pytest.mark.parametrize("d,b", [(128, 32), (64, 16)])
@pytest.mark.parametrize("exp", [-8, -30, -60])
def test_values_of_zero_first_for_some_rows(zp, d, b, exp):
    """A window: the first rows see values of 2^20, the others begin with values of 0 and go on with 2^exp."""
    rng = np.random.default_rng(b)
    Hq, new, L, window = 2, 240, 520, 140
    tables, NB = A._tables(rng, [L], b)
    codes = _codes(rng, (1, NB, 2, 1, b, d))
    scales = 2.0 ** rng.integers(-8, -4, (1, NB, 2, 1))
    # the item's list starts at the window of position 280: its tiles of 128 tokens are 128 .. 255, 256 .. 383 and so on
    scales[0, tables[0, :256 // b], 1] = 2.0 ** 20
    scales[0, tables[0, 256 // b:384 // b], 1] = 0
    scales[0, tables[0, 384 // b:], 1] = 2.0 ** exp
    q = torch.from_numpy(rng.standard_normal((new, Hq, d)) * 2).to(torch.bfloat16).cuda()
    p = A._params(Hq, 1, d, b)
    c, s, dt = torch.from_numpy(codes).cuda(), torch.from_numpy(scales.astype(np.float32)).cuda(), torch.from_numpy(tables).cuda()
    got = _attend(zp, c, s, q, [new], [L], dt, p, window)
    _check(c[0], s[0], dt[0], q, got, L, window, 0, p, exp)


@pytest.mark.gpu
@pytest.mark.parametrize("new", [4, 60])
def test_values_of_zero_alone(zp, new):
    """All of a row's values are 0; and values of 0 behind others count in the sum of weights alone."""
    rng = np.random.default_rng(new)
    Hq, d, b, L = 4, 128, 16, 600
    tables, NB = A._tables(rng, [L], b)
    codes = _codes(rng, (1, NB, 2, 1, b, d))
    scales = 2.0 ** rng.integers(-8, -4, (1, NB, 2, 1))
    q = torch.from_numpy(rng.standard_normal((new, Hq, d)) * 2).to(torch.bfloat16).cuda()
    p, c, dt = A._params(Hq, 1, d, b), torch.from_numpy(codes).cuda(), torch.from_numpy(tables).cuda()
    scales[0, :, 1] = 0
    s = torch.from_numpy(scales.astype(np.float32)).cuda()
    assert bool((_attend(zp, c, s, q, [new], [L], dt, p) == 0).all())
    for large in (2.0 ** -90, 1.0, 2.0 ** 90):
        scales[0, tables[0, :8], 1] = large
        s = torch.from_numpy(scales.astype(np.float32)).cuda()
        got = _attend(zp, c, s, q, [new], [L], dt, p)
        _check(c[0], s[0], dt[0], q, got, L, 0, 0, p, large, tiled=4 * new > 16)


@pytest.mark.gpu
@pytest.mark.parametrize("exp", [27, 60, 100])
@pytest.mark.parametrize("d,b,zeros", [(128, 16, 128), (64, 32, 256), (64, 16, 300), (128, 32, 5000)])
def test_values_of_zero_before_large_ones(zp, d, b, zeros, exp):
    """Values of 0 count in the sum of weights also where those behind them are larger by more than fp32's range; the last case is cut
    into parts, of which the first ones see values of 0 alone."""
    rng = np.random.default_rng(zeros)
    Hq, Hkv, new, L = 4, 2, 40, zeros + 400
    tables, NB = A._tables(rng, [L], b)
    codes = _codes(rng, (1, NB, 2, Hkv, b, d))
    scales = 2.0 ** rng.integers(-8, -4, (1, NB, 2, Hkv))
    scales[0, :, 1] = 2.0 ** exp
    scales[0, tables[0, :zeros // b], 1] = 0
    q = torch.from_numpy(rng.standard_normal((new, Hq, d)) * 2).to(torch.bfloat16).cuda()
    p = A._params(Hq, Hkv, d, b)
    c, s, dt = torch.from_numpy(codes).cuda(), torch.from_numpy(scales.astype(np.float32)).cuda(), torch.from_numpy(tables).cuda()
    if zeros == 5000:
        assert zp.zp_kv8_window_workspace_size(p, new, 1, new, tables.shape[1], 0, 0) > 256 + 4 * new * Hq * (d + 4)
    got = _attend(zp, c, s, q, [new], [L], dt, p)
    _check(c[0], s[0], dt[0], q, got, L, 0, 0, p, exp)


# ------------------------------------------------------------------ factors of the logits -----

@pytest.mark.gpu
@pytest.mark.parametrize("new", [3, 20, 150])
@pytest.mark.parametrize("d,b", [(128, 16), (64, 32)])
@pytest.mark.parametrize("size", [0.0, 2.0 ** -100, 2.0 ** -126])
def test_queries_of_zero_and_small_keys(zp, d, b, new, size):
    """Logits of 0, or as good as: rows are the means of what they see, however small the keys' scales are."""
    rng = np.random.default_rng(new)
    Hq, Hkv, L = 4, 2, 400 + new
    tables, NB = A._tables(rng, [L], b)
    codes = _codes(rng, (1, NB, 2, Hkv, b, d))
    scales = 2.0 ** rng.integers(-8, -4, (1, NB, 2, Hkv))
    q = (torch.from_numpy(rng.standard_normal((new, Hq, d))).double() * size).to(torch.bfloat16).cuda()
    p = A._params(Hq, Hkv, d, b)
    c, dt = torch.from_numpy(codes).cuda(), torch.from_numpy(tables).cuda()
    for k_scale in (2.0 ** -20, 2.0 ** -24, 2.0 ** -60, 2.0 ** -126):
        scales[0, :, 0] = k_scale
        s = torch.from_numpy(scales.astype(np.float32)).cuda()
        for window, sinks in ((0, 0), (150, 20)):
            got = _attend(zp, c, s, q, [new], [L], dt, p, window, sinks)
            _check(c[0], s[0], dt[0], q, got, L, window, sinks, p, (size, k_scale, window), tiled=2 * new > 16)


@pytest.mark.gpu
def test_queries_and_keys_whose_factor_is_beyond_fp32(zp):
    """Queries of 2^110 where the keys are 0: logits are 0, not 0 times infinity."""
    rng = np.random.default_rng(3)
    d, b, new, L = 128, 16, 40, 300
    tables, NB = A._tables(rng, [L], b)
    codes = _codes(rng, (1, NB, 2, 1, b, d))
    codes[0, :, 0, :, :, :64] = 0
    scales = 2.0 ** rng.integers(-8, -4, (1, NB, 2, 1))
    scales[0, :, 0] = 2.0 ** 60
    q = torch.zeros((new, 4, d))
    q[:, :, :64] = torch.from_numpy(rng.standard_normal((new, 4, 64))) * 2.0 ** 110
    q = q.to(torch.bfloat16).cuda()
    p = A._params(4, 1, d, b)
    c, s, dt = torch.from_numpy(codes).cuda(), torch.from_numpy(scales.astype(np.float32)).cuda(), torch.from_numpy(tables).cuda()
    got = _attend(zp, c, s, q, [new], [L], dt, p)
    _check(c[0], s[0], dt[0], q, got, L, 0, 0, p, "large")


# ------------------------------------------------------------------ what weights are held to --

@pytest.mark.gpu
@pytest.mark.parametrize("d,b", [(128, 16), (64, 32)])
@pytest.mark.parametrize("less", [0, 6, 11, 15])
def test_a_peak_among_values_of_a_smaller_scale(zp, d, b, less):
    """The token with the largest weight stands in a block whose V scale is 2^-less of its neighbours', before 4000 tokens of weights
    e^-20 of it."""
    new, L = 20, 4096
    NB = L // b
    p = A._params(1, 1, d, b, scale=0.125)
    rng = np.random.default_rng(less)
    codes = np.zeros((1, NB, 2, 1, b, d), dtype=np.uint8)
    codes[0, :, 1] = _codes(rng, (NB, 1, b, d))
    codes[0, :, 0, 0, :, 0] = S.e4m3_encode(np.array(-20.0))
    codes[0, 1, 0, 0, 3, 0] = 0                        # logits: 8 * -20 / 8, and 0
    scales = np.ones((1, NB, 2, 1), dtype=np.float32)
    scales[0, 1, 1] = 2.0 ** -less
    q = torch.zeros((new, 1, d), dtype=torch.bfloat16, device="cuda")
    q[:, 0, 0] = 8.0
    c, s, dt = torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda(), _i32(np.arange(NB)[None])
    got = _attend(zp, c, s, q, [new], [L], dt, p)
    _check(c[0], s[0], dt[0], q, got, L, 0, 0, p, less)


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,Hkv,d,b", [(32, 8, 128, 16), (28, 4, 128, 32), (8, 8, 64, 16), (16, 2, 64, 32), (16, 1, 128, 16), (3, 1, 64, 16)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (90, 5)])
def test_chunks_to_the_weights_rounding(zp, Hq, Hkv, d, b, window, sinks):
    rng = np.random.default_rng(Hq)
    new, cached = [40, 129, 300, 17], [0, 260, 31, 1500]
    lens = [c + n for c, n in zip(cached, new)]
    tables, NB = A._tables(rng, lens, b)
    codes = torch.from_numpy(_codes(rng, (1, NB, 2, Hkv, b, d))).cuda()
    scales = torch.from_numpy((2.0 ** rng.integers(-12, -4, (1, NB, 2, Hkv))).astype(np.float32)).cuda()
    q = torch.from_numpy(rng.standard_normal((sum(new), Hq, d)) * 2).to(torch.bfloat16).cuda()
    p, dt = A._params(Hq, Hkv, d, b), torch.from_numpy(tables).cuda()
    got = _attend(zp, codes, scales, q, new, lens, dt, p, window, sinks)
    lo = 0
    for r, n in enumerate(new):
        _check(codes[0], scales[0], dt[r], q[lo:lo + n], got[lo:lo + n], lens[r], window, sinks, p, r)
        lo += n


@pytest.mark.gpu
@pytest.mark.parametrize("d,b", [(128, 16), (128, 32), (64, 16), (64, 32)])
def test_every_code_and_packed_blocks_to_the_weights_rounding(zp, d, b):
    """All codes that are numbers; and blocks that the library packed, with the scales that it writes."""
    rng = np.random.default_rng(d + b)
    Hq, Hkv, new, L = 4, 2, 200, 900
    tables, NB = A._tables(rng, [L], b)
    p, dt = A._params(Hq, Hkv, d, b), torch.from_numpy(tables).cuda()
    q = torch.from_numpy(rng.standard_normal((new, Hq, d)) / 4).to(torch.bfloat16).cuda()
    codes = torch.from_numpy((rng.integers(0, 0x7F, (1, NB, 2, Hkv, b, d)) + 0x80 * rng.integers(0, 2, (1, NB, 2, Hkv, b, d))).astype(np.uint8)).cuda()
    scales = torch.from_numpy((2.0 ** rng.integers(-8, -4, (1, NB, 2, Hkv))).astype(np.float32)).cuda()
    pool = (torch.randn((1, NB, 2, Hkv, b, d), device="cuda") * 2.0 ** torch.randint(-6, 3, (1, NB, 2, Hkv, 1, 1), device="cuda")).to(torch.bfloat16)
    pool[0, int(tables[0, 1])] = 0
    ids, ws = torch.arange(NB, dtype=torch.int32, device="cuda"), zp.new_workspace(256)
    packed, written = torch.zeros_like(codes), torch.zeros_like(scales)
    zp.zp_kv8_pack_blocks(pool, ids, packed, written, ids, p, ws)
    for c, s in ((codes, scales), (packed, written)):
        for window, sinks in ((0, 0), (150, 20)):
            got = _attend(zp, c, s, q, [new], [L], dt, p, window, sinks)
            _check(c[0], s[0], dt[0], q, got, L, window, sinks, p, window)


@pytest.mark.gpu
def test_captured_drafts_to_the_weights_rounding(zp):
    """16 rows a head, the most that the form for few rows takes, captured and replayed over caches that grow."""
    rng = np.random.default_rng(1)
    Hq, Hkv, d, b, B, new = 8, 2, 128, 16, 5, 4
    tables, NB = A._tables(rng, [700] * B, b)
    codes = torch.from_numpy(_codes(rng, (1, NB, 2, Hkv, b, d))).cuda()
    scales = torch.from_numpy((2.0 ** rng.integers(-8, -4, (1, NB, 2, Hkv))).astype(np.float32)).cuda()
    q = torch.from_numpy(rng.standard_normal((B * new, Hq, d)) * 2).to(torch.bfloat16).cuda()
    p, dt, out = A._params(Hq, Hkv, d, b), torch.from_numpy(tables).cuda(), torch.empty_like(q)
    lens, start = _i32([4] * B), _i32(np.arange(B + 1) * new)
    ws = zp.new_workspace(zp.zp_kv8_window_workspace_size(p, B * new, B, new, tables.shape[1], 0, 0))
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        zp.zp_kv8_window_attn(codes, scales, 0, q, start, dt, lens, out, p, ws, 0, 0, new)
    for L in ([4, 5, 20, 300, 699], [700, 17, 33, 64, 4]):
        lens.copy_(_i32(L))
        graph.replay()
        for r in range(B):
            rows = slice(r * new, (r + 1) * new)
            _check(codes[0], scales[0], dt[r], q[rows], out[rows], L[r], 0, 0, p, r, tiled=False)
    assert zp.zp_read_error(ws) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("seed", range(24))
def test_random_scales(zp, seed):
    """Requests whose V scales are 0 here and there, for whole tiles, and of different sizes from one 128 tokens to the next."""
    rng = np.random.default_rng(seed)
    Hkv, G, d, b = int(rng.integers(1, 3)), int(rng.integers(1, 9)), int(rng.choice([64, 128])), int(rng.choice([16, 32]))
    B, top = int(rng.integers(1, 5)), int(rng.choice([3, 60, 300]))
    new = [int(x) for x in rng.integers(1, top + 1, B)]
    lens = [n + int(x) for n, x in zip(new, rng.integers(0, rng.choice([100, 1500]), B))]
    window, sinks = int(rng.choice([0, rng.integers(1, 600)])), int(rng.choice([0, rng.integers(1, 200)]))
    tables, NB = A._tables(rng, lens, b)
    codes = torch.from_numpy(_codes(rng, (1, NB, 2, Hkv, b, d))).cuda()
    scales = 2.0 ** rng.integers(-12, -4, (1, NB, 2, Hkv))
    for r, L in enumerate(lens):
        far = rng.integers(-40, 40, -(-L // 128))
        for i in range(-(-L // b)):
            off = rng.integers(-14, 1, Hkv) + far[i * b // 128] - 6
            scales[0, tables[r, i], 1] = np.where((far[i * b // 128] % 3 == 0) | (rng.random(Hkv) < 0.2), 0.0, 2.0 ** off)
    scales = torch.from_numpy(scales.astype(np.float32)).cuda()
    q = torch.from_numpy(rng.standard_normal((sum(new), G * Hkv, d)) * rng.choice([0.0, 0.5, 3.0])).to(torch.bfloat16).cuda()
    p, dt = A._params(G * Hkv, Hkv, d, b), torch.from_numpy(tables).cuda()
    got = _attend(zp, codes, scales, q, new, lens, dt, p, window, sinks)
    lo = 0
    for r, n in enumerate(new):
        _check(codes[0], scales[0], dt[r], q[lo:lo + n], got[lo:lo + n], lens[r], window, sinks, p, r, tiled=G * max(new) > 16)
        lo += n
