"""Calls at the edges of the attention operators around the cache: workspaces of other sizes, values
that are not finite or very large, strides, and waits that run out."""
import math
import os

import numpy as np
import pytest
import torch

import test_cache_attention as A
from oracle import serving_oracle as S


@pytest.fixture(scope="module")
def zp():
    from paged_kv_cache_obs_gb300 import build
    if not os.path.exists(build.LIB):
        build.build()
    from paged_kv_cache_obs_gb300 import zipage
    return zipage


def _i32(x):
    return torch.as_tensor(np.ascontiguousarray(x), dtype=torch.int32).cuda()


# ------------------------------------------------------------------ workspaces ----------------

def test_workspace_sizes_are_multiples_of_256(zp):
    # the sizes that a call takes although it asks for more
    for Hq, Hkv, d, b in A.SHAPES:
        p = A._params(Hq, Hkv, d, b)
        for B in (1, 2, 3, 5, 17, 300):
            for mb in (1, 40, 777, 8192):
                sizes = [zp.zp_kv8_decode_workspace_size(p, B, mb)]
                sizes += [zp.zp_paged_window_workspace_size(p, B * n, B, n, mb, w, 4) for n in (1, 3, 40, 700) for w in (0, 1000)]
                assert all(x >= 256 and x % 256 == 0 for x in sizes)


@pytest.mark.gpu
def test_splits_follow_the_devices_sms(zp):
    # one kv head and one item of queries: as many parts of 4 tiles as there are SMs; one row of 8, 7/8 of
    # four CTAs an SM, in clusters of 8
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    p = A._params(2, 1, 64, 16)
    size = zp.zp_paged_window_workspace_size(p, 64, 1, 64, 1 << 16, 0, 0)
    assert (size - 256) // (64 * 2 * 68 * 4) == sms
    size = zp.zp_kv8_decode_workspace_size(p, 1, 1 << 16)
    assert (size - 256) // (8 * 68 * 4) == sms * 4 * 7 // 8 // 8


def _exact(q, k, v, visible, scale):
    """Rows q [.., d] over k, v [L, d] in 64 bits: the outputs and the weighted magnitudes.  visible [.., L]."""
    x = (scale * (q.double() @ k.double().T)).masked_fill(~visible, -math.inf)
    w = torch.softmax(x, -1)
    return w @ v.double(), w @ v.double().abs()


def _visible(pos, L, window, sinks):
    t = torch.arange(L, device="cuda")
    p = torch.as_tensor(pos, device="cuda")[..., None]
    return (t <= p) & ((t > p - window) | (t < sinks) | (window == 0))


def _tokens(pool, layer, table, kv, h, L):
    return pool[layer][table.long()][:, kv, h].reshape(-1, pool.shape[-1])[:L]


def _check_rows(got, want, mass, rel):
    err = (got.double() - want).abs()
    tol = 2.0 ** -8 * want.abs() + (rel + 2.0 ** -14) * mass + 1e-30        # as in test_cache_attention
    assert bool((err <= tol).all()), float((err / tol).max())


def _check_kv8(codes, scales, layer, q, tables, seq, out, p, ws=None, window=0, sinks=0, rel=2.0 ** -11):
    Hkv, G = p["num_kv_heads"], p["num_q_heads"] // p["num_kv_heads"]
    pool = codes.view(torch.float8_e4m3fn).double() * scales.double()[..., None, None]
    for r, L in enumerate(seq.tolist()):
        vis = _visible(L - 1, L, window, sinks)
        for h in range(Hkv):
            k, v = (_tokens(pool, layer, tables[r][:-(-L // p["block_size"])], i, h, L) for i in (0, 1))
            _check_rows(out[r, h * G:(h + 1) * G], *_exact(q[r, h * G:(h + 1) * G], k, v, vis, p["scale"]), rel)


def _check_window(pool, layer, q, start, tables, seq, out, p, ws, window, sinks, max_q, rel):
    Hkv, G = p["num_kv_heads"], p["num_q_heads"] // p["num_kv_heads"]
    start = start.tolist()
    for r, L in enumerate(seq.tolist()):
        n = start[r + 1] - start[r]
        vis = _visible(range(L - n, L), L, window, sinks)[:, None].expand(n, G, L)
        rows = slice(start[r], start[r + 1])
        for h in range(Hkv):
            k, v = (_tokens(pool, layer, tables[r][:-(-L // p["block_size"])], i, h, L) for i in (0, 1))
            heads = slice(h * G, (h + 1) * G)
            _check_rows(out[rows, heads], *_exact(q[rows, heads], k, v, vis, p["scale"]), rel)


def _with_workspaces(args, sizes, call, check):
    """The call of `args` (output at 6, workspace at 8) with workspaces of other sizes and a band behind each."""
    for n in sizes:
        buf = torch.zeros(n + 512, dtype=torch.uint8, device="cuda")
        buf[n:] = 0xA5
        a = list(args)
        a[8], a[6] = buf[:n], torch.full_like(args[6], 7.0)
        for _ in range(2):
            call(*a)
        torch.cuda.synchronize()
        assert bool((buf[n:] == 0xA5).all()) and int(buf[:4].view(torch.int32)) == 0
        check(*a)


@pytest.mark.gpu
@pytest.mark.parametrize("lens", [[40000], [9000, 5], [3000, 2000, 70, 1]])
def test_decode_with_the_workspace_of_a_larger_batch(zp, lens):
    # 256 bytes: what a batch that is not split asks for, whose last requests these may be
    args = A._kv8_case(zp, 8, 2, 128, 16, lens, seed=len(lens), hidden_nan=False)
    p, mb = args[7], args[4].shape[1]
    own = zp.zp_kv8_decode_workspace_size(p, len(lens), mb)
    assert zp.zp_kv8_decode_workspace_size(p, 500, mb) == 256 and own > 256
    _with_workspaces(args, (256, own // 512 * 256, own, own + 256), zp.zp_kv8_decode_attn, _check_kv8)
    for n in (255, 300, own - 1):                               # no workspace's size
        with pytest.raises(zp.ZipageError):
            zp.zp_kv8_decode_attn(*args[:8], torch.zeros(n, dtype=torch.uint8, device="cuda"))


@pytest.mark.gpu
@pytest.mark.parametrize("new,window", [(2, 0), (2, 3000), (70, 0), (300, 0)])
def test_window_with_the_workspace_of_a_larger_batch(zp, new, window):
    rel = A.SPLIT if new <= 4 else A.TILED
    args = A._window_case(zp, 4, 1, 64, 16, [9000], [new], window, 4, seed=new, rel=rel)
    p, mb = args[7], args[4].shape[1]
    own = zp.zp_paged_window_workspace_size(p, new, 1, new, mb, window, 4)
    assert own > 256 and args[8].numel() == own
    _with_workspaces(args, (256, own // 512 * 256, own, own + 256), zp.zp_paged_window_attn,
                     lambda *a: _check_window(*a, rel=rel))
    with pytest.raises(zp.ZipageError):
        zp.zp_paged_window_attn(*args[:8], torch.zeros(own - 1, dtype=torch.uint8, device="cuda"), *args[9:])


# ------------------------------------------------------------------ special values ------------

def _same(got, want, mass, rel, where):
    """Finite where the exact value is, within the tolerance of test_cache_attention; else the same infinity
    or NaN."""
    nan, fin = np.isnan(want), np.isfinite(want)
    assert np.array_equal(nan, np.isnan(got)), (where, got[nan != np.isnan(got)][:4], want[nan != np.isnan(got)][:4])
    assert np.array_equal(want[~nan & ~fin], got[~nan & ~fin]), where
    err = np.abs(got[fin] - want[fin])
    assert (err <= A._tolerance(want[fin], mass[fin], rel)).all(), (where, float(err.max()))


def _window_rows(zp, x, cached, new, q, window, sinks, rel, b=16, max_q=None, ordered=False):
    """Requests over a bf16 pool whose keys and values are x [B][2][Hkv][L][d] (float64): every row
    against 64 bits over the tokens that it sees."""
    B, Hkv, d = len(x), x[0].shape[1], x[0].shape[-1]
    T, Hq, _ = q.shape
    G = Hq // Hkv
    lens = [y.shape[2] for y in x]
    rng = np.random.default_rng(0)
    tables, NB = A._tables(rng, lens, b)
    pool = torch.zeros((1, NB, 2, Hkv, b, d), dtype=torch.bfloat16)
    for r in range(B):
        for t in range(lens[r]):
            pool[0, tables[r, t // b], :, :, t % b] = torch.from_numpy(x[r][:, :, t]).to(torch.bfloat16)
    kv = [torch.from_numpy(y).to(torch.bfloat16).double().numpy() for y in x]
    qb = torch.from_numpy(q).to(torch.bfloat16)
    out = torch.full(qb.shape, 7.0, dtype=torch.bfloat16, device="cuda")
    p = A._params(Hq, Hkv, d, b)
    start = np.concatenate([[0], np.cumsum(new)])
    mq = max_q or max(new)
    ws = zp.new_workspace(zp.zp_paged_window_workspace_size(p, T, B, mq, tables.shape[1], window, sinks))
    zp.zp_paged_window_attn(pool.cuda(), 0, qb.cuda(), _i32(start), _i32(tables), _i32(lens), out, p, ws, window, sinks, mq)
    assert zp.zp_read_error(ws) == 0
    got, qd = out.double().cpu().numpy(), qb.double().numpy()
    for r in range(B):
        for i in range(new[r]):
            vis = S.window_visible(cached[r] + i, lens[r], window, sinks)
            for h in range(Hq):
                with np.errstate(all="ignore"):
                    want, mass = S.attention_row(qd[start[r] + i, h], kv[r][0, h // G], kv[r][1, h // G], p["scale"], vis)
                want = np.where(np.isfinite(want) & (np.abs(want) >= 3.3961775292304958e38), np.sign(want) * np.inf, want)  # past bf16
                _same(got[start[r] + i, h], want, mass, rel, (r, i, h))
    return got


FORMS = [(1, A.SPLIT), (3, A.SPLIT), (70, A.TILED)]


@pytest.mark.gpu
@pytest.mark.parametrize("new,rel", FORMS)
@pytest.mark.parametrize("window,sinks", [(0, 0), (100, 20)])
def test_infinite_values_of_tokens_that_are_seen(zp, new, rel, window, sinks):
    # an infinity that a row sees makes its output infinite, two of different signs NaN; beside the
    # row's largest weight, early, late, and in tiles that only some rows see
    rng = np.random.default_rng(new)
    L, d = 300 + new, 64
    x = rng.standard_normal((2, 2, L, d))
    q = rng.standard_normal((new, 4, d)) * 2
    for t, dim, value in ((3, 0, math.inf), (17, 1, -math.inf), (299, 2, math.inf), (L - 1, 3, math.inf), (L - 1, 4, -math.inf),
                          (L - 1, 5, math.nan), (10, 6, math.inf), (12, 6, -math.inf), (280, 7, math.inf), (L - 1, 7, -math.inf)):
        x[1, 0, t, dim] = value
    x[0, 1, L - 1] = 3 * q[-1, 2]        # the second kv head's last token takes nearly all of the weight
    x[1, 1, L - 1, :8] = math.inf
    _window_rows(zp, [x], [300], [new], q, window, sinks, rel)


@pytest.mark.gpu
@pytest.mark.parametrize("new,rel", FORMS)
def test_rows_whose_logits_are_all_minus_infinity_are_nan(zp, new, rel):
    # as the softmax of them is; the second request is an ordinary one
    rng = np.random.default_rng(1)
    L, d = 40 + new, 64
    x = [rng.standard_normal((2, 1, L, d)) for _ in range(2)]
    q = rng.standard_normal((2 * new, 4, d))
    q[:new, :2, 5], q[:new, 2:, 5] = 1.0, -1.0
    x[0][0, 0, :, 5] = -math.inf           # rows of heads 0 and 1: all -inf; of heads 2 and 3: all inf
    got = _window_rows(zp, x, [40, 40], [new, new], q, 0, 0, rel)
    assert np.isnan(got[:new]).all() and np.isfinite(got[new:]).all()


@pytest.mark.gpu
def test_8_bit_rows_whose_logits_are_all_minus_infinity_are_nan(zp):
    p = A._params(2, 1, 64, 16)
    codes = torch.full((1, 4, 2, 1, 16, 64), 0x38, dtype=torch.uint8, device="cuda")   # 1.0
    q = torch.zeros((3, 2, 64), dtype=torch.bfloat16, device="cuda")
    q[0] = -math.inf
    q[1, 0, :] = 1.0
    out = torch.full_like(q, 7.0)
    ws = zp.new_workspace(zp.zp_kv8_decode_workspace_size(p, 3, 4))
    zp.zp_kv8_decode_attn(codes, torch.ones((1, 4, 2, 1), device="cuda"), 0, q, _i32([[0, 1, 2, 3]] * 3), _i32([40, 50, 0]), out, p, ws)
    assert zp.zp_read_error(ws) == 0
    assert bool(torch.isnan(out[0]).all()) and bool((out[1] == 1).all()) and bool((out[2] == 0).all())


@pytest.mark.gpu
@pytest.mark.parametrize("new,rel", FORMS)
def test_values_near_the_types_largest(zp, new, rel):
    # Finite values of up to 2^122 with logits that rise from tile to tile by what the running maximum lets
    # pass before it is raised: weights are at most 1, and 300 tokens of them stay far below fp32's largest.
    rng = np.random.default_rng(2)
    L, d = 300 + new, 64
    x = rng.standard_normal((2, 1, L, d)) * 0.01
    x[1] = np.sign(x[1]) * 2.0 ** 122 * rng.uniform(0.5, 1.0, x[1].shape)
    q = np.zeros((new, 4, d))
    q[:, :, 0] = 8.0                                   # logit = x[0][.., 0] (scale 1/8)
    x[0, 0, :, 0] = 0.0
    x[0, 0, 150, 0], x[0, 0, 260, 0] = 5.25, 14.0      # 7.6 and 20.2 in log2
    _window_rows(zp, [x], [300], [new], q, 0, 0, rel)


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
def test_8_bit_values_near_the_types_largest(zp, d):
    rng = np.random.default_rng(3)
    p = A._params(1, 1, d, 16, scale=0.125)
    NB, L = 16, 256
    codes = S.e4m3_encode(rng.uniform(128, 256, (1, NB, 2, 1, 16, d)))           # values of 2^121 to 2^122
    codes[0, :, 0] = 0
    codes[0, 10, 0, 0, 3, 0] = S.e4m3_encode(np.array(5.0))                       # 7.2 in log2, in a warp's second tile or later
    scales = np.ones((1, NB, 2, 1), dtype=np.float32)
    scales[:, :, 1] = 2.0 ** 114
    q = torch.zeros((1, 1, d), dtype=torch.bfloat16, device="cuda")
    q[0, 0, 0] = 8.0
    # one long request among many: a warp takes a quarter of its tiles, one after another
    B = 700
    seq = np.zeros(B, dtype=np.int32)
    seq[0] = L
    qs = q.expand(B, 1, d).contiguous()
    out = torch.zeros_like(qs)
    ws = zp.new_workspace(zp.zp_kv8_decode_workspace_size(p, B, NB))
    tables = np.zeros((B, NB), dtype=np.int32)
    tables[0] = np.arange(NB)
    zp.zp_kv8_decode_attn(torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda(), 0, qs, _i32(tables), _i32(seq), out, p, ws)
    assert zp.zp_read_error(ws) == 0
    k, v = (S.e4m3_decode(codes[0, :, i, 0]).reshape(-1, d) * float(scales[0, 0, i, 0]) for i in (0, 1))
    want, mass = S.attention_row(qs[0, 0].double().cpu().numpy(), k, v, p["scale"], np.ones(L, dtype=bool))
    _same(out[0, 0].double().cpu().numpy(), want, mass, 2.0 ** -11, "row")


@pytest.mark.gpu
@pytest.mark.parametrize("ratio", [1.5, 3.0, 30.0, 60.0, 500.0, 2.0 ** 40])
@pytest.mark.parametrize("d", [64, 128])
def test_8_bit_values_behind_a_block_of_a_larger_scale(zp, d, ratio):
    # Blocks of weight 0 with a V scale `ratio` times the others' come first; then one token of each warp's
    # tiles takes most of the weight with a value of 0, and the result is the sum of 4000 equal weights of
    # e^-9 of it: an error of one weight is the result's.
    p = A._params(1, 1, d, 16, scale=0.125)
    first = 8 if d == 64 else 4                        # a tile, or two of them, for each of the four warps
    NB = 2 * first + 256
    L = NB * 16
    codes = np.zeros((1, NB, 2, 1, 16, d), dtype=np.uint8)
    enc = lambda v: S.e4m3_encode(np.array(float(v)))
    codes[0, :, 0, 0, :, 0] = enc(-9)
    codes[0, :, 1, 0] = enc(1.5)
    codes[0, :first, 0, 0, :, 0] = enc(-88)
    codes[0, first:2 * first, 0, 0, 0, 0] = 0
    codes[0, first:2 * first, 1, 0, 0] = 0
    scales = np.ones((1, NB, 2, 1), dtype=np.float32)
    scales[0, :, 1] = 2.0 ** -6
    scales[0, :first, 1] = 2.0 ** -6 * ratio
    B = 700                                            # not split: 4 warps take every fourth tile
    seq = np.zeros(B, dtype=np.int32)
    seq[0] = L
    qs = torch.zeros((B, 1, d), dtype=torch.bfloat16, device="cuda")
    qs[:, 0, 0] = 8.0
    out = torch.zeros_like(qs)
    tables = np.zeros((B, NB), dtype=np.int32)
    tables[0] = np.arange(NB)
    ws = zp.new_workspace(zp.zp_kv8_decode_workspace_size(p, B, NB))
    zp.zp_kv8_decode_attn(torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda(), 0, qs, _i32(tables), _i32(seq), out, p, ws)
    assert zp.zp_read_error(ws) == 0
    kv = S.e4m3_decode(codes[0]) * scales[0].astype(np.float64)[..., None, None]
    k, v = (kv[:, i, 0].reshape(-1, d) for i in (0, 1))
    want, mass = S.attention_row(qs[0, 0].double().cpu().numpy(), k, v, p["scale"], np.ones(L, dtype=bool))
    _same(out[0, 0].double().cpu().numpy(), want, mass, 2.0 ** -11, "row")



@pytest.mark.gpu
@pytest.mark.parametrize("gain", [2.0 ** 10, 2.0 ** 16, 2.0 ** 24])
def test_8_bit_queries_with_one_large_value(zp, gain):
    # a value of the query `gain` times the others, where the keys are 0: the logits are the others'
    rng = np.random.default_rng(5)
    p = A._params(4, 1, 128, 16)
    NB = 13
    codes = S.e4m3_encode(np.clip(rng.standard_normal((1, NB, 2, 1, 16, 128)) * 64, -448, 448))
    codes[0, :, 0, 0, :, 77] = 0
    scales = np.full((1, NB, 2, 1), 2.0 ** -6, dtype=np.float32)
    q = torch.from_numpy(rng.standard_normal((2, 4, 128)) * 2).to(torch.bfloat16)
    q[:, :, 77] = gain
    args = (torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda(), 0, q.cuda(), _i32([np.arange(NB)] * 2), _i32([200, 33]),
            torch.zeros(q.shape, dtype=torch.bfloat16, device="cuda"), p, zp.new_workspace(zp.zp_kv8_decode_workspace_size(p, 2, NB)))
    zp.zp_kv8_decode_attn(*args)
    assert zp.zp_read_error(args[8]) == 0
    _check_kv8(*args)


@pytest.mark.gpu
@pytest.mark.parametrize("d,heads,cached,new", [(64, 8, 100000, 5120), (128, 2, 20000, 300), (64, 1, 40000, 70)])
def test_odd_values_in_a_long_cache_cost_little_and_stay_where_they_are_seen(zp, d, heads, cached, new):
    # A value that only the last rows see is not finite: they get it in its dimension, every other result
    # keeps its bits, and the call stays far inside the time that its waits allow (whole items, and items
    # whose tiles are split).
    g = torch.Generator(device="cuda").manual_seed(d)
    L = cached + new
    nb = -(-L // 16)
    pool = torch.randn((1, nb, 2, heads, 16, d), generator=g, device="cuda").to(torch.bfloat16)
    tables = torch.randperm(nb, generator=g, device="cuda").to(torch.int32)[None]
    q = torch.randn((new, heads, d), generator=g, device="cuda").to(torch.bfloat16)
    p = A._params(heads, heads, d, 16)
    ws = zp.new_workspace(zp.zp_paged_window_workspace_size(p, new, 1, new, nb, 0, 0))

    def run():
        out = torch.full_like(q, 7.0)
        ev = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
        ev[0].record()
        zp.zp_paged_window_attn(pool, 0, q, _i32([0, new]), tables, _i32([L]), out, p, ws, 0, 0, new)
        ev[1].record()
        assert zp.zp_read_error(ws) == 0
        return out, ev[0].elapsed_time(ev[1])

    places = [(L - 1, 5, math.nan, 0), (L - 40, 9, math.inf, 0), (L - 3, 9, -math.inf, 0), (L - new + 1, 20, -math.inf, heads - 1),
              (L - new // 2, 33, math.inf, heads - 1)]
    for t, dim, _, h in places:
        pool[0, tables[0, t // 16], 1, h, t % 16, dim] = 0
    want, _ = run()
    for t, dim, value, h in places:
        pool[0, tables[0, t // 16], 1, h, t % 16, dim] = value
    got, ms = run()
    row = torch.arange(cached, L, device="cuda")
    for t, dim, value, h in places:
        seen = row >= t
        want[seen, h, dim] = want[seen, h, dim] + value
    assert torch.equal(torch.nan_to_num(got.float(), nan=1e38, posinf=2e38, neginf=-2e38),
                       torch.nan_to_num(want.float(), nan=1e38, posinf=2e38, neginf=-2e38))
    assert ms < 200


@pytest.mark.gpu
@pytest.mark.parametrize("window,sinks", [(0, 0), (40, 0), (100, 20), (130, 300)])
@pytest.mark.parametrize("d,Hq,Hkv,b", [(64, 4, 2, 16), (128, 7, 1, 32)])
def test_odd_keys_and_values_anywhere(zp, window, sinks, d, Hq, Hkv, b):
    # infinities and NaN in keys, in values and in both of a token: 0 times an infinity is NaN where an infinite
    # key gives a weight of 0
    rng = np.random.default_rng(d + window)
    cached, new = [150, 0], [70, 200]
    x = [rng.standard_normal((2, Hkv, c + n, d)) for c, n in zip(cached, new)]
    q = np.abs(rng.standard_normal((sum(new), Hq, d)))
    for r in range(2):
        L = x[r].shape[2]
        for t in rng.choice(L, 6, replace=False):
            x[r][1, rng.integers(Hkv), t, rng.integers(d, size=2)] = rng.choice([math.inf, -math.inf, math.nan])
        t, h = L - 30, Hkv - 1
        x[r][0, h, t, 3], x[r][1, h, t, 8] = -math.inf, math.inf          # weight 0: NaN in dim 8
        x[r][0, 0, L - 9, 4], x[r][1, 0, L - 9, 1] = math.nan, math.inf   # rows that see it: NaN
    _window_rows(zp, x, cached, new, q, window, sinks, A.TILED, b=b)


# ------------------------------------------------------------------ waits that run out --------

BAND = 4096


def _banded(t):
    """A copy of `t` with a band of 0xA5 behind it."""
    n = t.numel() * t.element_size()
    buf = torch.full((n + BAND,), 0xA5, dtype=torch.uint8, device="cuda")
    buf[:n] = t.contiguous().view(torch.uint8).flatten()
    return buf[:n].view(t.dtype).view(t.shape), buf[n:]


@pytest.mark.gpu
@pytest.mark.parametrize("name,form", [
    ("a cluster of splits", dict(kv8=(8, 2, 128, 16, [5, 300, 1100]))),
    ("parts of several clusters", dict(kv8=(8, 2, 128, 16, [9000, 1, 0, 4097]))),
    ("not split, two tiles at a time", dict(kv8=(4, 2, 64, 16, [40, 700, 3] * 110))),
    ("bf16, a ring of keys or values", dict(window=(32, 8, 128, 16, [0, 700, 1999], [1, 1, 1]))),
    ("bf16, 16 rows", dict(window=(8, 2, 128, 16, [0, 300, 3000], [4, 3, 4]))),
    ("one short item a CTA", dict(window=(4, 2, 64, 16, [0, 50], [40, 20]))),
    ("items of several tiles", dict(window=(4, 2, 128, 16, [900, 100], [300, 70]))),
    ("several items a CTA", dict(window=(4, 4, 64, 16, [0, 300] * 40, [40, 150] * 40))),
    ("items split over their tiles", dict(window=(4, 1, 128, 16, [9000], [70]))),
    ("queries without a tensor map", dict(window=(4, 2, 128, 16, [700] * 50, [60] * 50), off=1)),
])
def test_a_wait_that_runs_out_is_reported_and_the_next_call_is_exact(zp, name, form):
    if "kv8" in form:
        args = A._kv8_case(zp, *form["kv8"], seed=1, hidden_nan=False)
        call, stalled, tail = zp.zp_kv8_decode_attn, zp.zp_test_kv8_decode_stalled, ()
    else:
        Hq, Hkv, d, b, cached, new = form["window"]
        args = A._window_case(zp, Hq, Hkv, d, b, cached, new, 0, 0, seed=1, rel=A.TILED, off=form.get("off", 0))
        call, stalled, tail = zp.zp_paged_window_attn, zp.zp_test_paged_window_stalled, args[9:]
    want = args[6].clone()
    a = list(args[:9])
    bands = [None] * 9
    for i in (0, 6, 8):
        if i != 6 or not form.get("off"):
            a[i], bands[i] = _banded(a[i])
    if "kv8" in form:
        a[1], bands[1] = _banded(a[1])
    before = [x.clone() if isinstance(x, torch.Tensor) else None for x in a]
    for limit in (2_000_000, 1):
        stalled(*a, *tail, stall_limit_ns=limit)
        assert zp.zp_read_error(a[8]) == zp.ZP_ERR_TIMEOUT
        torch.cuda.synchronize()
        assert all(bool((x == 0xA5).all()) for x in bands if x is not None)
        for i in (0, 1, 2, 3, 4, 5):
            if isinstance(a[i], torch.Tensor):
                assert torch.equal(a[i].view(torch.uint8), before[i].view(torch.uint8)), i
        a[6].fill_(7.0)
        call(*a, *tail)
        assert zp.zp_read_error(a[8]) == 0
        assert torch.equal(a[6], want)
        assert all(bool((x == 0xA5).all()) for x in bands if x is not None)


def test_stall_limits_are_checked(zp):
    p = zp.make_params(A._params(2, 2, 64, 16))
    for ns in (0, -5, 2_000_000_000):
        assert zp.lib.zp_test_kv8_decode_stalled(None, 0, None, None, None, 1, 1, 0, 0, None, p, None, 0, ns, None) == zp.ZP_ERR_INVALID_ARG
        assert zp.lib.zp_test_paged_window_stalled(None, 0, None, None, 1, 1, None, None, 1, 1, 0, 0, None, p, None, 0, ns, None) == zp.ZP_ERR_INVALID_ARG

@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
def test_rows_behind_a_request_do_not_reach_it(zp, d):
    # q holds NaN and infinities in the rows of no request, and in those of the request behind
    for n in (1, 2, 50, 130):
        args = A._window_case(zp, 4, 2, d, 16, [100, 5], [n, n], 40, 3, seed=n, rel=A.TILED)
        T = args[2].shape[0]
        q = torch.empty((T + 150, 4, d), dtype=torch.bfloat16, device="cuda")
        q[0::3], q[1::3], q[2::3] = math.nan, math.inf, -math.inf
        q[:n] = args[2][:n]
        out = torch.full_like(q, 7.0)
        a = list(args)
        a[2], a[6] = q, out
        zp.zp_paged_window_attn(*a)
        assert zp.zp_read_error(args[8]) == 0
        assert torch.equal(out[:n], args[6][:n]) and bool((out[T:] == 7).all())
        assert not bool(torch.isfinite(out[n:T]).any())

# ------------------------------------------------------------------ strides -------------------

def _layouts(T, heads, d, g):
    """Rows [T, heads, d] in orders that a program has them in."""
    yield "fused", torch.zeros((T, heads + 5, d), dtype=torch.bfloat16, device="cuda")[:, 2:2 + heads]
    yield "head-major", torch.zeros((heads, T, d), dtype=torch.bfloat16, device="cuda").transpose(0, 1)
    yield "padded rows", torch.zeros((T, heads, d + 8), dtype=torch.bfloat16, device="cuda")[..., :d]
    yield "odd rows", torch.zeros((T, heads, d + 1), dtype=torch.bfloat16, device="cuda")[..., :d]
    yield "every other token", torch.zeros((2 * T, heads, d), dtype=torch.bfloat16, device="cuda")[::2]


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("form", ["kv8", "few", "many", "split"])
def test_strides_of_queries_and_outputs(zp, form, d):
    if form == "kv8":
        args = A._kv8_case(zp, 28, 4, d, 16, [40, 1, 500, 0, 17], seed=d, hidden_nan=False)
        call = zp.zp_kv8_decode_attn
    else:
        cached, new = dict(few=([30, 500, 0], [1, 2, 2]), many=([30, 500, 0], [90, 20, 41]), split=([3000], [70]))[form]
        args = A._window_case(zp, 28, 4, d, 16, cached, new, 100 if form != "split" else 0, 4, seed=d, rel=A.TILED)
        call = zp.zp_paged_window_attn
    qat = 3 if form == "kv8" else 2
    T, H, _ = args[qat].shape
    ins, outs = list(_layouts(T, H, d, None)), list(_layouts(T, H, d, None))
    for i, (name, q) in enumerate(ins):
        for oname, o in (outs[i], outs[(i + 1) % len(outs)], outs[(i + 3) % len(outs)]):
            whole = o._base
            whole.fill_(7.0)
            q.copy_(args[qat])
            a = list(args)
            a[qat], a[6] = q, o
            call(*a)
            assert zp.zp_read_error(args[8]) == 0
            assert torch.equal(o, args[6]), (name, oname)
            o.fill_(7.0)
            assert bool((whole == 7).all()), (name, oname)          # nothing between the rows


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("new", [2, 70])
def test_queries_may_be_broadcast(zp, new, d):
    args = A._window_case(zp, 4, 2, d, 16, [100], [new], 60, 3, seed=new, rel=A.TILED)
    one = torch.randn((1, 1, d), device="cuda").to(torch.bfloat16)
    outs = []
    for q in (one.expand(new, 4, d), one.expand(new, 4, d).contiguous()):
        a = list(args)
        a[2], a[6] = q, torch.zeros_like(args[6])
        zp.zp_paged_window_attn(*a)
        outs.append(a[6])
    assert zp.zp_read_error(args[8]) == 0 and torch.equal(*outs)


# ------------------------------------------------------------------ masks ---------------------

@pytest.mark.gpu
@pytest.mark.parametrize("cached,new,window", [(1000, 300, 700), (1500, 700, 1300), (3000, 200, 2100), (700, 64, 600), (4000, 130, 1000)])
@pytest.mark.parametrize("d,b", [(64, 16), (128, 32)])
def test_a_window_without_first_tokens(zp, cached, new, window, d, b):
    # positions of less than two windows, where the window's start lies before its middle, and further ones
    A._window_case(zp, 4, 2, d, b, [cached, 5], [new, 20], window, 0, seed=new, hidden_nan=True, rel=A.TILED)
