"""Attention of packed prompts over their own keys and values (zp_prompt_attn), against 64 bits."""
import math
import os

import numpy as np
import pytest
import torch

import test_cache_attention as A


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
    rows = zp.zp_rows(base, 128, 64)
    params = lambda **kw: zp.make_params({**p, **kw})

    def call(q=rows, k=rows, v=rows, start=base, T=2, B=2, max_len=2, window=0, sinks=0, out=rows, params=zp.make_params(p), w=base, nb=1 << 40):
        return zp.lib.zp_prompt_attn(q, k, v, start, T, B, max_len, window, sinks, out, params, w, nb, None)

    null, odd = zp.zp_rows(None, 0, 0), zp.zp_rows(base + 1, 128, 64)
    for kw in (dict(q=None), dict(k=None), dict(v=None), dict(out=None), dict(q=null), dict(k=null), dict(v=null), dict(out=null), dict(q=odd),
               dict(k=odd), dict(v=odd), dict(out=odd), dict(start=None), dict(T=-1), dict(B=-1), dict(max_len=0), dict(window=-1), dict(sinks=-1),
               dict(params=None), dict(w=None), dict(w=base + 64), dict(nb=255), dict(out=zp.zp_rows(base, 0, 64)), dict(out=zp.zp_rows(base, 128, 32)),
               dict(params=params(scale=0.0)), dict(params=params(scale=math.nan)), dict(params=params(scale=3.4e38)),
               dict(params=params(num_q_heads=3)), dict(params=params(num_kv_heads=0))):
        assert call(**kw) == zp.ZP_ERR_INVALID_ARG, kw
    for kw in (dict(params=params(head_dim=96)), dict(params=params(num_q_heads=34)), dict(B=65536), dict(max_len=(1 << 30) + 1)):
        assert call(**kw) == zp.ZP_ERR_UNSUPPORTED, kw
    assert call(T=0, q=null, k=null, v=null, out=null) == zp.ZP_OK and call(B=0, q=None, k=None, v=None, out=None, start=None) == zp.ZP_OK
    # a pool's sizes play no part
    assert call(T=0, params=params(block_size=7, num_layers=0)) == zp.ZP_OK


def test_workspace_sizes(zp):
    p = A._params(32, 8, 128, 16)
    size = zp.zp_prompt_workspace_size
    assert size(p, 8192, 4, 2048) == 256 and size(p, 64, 1, 64) == 256
    few = A._params(8, 2, 128, 16)                            # 32 items of 64 queries, which two CTAs share
    assert size(few, 1000, 1, 1000) == 256 + 2 * 1000 * 8 * 132 * 4 and size(few, 1000, 1, 2 ** 30) == size(few, 1000, 1, 1000)
    for T in (1, 17, 300, 5000):
        for B in (1, 3, 50):
            for window in (0, 100, 10 ** 6):
                n = size(p, T, B, T, window, 4)
                assert n >= 256 and n % 256 == 0 and n <= size(p, T, 1, T)
    for bad in ((-1, 1, 5), (4, -1, 5), (4, 1, 0), (4, 1, 2 ** 30 + 1)):
        assert size(p, *bad) == 0
    assert size(p, 4, 1, 4, -1) == 0 and size(p, 4, 1, 4, 0, -1) == 0 and size(A._params(400, 2, 128, 16), 4, 1, 4) == 0


def test_binding_refuses(zp):
    p = A._params(4, 2, 64, 16)
    q, k = torch.zeros((5, 4, 64), dtype=torch.bfloat16), torch.zeros((5, 2, 64), dtype=torch.bfloat16)
    ws, start = torch.zeros(256, dtype=torch.uint8), torch.zeros(3, dtype=torch.int32)
    good = dict(q=q, k=k, v=k, token_start=start, out=q.clone(), params=p, workspace=ws, max_len=5)
    for kw in (dict(k=k[:4]), dict(v=q), dict(out=q[:, :2]), dict(q=q.float()), dict(token_start=start[:0]), dict(token_start=start.long()),
               dict(token_start=start[None]), dict(k=torch.zeros((5, 2, 128), dtype=torch.bfloat16)[..., ::2]), dict(max_len=1 << 40)):
        with pytest.raises(ValueError, match="expected"):
            zp.zp_prompt_attn(**{**good, **kw})
    with pytest.raises(ValueError, match="current CUDA device"):
        zp.zp_prompt_attn(**good)


# ------------------------------------------------------------------ GPU -----------------------

def _rows(g, T, H, d, form, gain=1.0):
    """[T, H, d] rows on the device in memory of that form."""
    x = (torch.randn((T, H, d), generator=g) * gain).to(torch.bfloat16).cuda()
    if form == "fused":
        y = torch.full((T, 3 * H, d), math.nan, dtype=torch.bfloat16, device="cuda")[:, H:2 * H]
    elif form == "odd":
        y = torch.zeros(T * H * d + 1, dtype=torch.bfloat16, device="cuda")[1:].view(T, H, d)
    elif form == "head-major":
        y = torch.zeros((H, T, d), dtype=torch.bfloat16, device="cuda").transpose(0, 1)
    elif form == "padded":          # rows of d + 4 values: 8-byte steps
        y = torch.zeros((T, H, d + 4), dtype=torch.bfloat16, device="cuda")[..., :d]
    else:
        return x
    return y.copy_(x)


def _exact(q, k, v, window, sinks, scale):
    """One prompt in 64 bits: q [n, Hq, d], k, v [n, Hkv, d] -> outputs and weighted magnitudes [n, Hq, d]."""
    n, Hq, d = q.shape
    G = Hq // k.shape[1]
    p, t = torch.arange(n, device=q.device)[:, None], torch.arange(n, device=q.device)
    see = (t <= p) & ((t > p - window) | (t < sinks) | (window == 0))
    out, mass = (torch.empty((n, Hq, d), dtype=torch.float64, device=q.device) for _ in range(2))
    for h in range(Hq):
        key, value = k[:, h // G].double(), v[:, h // G].double()
        x = (scale * (q[:, h].double() @ key.T)).masked_fill(~see, -math.inf)
        w = torch.softmax(x, -1)
        out[:, h], mass[:, h] = w @ value, w @ value.abs()
    return out, mass


def _check(got, want, mass):
    # the output's bf16 rounding 2^-8, P's 2^-8, logits and sums in fp32 2^-14 (as in test_cache_attention)
    err = (got.double() - want).abs()
    tol = 2.0 ** -8 * want.abs() + (2.0 ** -8 + 2.0 ** -14) * mass + 1e-30
    assert bool((err <= tol).all()), float((err / tol).max())


def _case(zp, Hq, Hkv, d, lens, window=0, sinks=0, form="rows", qform=None, before=0, behind=0, seed=0, max_len=None, ws_bytes=None, check=True):
    """Packed prompts, with rows before the first and behind the last that hold NaN."""
    g = torch.Generator().manual_seed(seed)
    T = before + sum(lens) + behind
    q, k, v = _rows(g, T, Hq, d, qform or form, 2.0), _rows(g, T, Hkv, d, form), _rows(g, T, Hkv, d, form)
    for x in (q, k, v):
        x[:before] = math.nan
        x[T - behind:] = math.inf
    out = torch.full((T, Hq, d), 7.0, dtype=torch.bfloat16, device="cuda")
    if form == "odd":
        out = torch.full((T * Hq * d + 1,), 7.0, dtype=torch.bfloat16, device="cuda")[1:].view(T, Hq, d)
    start = before + np.concatenate([[0], np.cumsum(lens)])
    p = A._params(Hq, Hkv, d, 16)
    most = max_len or max(max(lens), 1)
    ws = zp.new_workspace(zp.zp_prompt_workspace_size(p, T, len(lens), most, window, sinks) if ws_bytes is None else ws_bytes)
    args = (q, k, v, _i32(start), out, p, ws, most)
    for _ in range(2):
        zp.zp_prompt_attn(*args, window=window, sinks=sinks)
    assert zp.zp_read_error(ws) == 0
    assert bool((out[:before] == 7).all()) and bool((out[T - behind:] == 7).all())
    for r, n in enumerate(lens):
        rows = slice(int(start[r]), int(start[r]) + n)
        if n and check:
            _check(out[rows], *_exact(q[rows], k[rows], v[rows], window, sinks, p["scale"]))
    return args


def _values_case(zp, lens, d, window, sinks, value, bad_at):
    """Three prompts; the second's keys and values are all `value`, and so are the values of the others at bad_at (row, head, dim)."""
    Hq, Hkv = 4, 2
    g = torch.Generator().manual_seed(4)
    T, (n0, n1, n2) = sum(lens), lens
    q, k, v = _rows(g, T, Hq, d, "rows", 2.0), _rows(g, T, Hkv, d, "rows"), _rows(g, T, Hkv, d, "rows")
    k[n0:n0 + n1] = value
    v[n0:n0 + n1] = value
    for row, head, dim in bad_at:
        v[row, head, dim] = value
    out, p = torch.full((T, Hq, d), 7.0, dtype=torch.bfloat16, device="cuda"), A._params(Hq, Hkv, d, 16)
    ws = zp.new_workspace(zp.zp_prompt_workspace_size(p, T, 3, max(lens), window, sinks))
    zp.zp_prompt_attn(q, k, v, _i32([0, n0, n0 + n1, T]), out, p, ws, max(lens), window=window, sinks=sinks)
    assert zp.zp_read_error(ws) == 0
    for lo, hi in ((0, n0), (n0 + n1, T)):
        n = hi - lo
        i, t = torch.arange(n, device="cuda")[:, None], torch.arange(n, device="cuda")
        see = (t <= i) & ((t > i - window) | (t < sinks) | (window == 0))
        for h in range(Hq):
            x = v[lo:hi, h // 2].double()
            bad = ~torch.isfinite(x)
            hit = see.double() @ bad.double() > 0                        # [n, d]
            got = out[lo:hi, h].double()
            assert bool((torch.isfinite(got) == ~hit).all())
            if math.isinf(value):
                assert bool((got[hit] == value).all())
            x = torch.where(bad, torch.zeros_like(x), x)
            lw = (p["scale"] * (q[lo:hi, h].double() @ k[lo:hi, h // 2].double().T)).masked_fill(~see, -math.inf)
            w = torch.softmax(lw, -1)
            _check(got[~hit], (w @ x)[~hit], (w @ x.abs())[~hit])


SHAPES = [(32, 8, 128), (28, 4, 128), (8, 8, 64), (16, 2, 64), (8, 4, 128), (3, 1, 128), (16, 1, 128), (10, 1, 64), (11, 1, 64)]


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,Hkv,d", SHAPES)
def test_lengths(zp, Hq, Hkv, d):
    _case(zp, Hq, Hkv, d, [1, 0, 2, 17, 127, 128, 129, 300, 0, 33], seed=Hq, before=3, behind=5)


@pytest.mark.gpu
@pytest.mark.parametrize("n", [1, 2, 31, 64, 255, 256, 257, 1000])
def test_one_prompt(zp, n):
    _case(zp, 4, 1, 64, [n], seed=n)
    _case(zp, 7, 1, 128, [n], seed=n, behind=1)


@pytest.mark.gpu
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (16, 17), (100, 0), (128, 128), (129, 300), (70, 33), (5000, 3), (31, 1000), (0, 5), (299, 4), (300, 4)])
def test_windows(zp, window, sinks):
    _case(zp, 4, 2, 128, [300, 1, 150, 40, 129], window, sinks, seed=window, before=2, behind=9)
    _case(zp, 2, 2, 64, [257, 300, 3], window, sinks, seed=sinks)


@pytest.mark.gpu
@pytest.mark.parametrize("form", ["fused", "odd", "head-major", "padded"])
@pytest.mark.parametrize("window,sinks", [(0, 0), (40, 5)])
def test_strides(zp, form, window, sinks):
    _case(zp, 4, 2, 128, [130, 5, 70], window, sinks, form=form, seed=1, before=1, behind=3)
    _case(zp, 3, 1, 64, [200, 33], window, sinks, form=form, seed=2)
    _case(zp, 2, 1, 64, [300, 33], window, sinks, form=form, seed=5, behind=2)
    # queries of one form with keys and values of another
    _case(zp, 4, 2, 64, [130, 5, 70], window, sinks, form=form, qform="rows", seed=3)
    _case(zp, 4, 2, 64, [130, 5, 70], window, sinks, form="rows", qform=form, seed=4)


@pytest.mark.gpu
def test_broadcast_keys_and_values(zp):
    """One key and value for all tokens and heads (strides of 0): every row is the value."""
    q = torch.randn((150, 4, 64), device="cuda").to(torch.bfloat16)
    k, v = (torch.randn((1, 1, 64), device="cuda").to(torch.bfloat16).expand(150, 2, 64) for _ in range(2))
    out, p, ws = torch.zeros_like(q), A._params(4, 2, 64, 16), zp.new_workspace(1 << 20)
    zp.zp_prompt_attn(q, k, v, _i32([0, 100, 150]), out, p, ws, 100)
    assert zp.zp_read_error(ws) == 0
    _check(out, v[:, :1].double().expand(150, 4, 64), v[:, :1].double().abs().expand(150, 4, 64))


@pytest.mark.gpu
@pytest.mark.parametrize("max_len", [700, 2 ** 30])
def test_a_loose_bound(zp, max_len):
    _case(zp, 8, 2, 128, [129, 40, 300], seed=5, max_len=max_len)
    _case(zp, 8, 2, 128, [129, 40, 300], 50, 3, seed=5, max_len=max_len, behind=4)


@pytest.mark.gpu
@pytest.mark.parametrize("lens,window", [([1500], 0), ([1500], 1000), ([2300], 0), ([900, 40], 0)])
def test_few_long_prompts_are_split(zp, lens, window):
    args = _case(zp, 2, 1, 128, lens, window, 4, seed=len(lens))
    own = args[6].numel()
    assert own > 256
    for n in (256, own // 512 * 256, own + 256):                # a larger batch's workspace: split less
        buf = torch.zeros(n + 512, dtype=torch.uint8, device="cuda")
        buf[n:] = 0xA5
        out = torch.full_like(args[4], 7.0)
        zp.zp_prompt_attn(*args[:4], out, args[5], buf[:n], args[7], window=window, sinks=4)
        torch.cuda.synchronize()
        assert bool((buf[n:] == 0xA5).all()) and int(buf[:4].view(torch.int32)) == 0
        at = 0
        for m in lens:
            _check(out[at:at + m], *_exact(*(x[at:at + m] for x in args[:3]), window, 4, args[5]["scale"]))
            at += m
    with pytest.raises(zp.ZipageError):
        zp.zp_prompt_attn(*args[:6], torch.zeros(own - 1, dtype=torch.uint8, device="cuda"), args[7], window=window, sinks=4)


@pytest.mark.gpu
def test_split_prompts_of_one_query_tile(zp):
    """100 items are cut into 3 parts, and some CTAs take two in a row of which one softmax group has no part: the long prompts'
    last 100 queries, and a short prompt."""
    _case(zp, 1, 1, 64, [4964, 4964, 100, 128, 70], seed=1)


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,Hkv,d", SHAPES)
def test_short_prompts(zp, Hq, Hkv, d):
    """Up to 128 tokens: the form in small CTAs."""
    _case(zp, Hq, Hkv, d, [1, 0, 2, 15, 16, 17, 63, 64, 65, 100, 0, 127, 128, 5], seed=Hq, before=3, behind=5)
    _case(zp, Hq, Hkv, d, [128], seed=Hq + 1)


@pytest.mark.gpu
@pytest.mark.parametrize("form", ["rows", "fused", "odd", "head-major", "padded"])
@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (1, 1), (16, 17), (40, 5), (64, 64), (65, 3), (100, 200), (128, 2), (7, 70)])
def test_short_prompts_in_windows_and_strides(zp, form, window, sinks):
    _case(zp, 4, 2, 128, [100, 5, 70, 128, 1], window, sinks, form=form, seed=1, before=1, behind=3)
    _case(zp, 7, 1, 64, [33, 127, 64], window, sinks, form=form, seed=2)


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("window,sinks", [(0, 0), (30, 3)])
@pytest.mark.parametrize("value", [math.inf, -math.inf, math.nan])
def test_values_of_short_prompts_reach_only_the_rows_that_see_them(zp, d, window, sinks, value):
    _values_case(zp, [100, 20, 128], d, window, sinks, value, ((60, 1, 7), (120 + 2, 0, 9), (120 + 100, 1, 60), (120 + 127, 0, 1)))


@pytest.mark.gpu
@pytest.mark.parametrize("form", ["rows", "odd"])
@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (1, 1), (16, 17), (64, 64), (65, 3), (100, 200), (130, 5), (200, 1), (7, 70), (255, 2), (3, 190)])
def test_narrow_heads_of_up_to_256_tokens(zp, form, window, sinks):
    """64-wide heads take the form in small CTAs up to 256 tokens: several tiles, of which a window leaves some out."""
    _case(zp, 4, 2, 64, [200, 5, 129, 1, 256, 193], window, sinks, form=form, seed=window, before=1, behind=3)
    _case(zp, 7, 1, 64, [255, 64, 192], window, sinks, form=form, seed=sinks)


@pytest.mark.gpu
@pytest.mark.parametrize("window,sinks", [(0, 0), (70, 3)])
@pytest.mark.parametrize("value", [math.inf, -math.inf, math.nan])
def test_values_of_narrow_heads_reach_only_the_rows_that_see_them(zp, window, sinks, value):
    _values_case(zp, [200, 30, 256], 64, window, sinks, value, ((60, 1, 7), (150, 0, 33), (230 + 2, 0, 9), (230 + 140, 1, 60), (230 + 255, 0, 1)))


@pytest.mark.gpu
def test_short_rows_whose_logits_are_all_minus_infinity_are_nan(zp):
    q, k = (torch.ones((40, 2, 64), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    q[20:, 0] = -math.inf
    out, ws = torch.zeros_like(q), zp.new_workspace(256)
    zp.zp_prompt_attn(q, k, k, _i32([0, 20, 40]), out, A._params(2, 2, 64, 16), ws, 20)
    assert bool(torch.isnan(out[20:, 0]).all()) and bool((out[:20] == 1).all()) and bool((out[20:, 1] == 1).all())


@pytest.mark.gpu
def test_many_short_prompts(zp):
    rng = np.random.default_rng(3)
    _case(zp, 8, 2, 64, [int(x) for x in rng.integers(0, 40, 500)], seed=6)
    _case(zp, 32, 8, 128, [int(x) for x in rng.integers(1, 9, 60)], seed=7, window=3, sinks=1)


@pytest.mark.gpu
@pytest.mark.parametrize("window,sinks", [(0, 0), (30, 3)])
@pytest.mark.parametrize("value", [math.inf, -math.inf, math.nan])
def test_values_reach_only_the_rows_that_see_them(zp, window, sinks, value):
    """Bad keys and values of other prompts, of later tokens and of tokens outside the window have no effect; the
    rows that see a bad value get it in that dim."""
    _values_case(zp, [100, 90, 200], 64, window, sinks, value, ((60, 1, 7), (190 + 2, 0, 9), (190 + 150, 1, 60)))
    _values_case(zp, [100, 90, 300], 64, window, sinks, value, ((60, 1, 7), (190 + 2, 0, 9), (190 + 250, 1, 60)))
    _values_case(zp, [100, 90, 200], 128, window, sinks, value, ((60, 1, 7), (190 + 2, 0, 90), (190 + 150, 1, 60)))


@pytest.mark.gpu
@pytest.mark.parametrize("n,d", [(140, 64), (300, 64), (140, 128)])
def test_odd_values_of_rows_at_odd_addresses(zp, n, d):
    """The same where keys and values are loaded value by value: the prompt's end stands inside of a run."""
    g = torch.Generator().manual_seed(8)
    q, k, v = _rows(g, n, 2, d, "rows"), _rows(g, n, 1, d, "odd"), _rows(g, n, 1, d, "odd")
    v[n - 10, 0, 3] = math.inf
    out, p, ws = torch.zeros_like(q), A._params(2, 1, d, 16), zp.new_workspace(256)
    zp.zp_prompt_attn(q, k, v, _i32([0, n]), out, p, ws, n)
    assert zp.zp_read_error(ws) == 0
    assert bool(torch.isinf(out[n - 10:, :, 3]).all()) and int((~torch.isfinite(out)).sum()) == 20


@pytest.mark.gpu
def test_skips_bad_prompts_and_reports(zp):
    g = torch.Generator().manual_seed(9)
    T, Hq, Hkv, d = 300, 4, 2, 64
    q, k, v = _rows(g, T, Hq, d, "rows", 2.0), _rows(g, T, Hkv, d, "rows"), _rows(g, T, Hkv, d, "rows")
    p = A._params(Hq, Hkv, d, 16)
    # (token_start, bound, prompts that are written)
    for start, most, good in (([0, 100, 260, 300], 120, (0, 2)), ([0, 100, 301], 300, (0,)), ([-1, 40, 90], 300, (1,)), ([0, 50, 20], 300, (0,)),
                              ([0, 100, 2 ** 31 - 1], 2 ** 30, (0,))):
        out = torch.full((T, Hq, d), 7.0, dtype=torch.bfloat16, device="cuda")
        ws = zp.new_workspace(zp.zp_prompt_workspace_size(p, T, len(start) - 1, most))
        zp.zp_prompt_attn(q, k, v, _i32(start), out, p, ws, most)
        assert zp.zp_read_error(ws) == zp.ZP_ERR_BAD_TABLE
        written = torch.zeros(T, dtype=torch.bool)
        for r in good:
            rows = slice(start[r], start[r + 1])
            written[rows] = True
            _check(out[rows], *_exact(q[rows], k[rows], v[rows], 0, 0, p["scale"]))
        assert bool((out[~written.cuda()] == 7).all())


@pytest.mark.gpu
def test_offsets_past_32_bits(zp):
    """Values 5 G elements apart: rows of a projection that is far wider than its values."""
    wide = 1 << 23
    buf = torch.zeros((640, wide), dtype=torch.bfloat16, device="cuda")
    g = torch.Generator().manual_seed(10)
    q, k = _rows(g, 640, 2, 64, "rows", 2.0), _rows(g, 640, 1, 64, "rows")
    v = buf[:, wide - 64:].view(640, 1, 64)
    v.copy_(_rows(g, 640, 1, 64, "rows"))
    out, p, ws = torch.zeros_like(q), A._params(2, 1, 64, 16), zp.new_workspace(256)
    zp.zp_prompt_attn(q, k, v, _i32([0, 640]), out, p, ws, 640)
    assert zp.zp_read_error(ws) == 0
    _check(out, *_exact(q, k, v, 0, 0, p["scale"]))


@pytest.mark.gpu
def test_a_wait_that_runs_out_is_reported(zp):
    args = _case(zp, 8, 2, 128, [700, 40, 300], seed=11)
    q, k, v, start, out, p, ws, most = args
    zp.zp_test_prompt_stalled(q, k, v, start, torch.zeros_like(out), p, ws, most, 1000000)
    assert zp.zp_read_error(ws) == zp.ZP_ERR_TIMEOUT
    again = torch.zeros_like(out)
    zp.zp_prompt_attn(q, k, v, start, again, p, ws, most)
    assert zp.zp_read_error(ws) == zp.ZP_OK and torch.equal(again, out)
    for ns in (0, -1, 10 ** 9 + 1):
        with pytest.raises(zp.ZipageError):
            zp.zp_test_prompt_stalled(q, k, v, start, again, p, ws, most, ns)


@pytest.mark.gpu
def test_captured_and_on_two_streams(zp):
    """A captured call replayed on new inputs, beside a call on another stream with a workspace of its own."""
    args = _case(zp, 8, 2, 64, [200, 31], seed=12)
    q, k, v, start, out, p, ws, most = args
    want = out.clone()
    other = _case(zp, 4, 2, 128, [500, 3], 90, 2, seed=13)
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        zp.zp_prompt_attn(q, k, v, start, out, p, ws, most)
    keep = q.clone()
    for step in range(3):
        q.copy_(keep * (step + 1))
        graph.replay()
        with torch.cuda.stream(side):
            mine = torch.zeros_like(other[4])
            zp.zp_prompt_attn(*other[:4], mine, *other[5:], window=90, sinks=2)
        torch.cuda.synchronize()
        assert torch.equal(mine, other[4])
        for lo, hi in ((0, 200), (200, 231)):
            _check(out[lo:hi], *_exact(q[lo:hi], k[lo:hi], v[lo:hi], 0, 0, p["scale"]))
        if step == 0:
            assert torch.equal(out, want)
    assert zp.zp_read_error(ws) == 0


@pytest.mark.gpu
def test_random_calls(zp):
    rng = np.random.default_rng(20)
    for i in range(60):
        Hkv = int(rng.integers(1, 5))
        G = int(rng.integers(1, 17))
        d = int(rng.choice([64, 128]))
        lens = [int(x) for x in rng.integers(0, rng.choice([5, 60, 400]), rng.integers(1, 7))]
        window = int(rng.choice([0, rng.integers(1, 450)]))
        _case(zp, G * Hkv, Hkv, d, lens, window, int(rng.choice([0, rng.integers(1, 200)])), form=str(rng.choice(["rows", "fused", "odd", "head-major"])),
              before=int(rng.integers(0, 4)), behind=int(rng.integers(0, 140)), seed=i, max_len=max(max(lens), 1) + int(rng.integers(0, 300)))
