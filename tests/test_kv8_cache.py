"""The 8-bit pool: quantising new tokens (zp_kv8_append) and whole blocks to and from the bf16 pool
(zp_kv8_pack_blocks, zp_kv8_unpack_blocks).  Scales are powers of two, so codes and scales are
compared exactly."""
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


def _params(Hkv, d, b, layers=1, n_max=8):
    return dict(num_layers=layers, num_q_heads=Hkv, num_kv_heads=Hkv, head_dim=d, block_size=b, n_max=n_max, window=1,
                alpha=0.5, beta=0.5, decay=0.9, scale=1.0 / math.sqrt(d), protect_window=1, causal=1)


# ------------------------------------------------------------------ the definition (CPU) ------

def test_oracle_codes_agree_with_torch():
    x = torch.randn(20000, generator=torch.Generator().manual_seed(0)).double() * torch.exp2(torch.linspace(-14, 7, 20000).double())
    x = torch.cat((x.clamp(-448, 448), torch.tensor([0.0, -0.0, 448.0, -448.0, 2.0 ** -9, 2.0 ** -10, 3 * 2.0 ** -10, 432.0, 440.0])))
    want = x.float().to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(S.e4m3_encode(x.float().double().numpy()), want)
    back = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(S.e4m3_decode(np.arange(256)), back, equal_nan=True)


def test_oracle_scale_is_the_smallest_power_of_two():
    for amax, want in ((448.0, 1.0), (449.0, 2.0), (447.0, 1.0), (224.0, 0.5), (225.0, 1.0), (1e-40, 2.0 ** -126), (0.0, 0.0)):
        assert S.block_scale(np.array([amax, -amax / 3, np.nan, -np.inf])) == want


# ------------------------------------------------------------------ refusals (CPU) ------------

def test_append_refuses(zp):
    x = torch.zeros((2, 2, 64), dtype=torch.bfloat16)
    ws = torch.zeros(512, dtype=torch.uint8)
    base = (ws.data_ptr() + 255) // 256 * 256
    p = zp.make_params(_params(2, 64, 16))
    rows = _rows(zp, x)
    at = ctypes.c_void_p(x.data_ptr())
    pool = zp.zp_kv8_pool(base, base, 4)

    def call(pool=pool, layer=0, k=rows, v=rows, T=2, start=at, cached=at, B=1, tables=at, mb=4, params=p, ws=base, nb=256):
        return zp.lib.zp_kv8_append(pool, layer, k, v, T, start, cached, B, tables, mb, params, ws, nb, None)

    bad, uns = zp.ZP_ERR_INVALID_ARG, zp.ZP_ERR_UNSUPPORTED
    for kw in (dict(pool=None), dict(layer=-1), dict(layer=1), dict(k=None), dict(v=None), dict(T=-1), dict(start=None),
               dict(cached=None), dict(B=-1), dict(B=0), dict(tables=None), dict(mb=0), dict(params=None), dict(ws=None),
               dict(ws=base + 16), dict(nb=255), dict(k=zp.zp_rows(None, 0, 0)), dict(v=zp.zp_rows(x.data_ptr() + 1, 128, 64)),
               dict(pool=zp.zp_kv8_pool(None, base, 4)), dict(pool=zp.zp_kv8_pool(base, None, 4)),
               dict(pool=zp.zp_kv8_pool(base, base, 0)), dict(pool=zp.zp_kv8_pool(base + 8, base, 4)),
               dict(pool=zp.zp_kv8_pool(base, base + 2, 4)), dict(params=zp.make_params(_params(0, 64, 16)))):
        assert call(**kw) == bad, kw
    assert call(params=zp.make_params(_params(2, 96, 16))) == uns
    assert call(params=zp.make_params(_params(2, 64, 8))) == uns
    assert call(T=0, B=0, k=None, v=None) == zp.ZP_OK
    assert call(T=0) == zp.ZP_OK


@pytest.mark.parametrize("pack", [True, False])
def test_block_conversion_refuses(zp, pack):
    ws = torch.zeros(512, dtype=torch.uint8)
    base = (ws.data_ptr() + 255) // 256 * 256
    p = zp.make_params(_params(2, 64, 16, layers=3))

    def call(pool=zp.zp_kv_pool(base, 4), kv8=zp.zp_kv8_pool(base, base, 4), src=base, dst=base, n=1, lb=0, lc=0, params=p,
             ws=base, nb=256):
        if pack:
            return zp.lib.zp_kv8_pack_blocks(pool, src, None, kv8, dst, n, lb, lc, params, ws, nb, None)
        return zp.lib.zp_kv8_unpack_blocks(kv8, src, pool, dst, n, lb, lc, params, ws, nb, None)

    bad, uns = zp.ZP_ERR_INVALID_ARG, zp.ZP_ERR_UNSUPPORTED
    for kw in (dict(pool=None), dict(kv8=None), dict(src=None), dict(dst=None), dict(n=-1), dict(lb=1), dict(lb=-1, lc=1),
               dict(lb=2, lc=2), dict(lc=-1), dict(lb=4, lc=1), dict(params=None), dict(ws=None), dict(ws=base + 8), dict(nb=100),
               dict(pool=zp.zp_kv_pool(base + 2, 4)), dict(pool=zp.zp_kv_pool(base, 0))):
        assert call(**kw) == bad, kw
    assert call(params=zp.make_params(_params(2, 32, 16, layers=3))) == uns
    assert call(n=1 << 30, params=zp.make_params(_params(60000, 64, 16, layers=3))) == uns
    assert call(n=0, src=None, dst=None) == zp.ZP_OK


def test_binding_refuses_what_it_would_misread(zp):
    """Types, layouts and places of tensors that the library could not tell from good ones."""
    bf = torch.zeros((4, 2, 64), dtype=torch.bfloat16)
    i32, i64 = torch.zeros(4, dtype=torch.int32), torch.zeros(4, dtype=torch.int64)
    pool = torch.zeros((1, 4, 2, 2, 16, 64), dtype=torch.bfloat16)
    codes, scales = torch.zeros(pool.shape, dtype=torch.uint8), torch.zeros((1, 4, 2, 2))
    tables, ws = torch.zeros((4, 6), dtype=torch.int32), torch.zeros(1024, dtype=torch.uint8)
    p = _params(2, 64, 16)
    rope = zp.zp_rope_init(64, 64, 1e4)
    for call in (lambda: zp.zp_rope_apply(rope, bf.half(), None, i32), lambda: zp.zp_rope_apply(rope, bf, None, i64),
                 lambda: zp.zp_rope_apply(rope, bf, None, i32),    # not on a CUDA device
                 lambda: zp.zp_kv8_append(pool, scales, 0, bf, bf, i32, i32, tables, p, ws),
                 lambda: zp.zp_kv8_append(codes, scales.half(), 0, bf, bf, i32, i32, tables, p, ws),
                 lambda: zp.zp_kv8_append(codes, scales, 0, bf, bf, i32, i32, tables[:, :3], p, ws),
                 lambda: zp.zp_kv8_append(codes.transpose(2, 3), scales, 0, bf, bf, i32, i32, tables, p, ws),
                 lambda: zp.zp_kv8_decode_attn(codes, scales, 0, bf, tables, i64, bf, p, ws),
                 lambda: zp.zp_kv8_decode_attn(codes, scales, 0, bf, tables, i32, bf.float(), p, ws),
                 lambda: zp.zp_paged_window_attn(codes, 0, bf, i32, tables, i32, bf, p, ws, 4, 1, 1),
                 lambda: zp.zp_paged_window_attn(pool, 0, bf, i32, tables.t(), i32, bf, p, ws, 4, 1, 1),
                 lambda: zp.zp_kv8_pack_blocks(pool, i64, codes, scales, i32, p, ws),
                 lambda: zp.zp_kv8_unpack_blocks(codes, scales, i32, pool.float(), i32, p, ws)):
        with pytest.raises(ValueError):
            call()
    # sizes that do not go together
    short, five = torch.zeros(3, dtype=torch.int32), torch.zeros(5, dtype=torch.int32)
    p8 = _params(2, 64, 16, layers=2)
    for call in (lambda: zp.zp_rope_apply(rope, bf, None, five), lambda: zp.zp_rope_apply(rope, None, bf[..., :32], i32),
                 lambda: zp.zp_rope_apply(rope, bf, None, i32, q_out=bf[:, :1]),
                 lambda: zp.zp_kv8_append(codes, scales, 0, bf, bf, i32, i32, tables, p, ws),       # B + 1 starts
                 lambda: zp.zp_kv8_append(codes, scales, 0, bf, bf[:3], five, i32, tables, p, ws),
                 lambda: zp.zp_kv8_append(codes, scales, 0, bf[:, :1], bf, five, i32, tables, p, ws),
                 lambda: zp.zp_kv8_append(codes, scales, 0, bf, bf, five, i32, tables[:3], p, ws),
                 lambda: zp.zp_kv8_append(codes, scales, 0, bf, bf, five, i32, tables, p8, ws),
                 lambda: zp.zp_kv8_append(codes, scales[:, :3].contiguous(), 0, bf, bf, five, i32, tables, p, ws),
                 lambda: zp.zp_kv8_append(codes, scales, 0, bf, bf, five, i32, tables, p, ws[::2]),
                 lambda: zp.zp_kv8_decode_attn(codes, scales, 0, bf, tables, short, bf, p, ws),
                 lambda: zp.zp_kv8_decode_attn(codes, scales, 0, bf, tables, i32, bf[:3], p, ws),
                 lambda: zp.zp_paged_window_attn(pool, 0, bf, i32, tables, i32, bf, p, ws, 4, 1, 1),
                 lambda: zp.zp_paged_window_attn(pool, 0, bf, five, tables, i32, bf, p8, ws, 4, 1, 1),
                 lambda: zp.zp_kv8_pack_blocks(pool, i32, codes, scales, short, p, ws),
                 lambda: zp.zp_kv8_pack_blocks(pool, i32, codes, scales, i32, p, ws, fill=short),
                 lambda: zp.zp_kv8_unpack_blocks(codes, scales, i32, pool[:, :, :1].contiguous(), i32, p, ws)):
        with pytest.raises(ValueError, match="expected"):
            call()
    # no tensor, or numbers that the library would cut
    for call, error in ((lambda: zp.zp_kv8_append(codes, scales, 0, bf, None, five, i32, tables, p, ws), ValueError),
                        (lambda: zp.zp_kv8_append(codes, scales, 1 << 32, bf, bf, five, i32, tables, p, ws), ValueError),
                        (lambda: zp.zp_kv8_append(codes, scales, None, bf, bf, five, i32, tables, p, ws), TypeError),
                        (lambda: zp.zp_kv8_append(codes.to_sparse(), scales, 0, bf, bf, five, i32, tables, p, ws), ValueError),
                        (lambda: zp.zp_kv8_append(codes.to("meta"), scales, 0, bf, bf, five, i32, tables, p, ws), ValueError),
                        (lambda: zp.zp_kv8_append(codes, scales, 0, bf, bf, five, i32, tables[0], p, ws), ValueError)):
        with pytest.raises(error):
            call()
    # and what is right but for its place
    with pytest.raises(ValueError, match="current CUDA device"):
        zp.zp_kv8_append(codes, scales, 0, bf, bf, five, i32, tables, p, ws)


# ------------------------------------------------------------------ append (GPU) --------------

class _Cache:
    """A pool on both sides, with every byte set, for B requests of up to max_blocks blocks."""

    def __init__(self, zp, B, Hkv, d, b, max_blocks, layers=2, seed=0):
        rng = np.random.default_rng(seed)
        NB = B * max_blocks + 3
        self.codes = rng.integers(0, 256, (layers, NB, 2, Hkv, b, d)).astype(np.uint8)
        self.scales = (2.0 ** rng.integers(-9, 0, (layers, NB, 2, Hkv))).astype(np.float64)
        self.tables = rng.permutation(NB)[:B * max_blocks].reshape(B, max_blocks).astype(np.int32)
        self.d_codes = torch.from_numpy(self.codes).cuda()
        self.d_scales = torch.from_numpy(self.scales).float().cuda()
        self.d_tables = torch.from_numpy(self.tables).cuda()
        self.p = _params(Hkv, d, b, layers)
        self.b, self.zp = b, zp
        self.ws = zp.new_workspace(256)

    def append(self, layer, k, v, start, cached):
        """k, v: device bf16 [T, H, d]."""
        self.zp.zp_kv8_append(self.d_codes, self.d_scales, layer, k, v, torch.tensor(start, dtype=torch.int32).cuda(),
                              torch.tensor(cached, dtype=torch.int32).cuda(), self.d_tables, self.p, self.ws)
        S.append(self.codes, self.scales, layer, k.double().cpu().numpy(), v.double().cpu().numpy(), start, cached,
                 self.tables, self.b)

    def check(self, err=0):
        assert self.zp.zp_read_error(self.ws) == err
        assert np.array_equal(self.d_scales.double().cpu().numpy(), self.scales)
        # NaN codes: the sign is not part of the definition
        got, want = self.d_codes.cpu().numpy(), self.codes
        same = (got == want) | (((got & 0x7F) == 0x7F) & ((want & 0x7F) == 0x7F))
        assert same.all(), int((~same).sum())


def _starts(new):
    return [0] + np.cumsum(new).tolist()


@pytest.mark.gpu
@pytest.mark.parametrize("Hkv,d,b", [(8, 128, 16), (4, 128, 32), (2, 64, 16), (3, 64, 32), (1, 128, 16)])
@pytest.mark.parametrize("off", [0, 1])
def test_append_ragged_steps(zp, Hkv, d, b, off):
    # prompts of odd lengths, then single tokens and chunks with idle requests, magnitudes that
    # rise and fall; `off`: rows that start at an odd element
    rng = np.random.default_rng(Hkv * d + b)
    g = torch.Generator(device="cuda").manual_seed(1)
    B, mb = 5, 6
    c = _Cache(zp, B, Hkv, d, b, mb, seed=d)
    lens = [0] * B
    for step, new in enumerate(([1, b, 2 * b + 3, b - 1, 0], [1, 1, 1, 1, 1], [0, 0, 0, 0, 0], [0, 5, 0, 1, 2 * b], [b + 1, 1, 1, 1, 1])):
        T = sum(new)
        buf = torch.randn(T * 2 * Hkv * d + 8, generator=g, device="cuda")
        buf = (buf * 2.0 ** float(rng.integers(-6, 7))).to(torch.bfloat16)
        kv = buf[off:off + T * 2 * Hkv * d].view(T, 2 * Hkv, d)
        c.append(1, kv[:, :Hkv], kv[:, Hkv:], _starts(new), lens)
        lens = [a + n for a, n in zip(lens, new)]
        c.check()


@pytest.mark.gpu
def test_append_many_requests_and_idle_ones(zp):
    # more requests than one round of the search covers (32 probes), many without tokens
    rng = np.random.default_rng(3)
    B = 1500
    new = rng.integers(0, 4, B) * (rng.random(B) < 0.5)
    cached = rng.integers(0, 28, B)
    c = _Cache(zp, B, 1, 64, 16, 2, layers=1, seed=5)
    T = int(new.sum())
    g = torch.Generator(device="cuda").manual_seed(2)
    kv = torch.randn((T, 2, 64), generator=g, device="cuda").to(torch.bfloat16)
    c.append(0, kv[:, :1], kv[:, 1:], _starts(new.tolist()), cached.tolist())
    c.check()


@pytest.mark.gpu
def test_append_special_values(zp):
    # zeros, subnormals, the largest values, infinities and NaN, values at rounding ties
    d, b = 64, 16
    c = _Cache(zp, 1, 1, d, b, 12, layers=1, seed=7)
    rows = [torch.zeros(d), torch.full((d,), 1e-40), torch.full((d,), 3.3e38), torch.linspace(-448, 448, d),
            torch.full((d,), -math.inf), torch.full((d,), math.nan), torch.tensor([math.nan, math.inf, 1.0, -2.0] * (d // 4)),
            2.0 ** torch.linspace(-30, 8, d), torch.full((d,), 17.0 / 16.0), torch.full((d,), -0.0)]
    cached = 0
    for n, row in enumerate(rows):  # each in a block of its own, then after it a block's worth of ordinary ones
        k = torch.zeros((b, 1, d))
        k[0, 0] = row
        k[b - 1, 0] = 0.25 * row
        k = k.to(torch.bfloat16).cuda()
        c.append(0, k, -k, [0, b], [cached])
        cached += b
        c.check()


@pytest.mark.gpu
def test_append_raises_scales_and_keeps_what_is_there(zp):
    # a block filled token by token with ever larger values: every code is rounded again only when
    # it leaves E4M3's normal range, and the result equals one append of the whole block then
    d, b = 128, 16
    one, whole = (_Cache(zp, 1, 2, d, b, 2, layers=1, seed=9) for _ in range(2))
    g = torch.Generator(device="cuda").manual_seed(4)
    x = torch.randn((b, 2, d), generator=g, device="cuda").sign() * (1 + torch.rand((b, 2, d), generator=g, device="cuda"))
    x = (x * 2.0 ** (torch.arange(b, device="cuda") / 4.0)[:, None, None]).to(torch.bfloat16)
    for t in range(b):
        one.append(0, x[t:t + 1], x[t:t + 1], [0, 1], [t])
        one.check()
    whole.append(0, x, x, [0, b], [0])
    whole.check()
    assert torch.equal(one.d_codes, whole.d_codes) and torch.equal(one.d_scales, whole.d_scales)


@pytest.mark.gpu
def test_append_skips_bad_requests_and_reports(zp):
    d, b, mb, B = 64, 16, 2, 4
    g = torch.Generator(device="cuda").manual_seed(6)
    for what in ("full", "negative", "block", "last"):
        c = _Cache(zp, B, 1, d, b, mb, layers=1, seed=11)
        new, cached = [3, 3, 3, 3], [4, 5, 6, 7]
        start = _starts(new)
        before = c.codes.copy(), c.scales.copy()
        x = torch.randn((12, 1, d), generator=g, device="cuda").to(torch.bfloat16)
        d_start = torch.tensor(start, dtype=torch.int32)
        if what == "full":
            cached[1] = mb * b - 2      # would pass max_blocks
        if what == "negative":
            cached[1] = -3
        bad_table = c.tables.copy()
        if what == "block":
            bad_table[1, 0] = c.codes.shape[1]
        if what == "last":
            bad_table[1, 0] = -1
        zp.zp_kv8_append(c.d_codes, c.d_scales, 0, x, x, d_start.cuda(), torch.tensor(cached, dtype=torch.int32).cuda(),
                         torch.from_numpy(bad_table).cuda(), c.p, c.ws)
        # the others are written
        keep = [0, 2, 3]
        xs = x.double().cpu().numpy()
        for r in keep:
            S.append(c.codes, c.scales, 0, xs[start[r]:start[r + 1]], xs[start[r]:start[r + 1]], [0, 3], [cached[r]],
                     [c.tables[r]], b)
        c.check(zp.ZP_ERR_BAD_TABLE)
        assert np.array_equal(c.codes[0, c.tables[1]], before[0][0, c.tables[1]])
        c.check()                       # the word was cleared by reading it


@pytest.mark.gpu
@pytest.mark.parametrize("start", [[0, 5, 3, 6], [1, 2, 4, 6], [0, 2, 4, 7], [-1, 2, 4, 6]])
def test_append_reports_bad_token_start(zp, start):
    # what is written is not defined then; nothing outside the requests' blocks is touched
    d, b, mb, B = 64, 16, 2, 3
    c = _Cache(zp, B, 1, d, b, mb, layers=2, seed=13)
    x = torch.ones((6, 1, d), dtype=torch.bfloat16, device="cuda")
    others = np.setdiff1d(np.arange(c.codes.shape[1]), c.tables.ravel())
    zp.zp_kv8_append(c.d_codes, c.d_scales, 0, x, x, torch.tensor(start, dtype=torch.int32).cuda(),
                     torch.tensor([0, 0, 0], dtype=torch.int32).cuda(), c.d_tables, c.p, c.ws)
    assert zp.zp_read_error(c.ws) == zp.ZP_ERR_BAD_TABLE
    got = c.d_codes.cpu().numpy()
    assert np.array_equal(got[1], c.codes[1]) and np.array_equal(got[0, others], c.codes[0, others])


@pytest.mark.gpu
def test_append_leaves_padded_rows_out(zp):
    # rows behind the last request's, as a step of fixed size has them; they hold NaN
    for new in ([1, 1, 0, 0], [20, 0, 3, 0]):
        c = _Cache(zp, 4, 2, 64, 16, 3, layers=1, seed=14)
        n = sum(new)
        x = torch.full((n + 40, 2, 64), math.nan, dtype=torch.bfloat16, device="cuda")
        x[:n] = torch.randn((n, 2, 64), device="cuda").to(torch.bfloat16)
        start, cached = _starts(new), [5, 16, 0, 7]
        zp.zp_kv8_append(c.d_codes, c.d_scales, 0, x, x, torch.tensor(start, dtype=torch.int32).cuda(),
                         torch.tensor(cached, dtype=torch.int32).cuda(), c.d_tables, c.p, c.ws)
        xs = x[:n].double().cpu().numpy()
        S.append(c.codes, c.scales, 0, xs, xs, start, cached, c.tables, 16)
        c.check()


# ------------------------------------------------------------------ whole blocks (GPU) --------

@pytest.mark.gpu
@pytest.mark.parametrize("Hkv,d,b", [(8, 128, 16), (4, 128, 32), (2, 64, 16), (3, 64, 32)])
def test_pack_and_unpack_blocks(zp, Hkv, d, b):
    layers, NB, n = 3, 11, 7
    g = torch.Generator().manual_seed(Hkv + d + b)
    pool = (torch.randn((layers, NB, 2, Hkv, b, d), generator=g) * 2.0 ** torch.randint(-5, 6, (layers, NB, 2, Hkv, 1, 1), generator=g)).to(torch.bfloat16)
    pool[0, 2, 0, 0, 1, 3] = math.inf
    pool[1, 3, 1, 0, 2, 5] = math.nan
    pool[2, 4] = 0
    rng = np.random.default_rng(1)
    src, dst = rng.permutation(NB)[:n].astype(np.int32), rng.permutation(NB)[:n].astype(np.int32)
    fill = rng.integers(0, b + 1, n).astype(np.int32)
    fill[0], fill[1] = 0, b
    p = _params(Hkv, d, b, layers)
    for use_fill, span in ((False, None), (True, None), (True, (1, 2)), (False, (2, 1))):
        codes = rng.integers(0, 256, pool.shape).astype(np.uint8)
        scales = rng.random((layers, NB, 2, Hkv)).astype(np.float32)
        dc, ds, ws = torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda(), zp.new_workspace(256)
        zp.zp_kv8_pack_blocks(pool.cuda(), torch.from_numpy(src).cuda(), dc, ds, torch.from_numpy(dst).cuda(), p, ws,
                              fill=torch.from_numpy(fill).cuda() if use_fill else None, layers=span)
        x = pool.double().numpy()
        for layer in range(*(0, layers) if span is None else (span[0], span[0] + span[1])):
            for i in range(n):
                rows = fill[i] if use_fill else b
                for kv in range(2):
                    for h in range(Hkv):
                        tile = x[layer, src[i], kv, h, :rows]
                        s = S.block_scale(tile)
                        codes[layer, dst[i], kv, h, :rows] = S.quantise(tile, s)
                        scales[layer, dst[i], kv, h] = s
        got = dc.cpu().numpy()
        assert (((got & 0x7F) == 0x7F) & ((codes & 0x7F) == 0x7F) | (got == codes)).all()
        assert np.array_equal(ds.cpu().numpy(), scales)
        assert zp.zp_read_error(ws) == 0
    # back, with scales that are not powers of two (rounded) and ones that are (exact)
    scales = (rng.random((layers, NB, 2, Hkv)) + 0.01).astype(np.float32)
    scales[:, ::2] = 2.0 ** rng.integers(-130, 100, scales[:, ::2].shape)
    codes = rng.integers(0, 256, pool.shape).astype(np.uint8)
    out = torch.full(pool.shape, 7.0, dtype=torch.bfloat16, device="cuda")
    ws = zp.new_workspace(256)
    zp.zp_kv8_unpack_blocks(torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda(), torch.from_numpy(src).cuda(),
                            out, torch.from_numpy(dst).cuda(), p, ws, layers=(1, 2))
    want = torch.full(pool.shape, 7.0, dtype=torch.bfloat16)
    # code * scale is exact in fp64; one rounding to fp32 in between needs no room: products of 4 and
    # 24 bits that are halfway between two bf16 after rounding to 24 bits would have to be seen
    val = torch.from_numpy(S.e4m3_decode(codes) * scales.astype(np.float64)[..., None, None])
    exact = val.float().to(torch.bfloat16)
    want[1:, dst] = exact[1:][:, src]
    assert torch.equal(out.cpu().nan_to_num(9.0), want.nan_to_num(9.0)) and zp.zp_read_error(ws) == 0


@pytest.mark.gpu
def test_unpack_to_a_pool_off_a_32_byte_boundary(zp):
    # (and the same bits on one: 32-byte stores)
    p = _params(2, 64, 16, 2)
    rng = np.random.default_rng(2)
    shape = (2, 4, 2, 2, 16, 64)
    codes = torch.from_numpy(rng.integers(0, 255, shape).astype(np.uint8)).cuda()
    scales = torch.full((2, 4, 2, 2), 0.25, device="cuda")
    ids = torch.arange(4, dtype=torch.int32, device="cuda")
    n = codes.numel()
    buf = torch.full((n + 64,), 7.0, dtype=torch.bfloat16, device="cuda")
    outs = []
    for off in (16, 8):
        out = buf[off:off + n].view(shape)
        zp.zp_kv8_unpack_blocks(codes, scales, ids, out, ids, p, zp.new_workspace(256))
        assert bool((buf[:off] == 7).all()) and bool((buf[off + n:] == 7).all())
        outs.append(out.clone())
        buf.fill_(7.0)
    want = torch.from_numpy(S.e4m3_decode(codes.cpu().numpy()) * 0.25).to(torch.bfloat16)
    assert torch.equal(outs[0].nan_to_num(9.0), outs[1].nan_to_num(9.0)) and torch.equal(outs[0].cpu().nan_to_num(9.0), want.nan_to_num(9.0))


@pytest.mark.gpu
def test_pack_then_unpack_is_the_rounded_pool(zp):
    # a power-of-two scale: reading back gives code * scale exactly, so a second round trip changes
    # nothing
    p = _params(2, 128, 16, 1)
    g = torch.Generator(device="cuda").manual_seed(0)
    pool = torch.randn((1, 5, 2, 2, 16, 128), generator=g, device="cuda").to(torch.bfloat16)
    ids = torch.arange(5, dtype=torch.int32, device="cuda")
    ws = zp.new_workspace(256)
    first = None
    src = pool
    for _ in range(2):
        codes = torch.zeros(pool.shape, dtype=torch.float8_e4m3fn, device="cuda")
        scales = torch.zeros((1, 5, 2, 2), device="cuda")
        zp.zp_kv8_pack_blocks(src, ids, codes, scales, ids, p, ws)
        back = torch.zeros_like(pool)
        zp.zp_kv8_unpack_blocks(codes, scales, ids, back, ids, p, ws)
        # half a step of 4 bits where the code is normal, half of 2^-9 of the scale below
        x, y = pool.double(), back.double()
        tol = torch.maximum(x.abs() * 2.0 ** -4, scales.double()[..., None, None] * 2.0 ** -10)
        if first is None:
            assert ((x - y).abs() <= tol).all()
            first = back
        assert torch.equal(first, back)
        src = back
    assert zp.zp_read_error(ws) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("pack", [True, False])
def test_block_conversion_skips_bad_blocks(zp, pack):
    p = _params(2, 64, 16, 2)
    g = torch.Generator(device="cuda").manual_seed(0)
    pool = torch.randn((2, 6, 2, 2, 16, 64), generator=g, device="cuda").to(torch.bfloat16)
    codes = torch.full(pool.shape, 3, dtype=torch.uint8, device="cuda")
    scales = torch.full((2, 6, 2, 2), 0.5, device="cuda")
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")
    for src, dst, fill in ((i32(0, 6, 2), i32(1, 2, 3), None), (i32(0, -1, 2), i32(1, 2, 3), None),
                           (i32(0, 1, 2), i32(1, 6, 3), None), (i32(0, 1, 2), i32(1, -7, 3), None),
                           (i32(0, 1, 2), i32(1, 2, 3), i32(16, 17, 16)), (i32(0, 1, 2), i32(1, 2, 3), i32(16, -1, 16))):
        if fill is not None and not pack:
            continue
        ws = zp.new_workspace(256)
        c, s, out = codes.clone(), scales.clone(), pool.clone()
        if pack:
            zp.zp_kv8_pack_blocks(pool, src, c, s, dst, p, ws, fill=fill)
            assert not torch.equal(c[:, 1], codes[:, 1]) and not torch.equal(c[:, 3], codes[:, 3])
            assert torch.equal(c[:, [0, 2, 4, 5]], codes[:, [0, 2, 4, 5]])
        else:
            zp.zp_kv8_unpack_blocks(c, s, src, out, dst, p, ws)
            assert not torch.equal(out[:, 1], pool[:, 1]) and not torch.equal(out[:, 3], pool[:, 3])
            assert torch.equal(out[:, [0, 2, 4, 5]], pool[:, [0, 2, 4, 5]])
        assert zp.zp_read_error(ws) == zp.ZP_ERR_BAD_TABLE
