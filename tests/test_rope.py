"""Rotary positions (zp_rope_init, zp_rope_apply): the table on the CPU, the kernel on the GPU."""
import math
import os

import numpy as np
import pytest
import torch

from oracle import serving_oracle as S

THETA = 1e4
SCALINGS = [("none", {}), ("linear", dict(factor=4.0)), ("base", dict(factor=8.0)),
            ("yarn", dict(factor=16.0, original_len=4096, low=1.0, high=32.0)),
            ("wavelength", dict(factor=8.0, original_len=8192, low=1.0, high=4.0))]


@pytest.fixture(scope="module")
def zp():
    from paged_kv_cache_obs_gb300 import build
    if not os.path.exists(build.LIB):
        build.build()
    from paged_kv_cache_obs_gb300 import zipage
    return zipage


def _rows(zp, t):
    return zp.zp_rows(t.data_ptr(), t.stride(0), t.stride(1))


def _init(zp, d, rd, inter, name, kw, theta=THETA):
    return zp.zp_rope_init(d, rd, theta, inter, getattr(zp, "ZP_ROPE_" + name.upper()), **kw)


@pytest.mark.parametrize("name,kw", SCALINGS)
@pytest.mark.parametrize("d,rd", [(128, 128), (128, 64), (64, 16), (80, 20), (512, 256)])
def test_table(zp, name, kw, d, rd):
    rope = _init(zp, d, rd, False, name, kw)
    f, size = S.rope_frequencies(rd, THETA, name, **kw)
    got = np.array([t / 2.0 ** 64 * 2 * math.pi for t in rope.turns[:rd // 2]])
    # a handful of fp64 roundings, and the table's own 2^-65 turns
    assert np.all(np.abs(got - f) <= 1e-14 * f + 2 * math.pi * 2.0 ** -64)
    assert abs(rope.mscale - size) <= 2.0 ** -24 * size
    assert all(t == 0 for t in rope.turns[rd // 2:])


def test_table_takes_a_given_factor(zp):
    assert zp.zp_rope_init(64, 64, THETA, mscale=0.5).mscale == 0.5


@pytest.mark.parametrize("kw", [dict(head_dim=63), dict(head_dim=0), dict(head_dim=514), dict(rotary_dim=0), dict(rotary_dim=130),
                                dict(rotary_dim=7), dict(theta=1.0), dict(theta=math.inf), dict(theta=math.nan),
                                dict(scaling=5), dict(scaling=-1), dict(scaling=1, factor=0.5), dict(scaling=1, factor=math.nan),
                                dict(scaling=3, factor=2.0, original_len=0), dict(scaling=4, factor=2.0, original_len=10, low=0.0),
                                dict(scaling=4, factor=2.0, original_len=10, low=4.0, high=4.0), dict(scaling=2, factor=2.0, rotary_dim=2),
                                dict(mscale=math.inf), dict(mscale=1e39), dict(head_dim=512, rotary_dim=258)])
def test_table_refuses(zp, kw):
    full = dict(head_dim=128, rotary_dim=128, theta=THETA)
    full.update(kw)
    with pytest.raises(zp.ZipageError) as e:
        zp.zp_rope_init(**full)
    assert e.value.status == zp.ZP_ERR_INVALID_ARG


def test_apply_refuses(zp):
    """Argument errors are found on the host, before any launch."""
    import ctypes
    rope = zp.zp_rope_init(64, 64, THETA)
    x = torch.zeros((2, 3, 64), dtype=torch.bfloat16)
    rows, null = _rows(zp, x), zp.zp_rows(None, 0, 0)
    other = zp.zp_rows(rows.data, rows.token_stride * 2, rows.head_stride)
    odd = zp.zp_rows(rows.data + 1, rows.token_stride, rows.head_stride)
    call = lambda r, q, qo, hq, k, ko, hk, pos, T: zp.lib.zp_rope_apply(r, q, qo, hq, k, ko, hk, pos, T, None)
    pos = ctypes.c_void_p(x.data_ptr())
    bad = zp.ZP_ERR_INVALID_ARG
    assert call(None, rows, rows, 3, None, None, 0, pos, 2) == bad
    assert call(rope, rows, rows, 3, None, None, 0, None, 2) == bad
    assert call(rope, rows, rows, 3, None, None, 0, pos, -1) == bad
    assert call(rope, rows, rows, -3, None, None, 0, pos, 2) == bad
    assert call(rope, rows, None, 3, None, None, 0, pos, 2) == bad
    assert call(rope, null, rows, 3, None, None, 0, pos, 2) == bad
    assert call(rope, rows, other, 3, None, None, 0, pos, 2) == bad    # in place with other strides
    assert call(rope, odd, rows, 3, None, None, 0, pos, 2) == bad
    assert call(zp.zp_rope(), rows, rows, 3, None, None, 0, pos, 2) == bad  # a handle that no init filled
    assert call(rope, rows, rows, 5000, None, None, 0, pos, 2) == zp.ZP_ERR_UNSUPPORTED
    assert call(rope, rows, rows, 3, None, None, 0, pos, 0) == zp.ZP_OK
    assert call(rope, None, None, 0, None, None, 0, pos, 2) == zp.ZP_OK
    strided = torch.zeros((2, 3, 128), dtype=torch.bfloat16)[:, :, ::2]
    with pytest.raises(ValueError, match="contiguous last dimension"):
        zp.zp_rope_apply(rope, strided, None, torch.zeros(2, dtype=torch.int32))


def _check(got, x, pos, freqs, size, inter):
    want = S.rope(x, pos, freqs, size, inter)
    # bf16 rounding: 2^-8 of the value.  fp32: the angle within 2^-22, cos and sin within 2^-22, two
    # products and a sum: 2^-20 of the pair.  Both sides hold f_i in fp64, rounded a few times, and
    # the oracle its angle: |position| * 2^-51 radians together.
    pair = np.abs(x).max() * size
    err = np.abs(got - want)
    far = np.abs(np.asarray(pos, dtype=np.float64))[:, None, None] * 2.0 ** -51
    assert (err <= 2.0 ** -8 * np.abs(want) + (2.0 ** -20 + far) * pair).all(), float(err.max())


def _f64(t):
    return t.detach().double().cpu().numpy()


POSITIONS = [0, 1, -1, 7, 2047, 131072, 1000003, 2 ** 31 - 1, -2 ** 31, 12345678]


@pytest.mark.gpu
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("d,rd", [(128, 128), (128, 64), (128, 32), (64, 64), (64, 16), (64, 8), (80, 80), (96, 48), (20, 6), (2, 2), (512, 256)])
def test_apply_matches_oracle(zp, d, rd, inter):
    g = torch.Generator().manual_seed(d * 1000 + rd)
    T, Hq, Hkv = len(POSITIONS), 5, 2
    qkv = torch.randn((T, Hq + 2 * Hkv, d), generator=g).to(torch.bfloat16)
    dev = qkv.cuda()
    pos = torch.tensor(POSITIONS, dtype=torch.int32).cuda()
    name, kw = SCALINGS[(d + rd) % len(SCALINGS)]
    if name == "base" and rd < 4:
        name, kw = SCALINGS[0]
    rope = _init(zp, d, rd, inter, name, kw)
    f, size = S.rope_frequencies(rd, THETA, name, **kw)
    qo = torch.full((T, Hq, d), 7.0, dtype=torch.bfloat16, device="cuda")
    ko = torch.full((T, Hkv, d), 7.0, dtype=torch.bfloat16, device="cuda")
    zp.zp_rope_apply(rope, dev[:, :Hq], dev[:, Hq:Hq + Hkv], pos, q_out=qo, k_out=ko)
    assert torch.equal(dev.cpu(), qkv)                              # inputs stay
    x, p = _f64(qkv), np.array(POSITIONS, dtype=np.int64)
    _check(_f64(qo), x[:, :Hq], p, f, size, inter)
    _check(_f64(ko), x[:, Hq:Hq + Hkv], p, f, size, inter)
    assert torch.equal(qo.cpu()[..., rd:], qkv[:, :Hq, rd:])          # the rest passes through
    # in place: the same bits, and the values (and what follows the keys) stay
    zp.zp_rope_apply(rope, dev[:, :Hq], dev[:, Hq:Hq + Hkv], pos)
    assert torch.equal(dev[:, :Hq], qo) and torch.equal(dev[:, Hq:Hq + Hkv], ko)
    assert torch.equal(dev[:, Hq + Hkv:].cpu(), qkv[:, Hq + Hkv:])


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 3, 255, 4097])
@pytest.mark.parametrize("off", [0, 1])
def test_apply_lengths_and_alignment(zp, T, off):
    # `off`: rows that start at an odd element, so that the narrow form runs; the same bits as the
    # wide form's on the same values
    g = torch.Generator(device="cuda").manual_seed(T)
    Hq, Hkv, d = 4, 2, 128
    buf = torch.randn(T * (Hq + Hkv) * d + 8, generator=g, device="cuda").to(torch.bfloat16)
    x = buf[off:off + T * (Hq + Hkv) * d].view(T, Hq + Hkv, d)
    pos = torch.randint(-5, 100000, (T,), generator=g, device="cuda", dtype=torch.int32)
    rope = zp.zp_rope_init(d, 64, THETA, interleaved=True)
    flat = torch.zeros_like(buf)
    y = flat[off:off + T * (Hq + Hkv) * d].view(T, Hq + Hkv, d)
    zp.zp_rope_apply(rope, x[:, :Hq], x[:, Hq:], pos, q_out=y[:, :Hq], k_out=y[:, Hq:])
    f, size = S.rope_frequencies(64, THETA)
    _check(_f64(y), _f64(x), pos.cpu().numpy(), f, size, True)
    assert flat[:off].abs().sum() == 0 and flat[off + T * (Hq + Hkv) * d:].abs().sum() == 0
    wide = x.clone()
    zp.zp_rope_apply(rope, wide[:, :Hq], wide[:, Hq:], pos)
    assert torch.equal(wide, y)


@pytest.mark.gpu
def test_apply_one_side_only_and_head_major_rows(zp):
    g = torch.Generator().manual_seed(3)
    T, H, d = 9, 3, 64
    x = torch.randn((H, T, d), generator=g).to(torch.bfloat16)          # heads outermost
    pos = torch.arange(T, dtype=torch.int32).cuda()
    rope = zp.zp_rope_init(d, d, THETA)
    f, size = S.rope_frequencies(d, THETA)
    want = _f64(x.transpose(0, 1))
    for side in ("q", "k"):
        dev = x.cuda().transpose(0, 1)
        zp.zp_rope_apply(rope, dev if side == "q" else None, dev if side == "k" else None, pos)
        _check(_f64(dev), want, np.arange(T), f, size, False)


@pytest.mark.gpu
def test_non_finite_values_stay_in_their_pair(zp):
    x = torch.ones((1, 1, 64), dtype=torch.bfloat16)
    x[0, 0, 3] = math.inf
    x[0, 0, 5] = math.nan
    dev = x.cuda()
    zp.zp_rope_apply(zp.zp_rope_init(64, 64, THETA), dev, None, torch.tensor([5], dtype=torch.int32).cuda())
    bad = ~torch.isfinite(dev.cpu()[0, 0])
    assert set(bad.nonzero().flatten().tolist()) <= {3, 35, 5, 37} and bool(bad[5]) and bool(bad[37])
