"""Rotary positions with several axes (zp_rope_axes_init, zp_rope_apply_axes)."""
import ctypes
import math
import os

import numpy as np
import pytest
import torch

from oracle import serving_oracle as S

THETA = 1e4
LAYOUTS = ("sections", "cycle", "restart")


@pytest.fixture(scope="module")
def zp():
    from paged_kv_cache_obs_gb300 import build
    if not os.path.exists(build.LIB):
        build.build()
    from paged_kv_cache_obs_gb300 import zipage
    return zipage


def _init(zp, d, rd, sections, layout, inter=False, **kw):
    return zp.zp_rope_axes_init(d, rd, THETA, sections, getattr(zp, "ZP_AXES_" + layout.upper()), inter, **kw)


def test_tables(zp):
    axes = _init(zp, 64, 32, [8, 4, 4], "sections")
    assert list(axes.axis[:16]) == [0] * 8 + [1] * 4 + [2] * 4 and axes.num_axes == 3
    plain = zp.zp_rope_init(64, 32, THETA)
    assert list(axes.rope.turns) == list(plain.turns)
    axes = _init(zp, 64, 32, [8, 4, 4], "cycle")
    assert list(axes.axis[:16]) == [0, 1, 2] * 4 + [0] * 4 and list(axes.rope.turns) == list(plain.turns)
    axes = _init(zp, 64, 32, [6, 10], "restart")
    assert list(axes.axis[:16]) == [0] * 6 + [1] * 10
    assert list(axes.rope.turns[:6]) == list(zp.zp_rope_init(64, 12, THETA).turns[:6])
    assert list(axes.rope.turns[6:16]) == list(zp.zp_rope_init(64, 20, THETA).turns[:10])
    assert list(_init(zp, 64, 32, [16], "cycle").axis[:16]) == [0] * 16
    # four axes, and the first may have as many pairs more as there are
    assert list(_init(zp, 64, 32, [13, 1, 1, 1], "cycle").axis[:16]) == [0, 1, 2, 3] + [0] * 12


def test_init_refuses(zp):
    for sections, layout in (([], "sections"), ([8, 7], "sections"), ([8, 9], "cycle"), ([16, 0], "sections"), ([17, -1], "restart"),
                             ([4, 8, 4], "cycle"), ([5, 5, 6], "cycle"), ([2 ** 31 - 1, 17], "sections")):
        with pytest.raises(zp.ZipageError) as e:
            _init(zp, 64, 32, sections, layout)
        assert e.value.status == zp.ZP_ERR_INVALID_ARG
    for kw in (dict(layout=3), dict(layout=-1), dict(theta=1.0), dict(rotary_dim=66), dict(scaling=zp.ZP_ROPE_BASE, factor=2.0, layout=2)):
        full = dict(head_dim=64, rotary_dim=32, theta=THETA, sections=[15, 1], layout=0)
        full.update(kw)
        with pytest.raises(zp.ZipageError):
            zp.zp_rope_axes_init(**full)
    with pytest.raises(ValueError, match="at most"):
        _init(zp, 64, 32, [4, 4, 4, 2, 2], "sections")


def test_apply_refuses(zp):
    axes = _init(zp, 64, 32, [8, 8], "sections")
    x = torch.zeros((2, 3, 64), dtype=torch.bfloat16)
    rows = zp.zp_rows(x.data_ptr(), 192, 64)
    pos = ctypes.c_void_p(x.data_ptr())
    call = lambda a, q=rows, p=pos, T=2, step=2: zp.lib.zp_rope_apply_axes(a, q, q, 3, None, None, 0, p, step, T, None)
    bad = zp.ZP_ERR_INVALID_ARG
    assert call(None) == bad and call(zp.zp_rope_axes()) == bad and call(axes, p=None) == bad and call(axes, T=-1) == bad
    assert call(axes, q=zp.zp_rows(None, 0, 0)) == bad
    broken = _init(zp, 64, 32, [8, 8], "sections")
    broken.axis[3] = 2
    assert call(broken) == bad
    broken = _init(zp, 64, 32, [8, 8], "sections")
    broken.rope.rotary_dim = 4096
    assert call(broken) == bad
    assert call(axes, T=0) == zp.ZP_OK
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)
    for p in (i32(2), i32(3, 2), i32(2, 2, 1), i32(2, 2).long(), i32(2, 4)[:, ::2], i32(2, 3)):
        with pytest.raises(ValueError, match="expected"):
            zp.zp_rope_apply_axes(axes, x, None, p)
    with pytest.raises(ValueError, match="current CUDA device"):
        zp.zp_rope_apply_axes(axes, x, None, i32(2, 2))


def _f64(t):
    return t.detach().double().cpu().numpy()


POSITIONS = np.array([[0, 1, -1, 7, 2047, 131072, 1000003, 2 ** 31 - 1, -2 ** 31, 12345678],
                      [0, 3, 5, -7, 99, 4096, 1000003, -2 ** 31, 2 ** 31 - 1, 1],
                      [0, 2, 500, 7, 2046, 17, 3, 6, 4, -12345678],
                      [9, 8, 7, 6, 5, 4, 3, 2, 1, 0]], dtype=np.int64)


def _check(got, want, x, pos, size):
    # as one axis: bf16's rounding 2^-8, angles, cos and sin within 2^-22 each and two products and a sum (2^-20 of the
    # pair), both sides' f_i in fp64 and the oracle's angle (|position| 2^-51 radians together)
    pair = np.abs(x).max() * size
    far = np.abs(pos).max(0).astype(np.float64)[:, None, None] * 2.0 ** -51
    err = np.abs(got - want)
    assert (err <= 2.0 ** -8 * np.abs(want) + (2.0 ** -20 + far) * pair).all(), float(err.max())


@pytest.mark.gpu
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("d,rd,sections", [(128, 128, [24, 20, 20]), (128, 64, [16, 8, 8]), (64, 64, [16, 16]), (80, 80, [20, 20]), (80, 20, [4, 3, 3]),
                                           (512, 256, [32, 32, 32, 32]), (64, 64, [32]), (6, 4, [1, 1])])
def test_matches_oracle(zp, d, rd, sections, layout, inter):
    g = torch.Generator().manual_seed(d * 1000 + rd)
    pos = POSITIONS[:len(sections)]
    T, Hq, Hkv = pos.shape[1], 5, 2
    scaling, kw = [("none", {}), ("yarn", dict(factor=16.0, original_len=4096, low=1.0, high=32.0)), ("linear", dict(factor=4.0))][len(sections) % 3]
    axes = _init(zp, d, rd, sections, layout, inter, scaling=getattr(zp, "ZP_ROPE_" + scaling.upper()), **kw)
    size = axes.rope.mscale
    qkv = torch.randn((T, Hq + 2 * Hkv, d), generator=g).to(torch.bfloat16)
    dev, dpos = qkv.cuda(), torch.as_tensor(pos, dtype=torch.int32).cuda()
    qo = torch.full((T, Hq, d), 7.0, dtype=torch.bfloat16, device="cuda")
    ko = torch.full((T, Hkv, d), 7.0, dtype=torch.bfloat16, device="cuda")
    zp.zp_rope_apply_axes(axes, dev[:, :Hq], dev[:, Hq:Hq + Hkv], dpos, q_out=qo, k_out=ko)
    assert torch.equal(dev.cpu(), qkv)
    x = _f64(qkv)
    want = S.rope_axes(x, pos, rd, THETA, sections, layout, inter, scaling, **kw)
    _check(_f64(qo), want[:, :Hq], x, pos, size)
    _check(_f64(ko), want[:, Hq:Hq + Hkv], x, pos, size)
    assert torch.equal(qo.cpu()[..., rd:], qkv[:, :Hq, rd:])
    zp.zp_rope_apply_axes(axes, dev[:, :Hq], dev[:, Hq:Hq + Hkv], dpos)        # in place: the same bits
    assert torch.equal(dev[:, :Hq], qo) and torch.equal(dev[:, Hq:Hq + Hkv], ko)
    assert torch.equal(dev[:, Hq + Hkv:].cpu(), qkv[:, Hq + Hkv:])


@pytest.mark.gpu
@pytest.mark.parametrize("layout", ("sections", "cycle"))
@pytest.mark.parametrize("T", [1, 5, 1023, 1024, 3001])
@pytest.mark.parametrize("off", [0, 1])
def test_equal_positions_turn_as_one_axis(zp, T, layout, off):
    """Text, whose axes agree: bit for bit zp_rope_apply, in the wide and the narrow form (`off`)."""
    g = torch.Generator(device="cuda").manual_seed(T)
    buf = torch.randn(T * 6 * 128 + 8, generator=g, device="cuda").to(torch.bfloat16)
    x = buf[off:off + T * 6 * 128].view(T, 6, 128)
    pos = torch.randint(-5, 100000, (T,), generator=g, device="cuda", dtype=torch.int32)
    a, b = x.clone(), x.clone()
    if off:
        a, b = (torch.zeros_like(buf)[1:1 + x.numel()].view_as(x).copy_(x) for _ in range(2))
    zp.zp_rope_apply(zp.zp_rope_init(128, 128, THETA), a[:, :4], a[:, 4:], pos)
    axes = _init(zp, 128, 128, [24, 20, 20], layout)
    zp.zp_rope_apply_axes(axes, b[:, :4], b[:, 4:], pos.expand(3, T))          # one row for all axes
    assert torch.equal(a, b)
    c = x.clone()
    zp.zp_rope_apply_axes(axes, c[:, :4], c[:, 4:], torch.stack((pos,) * 3))
    assert torch.equal(a, c)


@pytest.mark.gpu
def test_a_slice_of_longer_positions(zp):
    """Positions of a step are columns of a longer array: the stride between axes is the array's."""
    x = torch.randn((9, 3, 64), device="cuda").to(torch.bfloat16)
    pos = torch.randint(0, 5000, (3, 40), device="cuda", dtype=torch.int32)
    axes = _init(zp, 64, 64, [12, 10, 10], "cycle", True)
    a, b = torch.empty_like(x), torch.empty_like(x)
    zp.zp_rope_apply_axes(axes, x, None, pos[:, 20:29], q_out=a)
    zp.zp_rope_apply_axes(axes, None, x, pos[:, 20:29].contiguous(), k_out=b)
    assert torch.equal(a, b) and bool((a != x).any())
