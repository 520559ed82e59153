"""Rotary positions at the sizes of whole models: a CTA's rows take several passes there, and tokens go
two to a CTA from 1024 on."""
import os

import numpy as np
import pytest
import torch

from oracle import serving_oracle as S
from test_rope import THETA, _check, _f64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def zp():
    from paged_kv_cache_obs_gb300 import build
    if not os.path.exists(build.LIB):
        build.build()
    from paged_kv_cache_obs_gb300 import zipage
    return zipage


@pytest.mark.parametrize("T", [1, 3, 1023, 1024, 1025])
@pytest.mark.parametrize("Hq,Hkv,rd", [(32, 8, 128), (28, 4, 64)])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("off", [0, 1])
def test_apply_at_model_sizes(zp, T, Hq, Hkv, rd, inter, off):
    d = 128
    g = torch.Generator(device="cuda").manual_seed(T + Hq)
    n = T * (Hq + 2 * Hkv) * d
    buf = torch.randn(n + 8, generator=g, device="cuda").to(torch.bfloat16)
    x = buf[off:off + n].view(T, Hq + 2 * Hkv, d)
    before = x.clone()
    pos = torch.randint(-5, 1000000, (T,), generator=g, device="cuda", dtype=torch.int32)
    rope = zp.zp_rope_init(d, rd, THETA, interleaved=inter)
    qo, ko = (torch.full((T, h, d), 7.0, dtype=torch.bfloat16, device="cuda") for h in (Hq, Hkv))
    zp.zp_rope_apply(rope, x[:, :Hq], x[:, Hq:Hq + Hkv], pos, q_out=qo, k_out=ko)
    assert torch.equal(x, before)
    f, size = S.rope_frequencies(rd, THETA)
    p = pos.cpu().numpy().astype(np.int64)
    # the ends and a stretch in the middle against 64 bits; the rest against the narrow form's bits below
    for rows in (slice(0, 3), slice(T // 2, T // 2 + 3), slice(max(T - 3, 0), T)):
        _check(_f64(qo[rows]), _f64(before[rows, :Hq]), p[rows], f, size, inter)
        _check(_f64(ko[rows]), _f64(before[rows, Hq:Hq + Hkv]), p[rows], f, size, inter)
    # every token by itself gives the same bits, whatever its neighbours
    if T >= 1023:
        y = before.clone()
        for a in range(0, T, 511):
            zp.zp_rope_apply(rope, y[a:a + 511, :Hq], y[a:a + 511, Hq:Hq + Hkv], pos[a:a + 511].contiguous())
        assert torch.equal(y[:, :Hq], qo) and torch.equal(y[:, Hq:Hq + Hkv], ko)
    # in place: the same bits, the values behind the keys stay
    zp.zp_rope_apply(rope, x[:, :Hq], x[:, Hq:Hq + Hkv], pos)
    assert torch.equal(x[:, :Hq], qo) and torch.equal(x[:, Hq:Hq + Hkv], ko)
    assert torch.equal(x[:, Hq + Hkv:], before[:, Hq + Hkv:])
    assert torch.equal(qo[..., rd:], before[:, :Hq, rd:])
