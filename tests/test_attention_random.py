"""Random calls of the attention operators around the cache (seeded): shapes, lengths, windows, first
tokens, strides, workspaces, values that are not finite and one bad request, every checked row against
64 bits."""
import math
import os
import random

import numpy as np
import pytest
import torch

import test_attention_edges as E
import test_cache_attention as A

pytestmark = pytest.mark.gpu

SHAPES = A.SHAPES + [(12, 4, 128, 16), (24, 2, 64, 32), (13, 1, 128, 32), (32, 32, 64, 16), (5, 5, 128, 16)]


@pytest.fixture(scope="module")
def zp():
    from paged_kv_cache_obs_gb300 import build
    if not os.path.exists(build.LIB):
        build.build()
    from paged_kv_cache_obs_gb300 import zipage
    return zipage


def _exact(q, k, v, seen, scale):
    """Rows q [n, d] in 64 bits over the tokens seen [n, L] (values that are not finite reach those alone)."""
    w = torch.softmax((scale * (q.double() @ k.double().T)).masked_fill(~seen, -math.inf), -1)
    v = v.double()
    out, mass = (w @ torch.where(torch.isfinite(v), x, torch.zeros_like(v)) for x in (v, v.abs()))
    up, down, nan = (seen.double() @ x.double() > 0 for x in (v == math.inf, v == -math.inf, torch.isnan(v)))
    out[up], out[down] = math.inf, -math.inf
    out[nan | (up & down)] = math.nan
    return out, mass


def _check(got, want, mass, rel, floor, info):
    got = got.double()
    nan, fin = torch.isnan(want), torch.isfinite(want)
    assert torch.equal(nan, torch.isnan(got)), info
    assert torch.equal(want[~nan & ~fin], got[~nan & ~fin]), info
    err = (got - want).abs()[fin]
    # as in test_cache_attention; E4M3: weights below 2^-28 of the largest are lost beside it
    assert bool((err <= 2.0 ** -8 * want[fin].abs() + (rel + 2.0 ** -14) * mass[fin] + 1e-30 + floor).all()), info


def _layout(rng, T, heads, d):
    plain = torch.zeros((T, heads, d), dtype=torch.bfloat16, device="cuda")
    return plain if rng.random() < 0.5 else rng.choice(list(E._layouts(T, heads, d, None)))[1]


def _case(zp, kind, seed):
    rng = random.Random(f"{kind} {seed}")
    g = torch.Generator(device="cuda").manual_seed(seed)
    spread = lambda a, b: int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))
    randn = lambda *s: torch.randn(s, generator=g, device="cuda")
    Hq, Hkv, d, b = rng.choice(SHAPES)
    G = Hq // Hkv
    B = rng.choice([1, 1, 2, 3, 5, rng.randint(6, 60)])
    top = spread(1, 12000 if B < 4 else 3000 if B < 10 else 600)
    most = {"kv8": 0, "few": max(1, 16 // G), "many": spread(1, 1500 if B < 4 else 200)}[kind]
    new = [rng.randint(0, most) for _ in range(B)]
    if most and not sum(new):
        new[0] = 1
    lens = [rng.randint(0, top) + n for n in new]
    window = rng.choice([0, 0, 1, spread(1, 5000), spread(1, 300), max(1, int(max(lens) * rng.uniform(0.3, 1.0)))])
    sinks = rng.choice([0, 0, 1, 4, spread(1, 400)]) if window else 0
    mb = max(1, max(-(-L // b) for L in lens)) + rng.randint(0, 3)
    NB = sum(-(-L // b) for L in lens) + 3
    order = torch.randperm(NB, generator=g, device="cuda").to(torch.int32)
    tables = torch.full((B, mb), -1, dtype=torch.int32, device="cuda")
    at = 0
    for r, L in enumerate(lens):
        n = -(-L // b)
        tables[r, :n] = order[at:at + n]
        at += n
    p = A._params(Hq, Hkv, d, b, 2)
    T, pad = (B, 0) if kind == "kv8" else (sum(new), rng.choice([0, 7]))
    q, out = _layout(rng, T + pad, Hq, d), _layout(rng, T + pad, Hq, d)
    q.copy_(randn(T + pad, Hq, d) * rng.choice([0.5, 2.0, 4.0]))
    q[T:] = math.nan
    out.fill_(7.0)
    seq = E._i32(lens)
    # one request may be bad: the others do not notice
    bad = rng.choice([None, None, rng.randrange(B)]) if B > 1 else None
    if bad is not None and (kind == "kv8" or new[bad] > 0) and lens[bad] > 0:
        if rng.random() < 0.5:
            seq[bad] = rng.choice([-1, mb * b + 1, 2 ** 31 - 1, -2 ** 31])
        else:
            tables[bad, (lens[bad] - 1) // b] = rng.choice([-1, NB, 2 ** 31 - 1, -2 ** 31])
    else:
        bad = None
    info = (kind, seed, Hq, Hkv, d, b, B, lens[:5], new[:5], window, sinks)
    if kind == "kv8":
        codes = (randn(2, NB, 2, Hkv, b, d) * 64).clamp(-448, 448).to(torch.float8_e4m3fn)
        low = rng.choice([-9, -20])
        scales = torch.exp2(torch.randint(low, -4, (2, NB, 2, Hkv), generator=g, device="cuda").float())
        scales *= 1 + torch.rand(scales.shape, generator=g, device="cuda")
        pool = codes.double() * scales.double()[..., None, None]
        own = zp.zp_kv8_decode_workspace_size(p, B, mb)
        start, mq, rel = list(range(B + 1)), 1, 2.0 ** -11
        call = lambda ws: zp.zp_kv8_decode_attn(codes, scales, 1, q, tables, seq, out, p, ws, window=window, sinks=sinks)
    else:
        pool = randn(2, NB, 2, Hkv, b, d).to(torch.bfloat16)
        for _ in range(rng.choice([0, 0, 1, 30])):
            pool[1, rng.randrange(NB), 1, rng.randrange(Hkv), rng.randrange(b), rng.randrange(d)] = rng.choice([math.inf, -math.inf, math.nan])
        mq = max(new) + rng.choice([0, 0, rng.randint(0, 100)])
        own = zp.zp_paged_window_workspace_size(p, T + pad, B, mq, mb, window, sinks)
        start, rel = np.concatenate([[0], np.cumsum(new)]).tolist(), A.SPLIT if G * mq <= 16 else A.TILED
        d_start = E._i32(start)
        call = lambda ws: zp.zp_paged_window_attn(pool, 1, q, d_start, tables, seq, out, p, ws, window, sinks, mq)
    ws = zp.new_workspace(rng.choice([own, own, 256, max(256, own // 512 * 256)]))
    call(ws)
    first = out.clone()
    call(ws)
    assert torch.equal(first.view(torch.int16), out.contiguous().view(torch.int16)), info
    assert zp.zp_read_error(ws) == (0 if bad is None else zp.ZP_ERR_BAD_TABLE), info
    assert bool((out[T:] == 7).all()), info
    for r in rng.sample(range(B), min(B, 4)):
        L, n = lens[r], start[r + 1] - start[r]
        if r == bad or n == 0:
            continue
        if L == 0:
            assert not bool(out[r].any()), info
            continue
        rows = torch.tensor(sorted(rng.sample(range(n), min(n, 64))), device="cuda")
        seen = E._visible(L - n + rows, L, window, sinks)
        for h in rng.sample(range(Hkv), min(Hkv, 2)):
            k, v = (E._tokens(pool, 1, tables[r][:-(-L // b)], i, h, L) for i in (0, 1))
            floor = 2.0 ** -28 * float(v.abs().max()) if kind == "kv8" else 0.0
            for head in rng.sample(range(h * G, (h + 1) * G), min(G, 3)):
                _check(out[start[r] + rows, head], *_exact(q[start[r] + rows, head], k, v, seen, p["scale"]), rel, floor,
                       info + (r, head))


@pytest.mark.parametrize("seeds", range(8))
@pytest.mark.parametrize("kind", ["kv8", "few", "many"])
def test_random_calls(zp, kind, seeds):
    for seed in range(seeds * 60, seeds * 60 + 60):
        _case(zp, kind, seed)
