"""Measured cases of the operators around the paged cache: rotary positions, the 8-bit cache
(quantised as it is written, converted block by block from and to the bf16 pool, read by decode
attention) and attention with a sliding window and first tokens that stay visible.

A case names its operator in "op" and its sizes; head shapes and block sizes are those of the
synthetic workloads (32 / 8 heads with 16-token blocks, 28 / 4 heads with 32-token blocks, and 4 / 2
heads of 64).  `run` computes the plain form in elementary torch operations, or, where `own` is
true, makes the calls of the library.
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

# (query heads, kv heads, head size, tokens of a block)
SHAPES = {"32x8": (32, 8, 128, 16), "28x4": (28, 4, 128, 32), "4x2": (4, 2, 64, 16)}
QMAX = 448.0      # largest E4M3 value
MIN_EXP = -126    # smallest exponent of a block scale


def listed():
    return [
        # one decode step of 256 running requests: the new token's queries and keys
        {"name": "rope decode", "op": "rope", "shape": "32x8", "tokens": 256, "far": 2048, "rotary": 128,
         "interleaved": False, "scaling": "none"},
        # a prefill batch of long-context positions, interleaved pairs on half of the head
        {"name": "rope prefill", "op": "rope", "shape": "28x4", "tokens": 8192, "far": 1000000, "rotary": 64,
         "interleaved": True, "scaling": "yarn"},
        # one decode step: each of 256 requests appends its new token to a cache of up to 2048
        {"name": "append decode", "op": "append", "shape": "32x8", "requests": 256, "cached": 2047, "new": 1},
        # prompts of 1 to 1024 tokens written behind what chunked prefill left in the cache
        {"name": "append prefill", "op": "append", "shape": "32x8", "requests": 16, "cached": 1000, "new": 1024},
        # what a compression pass left of 8 requests (127 blocks each, 32 layers) moves to the 8-bit pool
        {"name": "pack blocks", "op": "pack", "shape": "32x8", "layers": 32, "blocks": 1016, "fill": 16},
        # a request at its cap (64 blocks of 32 tokens, 28 layers) is read back for its compression pass
        {"name": "unpack blocks", "op": "unpack", "shape": "28x4", "layers": 28, "blocks": 64, "fill": 32},
        # the smallest decode: four requests, short caches
        {"name": "kv8 decode small", "op": "kv8_decode", "shape": "32x8", "requests": 4, "least": 100, "most": 500,
         "window": 0, "sinks": 0},
        # the decoding requests of the mixed serving step
        {"name": "kv8 decode mixed", "op": "kv8_decode", "shape": "32x8", "requests": 224, "least": 1, "most": 2048,
         "window": 0, "sinks": 0},
        # few requests with long caches
        {"name": "kv8 decode long", "op": "kv8_decode", "shape": "28x4", "requests": 8, "least": 100000,
         "most": 131072, "window": 0, "sinks": 0},
        # decode of a layer with a window of 1024 over caches of up to 8192 tokens
        {"name": "window decode", "op": "window", "shape": "32x8", "requests": 64, "cached_least": 1,
         "cached_most": 8191, "new_least": 1, "new_most": 1, "window": 1024, "sinks": 4},
        # chunked prefill: 2048 new tokens of each of 4 requests
        {"name": "window chunk", "op": "window", "shape": "32x8", "requests": 4, "cached_least": 0,
         "cached_most": 6144, "new_least": 2048, "new_most": 2048, "window": 2048, "sinks": 16},
        # a whole prompt with a wide window
        {"name": "window prompt", "op": "window", "shape": "28x4", "requests": 1, "cached_least": 0,
         "cached_most": 0, "new_least": 8191, "new_most": 8191, "window": 4096, "sinks": 4},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["rope", "append", "pack", "unpack", "kv8_decode", "kv8_decode", "window", "window"])
    shape = rng.choice(sorted(SHAPES))
    Hq, Hkv, d, b = SHAPES[shape]
    if op == "rope":
        return {"op": op, "shape": shape, "tokens": _log(rng, 1, 8192), "far": _log(rng, 1000, 1000000),
                "rotary": rng.choice([d, d // 2, d // 4]), "interleaved": rng.random() < 0.5,
                "scaling": rng.choice(["none", "linear", "base", "yarn", "wavelength"])}
    if op == "append":
        requests = _log(rng, 1, 256)
        return {"op": op, "shape": shape, "requests": requests, "cached": _log(rng, 1, 4000),
                "new": _log(rng, 1, max(1, min(8192, 8192 // requests)))}
    if op in ("pack", "unpack"):
        layers = rng.choice([1, 2, 28, 32])
        return {"op": op, "shape": shape, "layers": layers, "blocks": _log(rng, 1, 1000 * 32 // max(layers, 16)),
                "fill": rng.randint(1, b)}
    if op == "kv8_decode":
        requests = _log(rng, 1, 256)
        most = _log(rng, 1, min(131072, (1 << 19) // requests))
        return {"op": op, "shape": shape, "requests": requests, "least": rng.randint(1, most), "most": most,
                "window": rng.choice([0, _log(rng, 1, most)]), "sinks": rng.choice([0, 4, rng.randint(1, 64)])}
    new = _log(rng, 1, 4096)
    requests = _log(rng, 1, max(1, min(64, 4096 // new)))
    cached = _log(rng, 1, min(16384, max(1, (1 << 25) // (new * requests) - new)))
    return {"op": op, "shape": shape, "requests": requests, "cached_least": rng.randint(0, cached),
            "cached_most": cached, "new_least": rng.randint(1, new), "new_most": new,
            "window": _log(rng, 1, cached + new), "sinks": rng.choice([0, 4, rng.randint(1, 64)])}


# ---------------------------------------------------------------------------- sizes ----------

def _spread(lo, hi, n):
    """n whole numbers from lo to hi at even steps: a ragged batch whose total is the case's own."""
    return np.rint(np.linspace(lo, hi, n)).astype(np.int64)


def _rows(case):
    """(tokens cached before the call, new tokens) of each request, in increasing order."""
    op, n = case["op"], case.get("requests", 0)
    if op == "append":
        new = _spread(1, case["new"], n) if n > 1 else np.array([case["new"]])
        return _spread(min(1, case["cached"]), case["cached"], n)[::-1], new
    if op == "kv8_decode":
        return _spread(case["least"], case["most"], n) - 1, np.ones(n, dtype=np.int64)
    return _spread(case["cached_least"], case["cached_most"], n)[::-1], _spread(case["new_least"], case["new_most"], n)


def _visible(cached, new, window, sinks):
    """Visible keys of every query of a request, and the rows of the cache that any of them sees."""
    p = np.arange(cached, cached + new)
    recent = p + 1 if window == 0 else np.minimum(p + 1, window)
    seen = recent + np.minimum(sinks, p + 1 - recent)
    first = 0 if window == 0 else max(0, cached + 1 - window)
    return int(seen.sum()), cached + new - first + min(sinks, first)


def work(case):
    Hq, Hkv, d, b = SHAPES[case["shape"]]
    op = case["op"]
    if op == "rope":
        T = case["tokens"]
        return {"bytes": 2 * 2 * T * (Hq + Hkv) * d + 4 * T, "flops": 3 * T * (Hq + Hkv) * case["rotary"]}
    if op in ("pack", "unpack"):
        tiles = case["layers"] * case["blocks"] * 2 * Hkv
        rows = case["blocks"] * b - (b - case["fill"] if op == "pack" else 0)  # of a layer and head
        values = case["layers"] * 2 * Hkv * rows * d
        return {"bytes": 3 * values + 4 * tiles, "flops": 2 * values}
    cached, new = _rows(case)
    T = int(new.sum())
    if op == "append":
        tiles = int(((cached + new + b - 1) // b - cached // b).sum()) * 2 * Hkv
        return {"bytes": T * 2 * Hkv * d * 3 + 4 * tiles, "flops": 2 * T * 2 * Hkv * d}
    pairs, rows = (sum(x) for x in zip(*(_visible(int(c), int(n), case["window"], case["sinks"])
                                         for c, n in zip(cached, new))))
    per_row = 2 * Hkv * d * (1 if op == "kv8_decode" else 2)
    return {"bytes": rows * per_row + T * Hq * d * 4, "flops": 4 * pairs * Hq * d}


# ---------------------------------------------------------------------------- inputs ---------

ROPE_THETA = 1e6
ROPE_SCALING = {"none": dict(), "linear": dict(factor=4.0), "base": dict(factor=8.0),
                "yarn": dict(factor=8.0, original_len=8192, low=1.0, high=32.0),
                "wavelength": dict(factor=8.0, original_len=8192, low=1.0, high=4.0)}


def _codes(g, shape):
    """E4M3 codes of normal values at a scale of 2^-6, made in pieces."""
    out = torch.empty(shape, dtype=torch.uint8, device="cuda")
    flat, step = out.view(-1), 1 << 28
    for i in range(0, flat.numel(), step):
        n = min(step, flat.numel() - i)
        x = torch.randn(n, generator=g, device="cuda").mul_(64.0).clamp_(-QMAX, QMAX)
        flat[i:i + n] = x.to(torch.float8_e4m3fn).view(torch.uint8)
    return out


def _scales(g, shape):
    return torch.exp2(torch.randint(-7, -4, shape, generator=g, device="cuda").float())


def _normal(g, *shape):
    return torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16)


def _i32(x):
    return torch.as_tensor(np.ascontiguousarray(x), dtype=torch.int32).cuda()


def _params(case, layers, max_blocks):
    Hq, Hkv, d, b = SHAPES[case["shape"]]
    return dict(num_layers=layers, num_q_heads=Hq, num_kv_heads=Hkv, head_dim=d, block_size=b, n_max=max(2, max_blocks),
                window=1, alpha=0.5, beta=0.5, decay=0.9, scale=1.0 / math.sqrt(d), protect_window=1, causal=1)


def prepare(case, seed):
    Hq, Hkv, d, b = SHAPES[case["shape"]]
    g = torch.Generator(device="cuda").manual_seed(seed)
    rng = np.random.default_rng(seed)
    op = case["op"]
    s = {"case": case}
    if op == "rope":
        T = case["tokens"]
        qkv = _normal(g, T, Hq + 2 * Hkv, d)  # one fused projection: queries, keys and values of a token
        s["q"], s["k"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv]
        s["positions"] = torch.randint(0, case["far"], (T,), generator=g, device="cuda", dtype=torch.int32)
        if own:
            from paged_kv_cache_obs_gb300 import zipage
            kinds = {"none": zipage.ZP_ROPE_NONE, "linear": zipage.ZP_ROPE_LINEAR, "base": zipage.ZP_ROPE_BASE,
                     "yarn": zipage.ZP_ROPE_YARN, "wavelength": zipage.ZP_ROPE_WAVELENGTH}
            s["rope"] = zipage.zp_rope_init(d, case["rotary"], ROPE_THETA, case["interleaved"],
                                            kinds[case["scaling"]], **ROPE_SCALING[case["scaling"]])
            s["q_out"] = torch.empty((T, Hq, d), dtype=torch.bfloat16, device="cuda")
            s["k_out"] = torch.empty((T, Hkv, d), dtype=torch.bfloat16, device="cuda")
        return s

    if op in ("pack", "unpack"):
        layers, n = case["layers"], case["blocks"]
        NB = n + 3
        s["src"], s["dst"] = _i32(rng.permutation(NB)[:n]), _i32(rng.permutation(NB)[:n])
        s["pool"] = torch.empty((layers, NB, 2, Hkv, b, d), dtype=torch.bfloat16, device="cuda")
        if op == "pack":
            for layer in range(layers):
                s["pool"][layer] = _normal(g, NB, 2, Hkv, b, d)
            s["codes"] = torch.zeros(s["pool"].shape, dtype=torch.uint8, device="cuda")
            s["scales"] = torch.zeros((layers, NB, 2, Hkv), device="cuda")
            # the last block of a request may be part full
            fill = np.full(n, b)
            fill[-1] = case["fill"]
            s["fill"] = _i32(fill)
        else:
            s["pool"].zero_()
            s["codes"], s["scales"] = _codes(g, s["pool"].shape), _scales(g, (layers, NB, 2, Hkv))
        if own:
            from paged_kv_cache_obs_gb300 import zipage
            s["params"] = zipage.make_params(_params(case, layers, n))
            s["workspace"] = zipage.new_workspace(256)
        return s

    order = rng.permutation(case["requests"])
    cached, new = (x[order] for x in _rows(case))
    total = cached + new
    T, n = int(new.sum()), len(new)
    used = -(-total // b)
    max_blocks = int(used.max())
    start = np.concatenate([[0], np.cumsum(new)])
    if op == "append":
        # the pool holds the blocks that the call writes; entries of earlier blocks are not read
        first = cached // b
        NB = int((used - first).sum()) + 2
        ids, at = rng.permutation(NB), 0
        tables = np.zeros((n, max_blocks), dtype=np.int64)
        for r in range(n):
            tables[r, first[r]:used[r]] = ids[at:at + used[r] - first[r]]
            at += used[r] - first[r]
        s["codes"], s["scales"] = _codes(g, (1, NB, 2, Hkv, b, d)), _scales(g, (1, NB, 2, Hkv))
        qkv = _normal(g, T, Hq + 2 * Hkv, d)
        s["k"], s["v"] = _normal(g, T, Hkv, d), qkv[:, Hq + Hkv:]  # keys come from the rotation, values from the projection
        s["cached"] = _i32(cached)
    else:
        NB = int(used.sum()) + 3
        ids = rng.permutation(NB)
        tables = np.zeros((n, max_blocks), dtype=np.int64)
        tables[np.arange(max_blocks)[None, :] < used[:, None]] = ids[:used.sum()]
        s["q"] = (3.0 * torch.randn((T, Hq, d), generator=g, device="cuda")).to(torch.bfloat16)
        if op == "kv8_decode":
            s["codes"], s["scales"] = _codes(g, (1, NB, 2, Hkv, b, d)), _scales(g, (1, NB, 2, Hkv))
        else:
            s["pool"] = _normal(g, 1, NB, 2, Hkv, b, d)
        s["seq"] = _i32(total)
        s["max_new"] = int(new.max())
    s["tables"], s["start"] = _i32(tables), _i32(start)
    if own:
        from paged_kv_cache_obs_gb300 import zipage
        p = _params(case, 1, max_blocks)
        s["params"] = zipage.make_params(p)
        nbytes = 256
        if op == "kv8_decode":
            nbytes = zipage.zp_kv8_decode_workspace_size(p, n, max_blocks)
        if op == "window":
            nbytes = zipage.zp_paged_window_workspace_size(p, T, n, s["max_new"], max_blocks, case["window"], case["sinks"])
        s["workspace"] = zipage.new_workspace(nbytes)
        if op != "append":
            s["out"] = torch.empty((T, Hq, d), dtype=torch.bfloat16, device="cuda")
    return s


# ---------------------------------------------------------------------------- plain forms ----

def _frequencies(case):
    """Radians per position of each rotated pair, and the factor on cos and sin, in 64 bits."""
    rd, c = case["rotary"], ROPE_SCALING[case["scaling"]]
    i = torch.arange(0, rd // 2, dtype=torch.float64, device="cuda")
    kind, factor = case["scaling"], c.get("factor", 1.0)
    theta = ROPE_THETA * factor ** (rd / (rd - 2)) if kind == "base" else ROPE_THETA
    f = theta ** (-2.0 * i / rd)
    if kind == "linear":
        f = f / factor
    if kind == "yarn":
        def turn(beta):  # the pair that makes beta turns over the original length
            return rd * math.log(c["original_len"] / (beta * 2 * math.pi)) / (2 * math.log(theta))
        lo, hi = max(math.floor(turn(c["high"])), 0), min(math.ceil(turn(c["low"])), rd - 1)
        ramp = ((i - lo) / max(hi - lo, 0.001)).clamp(0, 1)
        return f * (1 - ramp) + f / factor * ramp, 0.1 * math.log(factor) + 1.0
    if kind == "wavelength":
        turns = c["original_len"] * f / (2 * math.pi)
        mix = ((turns - c["low"]) / (c["high"] - c["low"])).clamp(0, 1)
        f = (1 - mix) * f / factor + mix * f
    return f, 1.0


def _plain_rope(s):
    case = s["case"]
    rd = case["rotary"]
    f, m = _frequencies(case)
    angle = s["positions"].double()[:, None, None] * f
    cos, sin = (angle.cos() * m).float(), (angle.sin() * m).float()

    def turned(x):
        x = x.float()
        rot, rest = x[..., :rd], x[..., rd:]
        if case["interleaved"]:
            a, c = rot[..., 0::2], rot[..., 1::2]
            y = torch.stack((a * cos - c * sin, c * cos + a * sin), dim=-1).flatten(-2)
        else:
            a, c = rot[..., :rd // 2], rot[..., rd // 2:]
            y = torch.cat((a * cos - c * sin, c * cos + a * sin), dim=-1)
        return torch.cat((y, rest), dim=-1).to(torch.bfloat16)

    return turned(s["q"]), turned(s["k"])


def _block_scale(amax):
    """The smallest power of two that brings amax to 448 or below (0 for an empty block)."""
    m, e = torch.frexp(amax)
    e = torch.where(m <= QMAX / 512, e - 9, e - 8).clamp(min=MIN_EXP)
    return torch.where(amax > 0, torch.exp2(e.float()), torch.zeros_like(amax))


def _inverse(scale):
    return torch.where(scale > 0, 1.0 / scale, torch.zeros_like(scale))


def _encode(x):
    return x.to(torch.float8_e4m3fn).view(torch.uint8)


def _decode(codes):
    return codes.view(torch.float8_e4m3fn).float()


def _plain_append(s):
    codes, scales, tables, cached, start = s["codes"][0], s["scales"][0], s["tables"].long(), s["cached"].long(), s["start"].long()
    b = codes.shape[3]
    x = torch.stack((s["k"], s["v"]), dim=1).float()  # [T, 2, H, d]
    t = torch.arange(x.shape[0], device=x.device)
    r = torch.searchsorted(start, t, right=True) - 1
    pos = cached[r] + t - start[r]
    block, slot = tables[r, pos // b], pos % b
    amax = torch.zeros_like(scales)
    amax.index_reduce_(0, block, x.abs().amax(-1), "amax")
    # rows already in the first block that each request writes
    first = tables[torch.arange(len(cached), device=x.device), cached // b]
    kept = (cached % b)[:, None, None, None, None] > torch.arange(b, device=x.device)[:, None]
    old = torch.where((cached % b > 0)[:, None, None], scales[first], torch.zeros_like(scales[first]))
    new = _block_scale(amax)
    new[first] = torch.maximum(new[first], old)
    again = _encode(_decode(codes[first]) * (old * _inverse(new[first]))[..., None, None])
    codes[first] = torch.where(kept, again, codes[first])
    codes[block, :, :, slot] = _encode(x * _inverse(new[block])[..., None])
    scales[block] = new[block]
    return s["codes"].view(torch.float8_e4m3fn), s["scales"]


def _plain_pack(s):
    src, dst = s["src"].long(), s["dst"].long()
    x = s["pool"][:, src].float()
    b = x.shape[4]
    valid = s["fill"].long()[:, None, None, None, None] > torch.arange(b, device=x.device)[:, None]
    scale = _block_scale((x.abs() * valid).amax((-1, -2)))
    s["codes"][:, dst] = torch.where(valid, _encode(x * _inverse(scale)[..., None, None]), s["codes"][:, dst])
    s["scales"][:, dst] = scale
    return s["codes"].view(torch.float8_e4m3fn), s["scales"]


def _plain_unpack(s):
    src, dst = s["src"].long(), s["dst"].long()
    s["pool"][:, dst] = (_decode(s["codes"][:, src]) * s["scales"][:, src][..., None, None]).to(torch.bfloat16)
    return s["pool"]


def _attend(q, k, v, see, scale):
    """q [B, H, G, n, d], k and v [B, H, L, d], see [B, 1, 1, n, L] -> [B, H, G, n, d] in 32 bits."""
    x = torch.einsum("bhgnd,bhld->bhgnl", q, k).mul_(scale).masked_fill_(~see, -math.inf)
    top = x.amax(-1, keepdim=True)
    x = x.sub_(torch.where(top > -math.inf, top, torch.zeros_like(top))).exp_()
    total = x.sum(-1, keepdim=True)
    return torch.einsum("bhgnl,bhld->bhgnd", x, v) / torch.where(total > 0, total, torch.ones_like(total))


def _seen(case, pos, length):
    """Which of the first `length` tokens a query at `pos` sees."""
    t = torch.arange(length, device=pos.device)
    p = pos[..., None]
    return (t <= p) & ((t > p - case["window"]) | (t < case["sinks"]) | (case["window"] == 0))


def _by_head(x):
    """[B, blocks, H, b, d] -> [B, H, blocks * b, d]"""
    return x.transpose(1, 2).flatten(2, 3)


def _plain_kv8_decode(s):
    case, tables = s["case"], s["tables"].long()
    Hq, Hkv, d, b = SHAPES[case["shape"]]
    codes, scales = s["codes"][0], s["scales"][0]
    k, v = (_by_head(_decode(codes[tables, i]) * scales[tables, i][..., None, None]) for i in (0, 1))
    q = s["q"].float().view(-1, Hkv, Hq // Hkv, 1, d)
    see = _seen(case, s["seq"].long()[:, None] - 1, k.shape[2])[:, None, None]
    return _attend(q, k, v, see, 1.0 / math.sqrt(d)).reshape(-1, Hq, d).to(torch.bfloat16)


def _plain_window(s):
    case, tables, start, seq = s["case"], s["tables"].long(), s["start"].long(), s["seq"].long()
    Hq, Hkv, d, b = SHAPES[case["shape"]]
    k, v = (_by_head(s["pool"][0][tables, i].float()) for i in (0, 1))
    T, B, n = s["q"].shape[0], len(seq), s["max_new"]
    t = torch.arange(T, device=start.device)
    r = torch.searchsorted(start, t, right=True) - 1
    i = t - start[r]
    q = torch.zeros((B, n, Hkv, Hq // Hkv, d), device=k.device)
    q[r, i] = s["q"].float().view(T, Hkv, Hq // Hkv, d)
    pos = seq[:, None] - (start[1:] - start[:-1])[:, None] + torch.arange(n, device=k.device)
    out = _attend(q.permute(0, 2, 3, 1, 4), k, v, _seen(case, pos, k.shape[2])[:, None, None], 1.0 / math.sqrt(d))
    return out.permute(0, 3, 1, 2, 4)[r, i].reshape(T, Hq, d).to(torch.bfloat16)


PLAIN = {"rope": _plain_rope, "append": _plain_append, "pack": _plain_pack, "unpack": _plain_unpack,
         "kv8_decode": _plain_kv8_decode, "window": _plain_window}


def run(s):
    case = s["case"]
    op = case["op"]
    if not own:
        return PLAIN[op](s)
    from paged_kv_cache_obs_gb300 import zipage
    if op == "rope":
        zipage.zp_rope_apply(s["rope"], s["q"], s["k"], s["positions"], q_out=s["q_out"], k_out=s["k_out"])
        return s["q_out"], s["k_out"]
    if op == "append":
        zipage.zp_kv8_append(s["codes"], s["scales"], 0, s["k"], s["v"], s["start"], s["cached"], s["tables"],
                             s["params"], s["workspace"])
        return s["codes"].view(torch.float8_e4m3fn), s["scales"]
    if op == "pack":
        zipage.zp_kv8_pack_blocks(s["pool"], s["src"], s["codes"], s["scales"], s["dst"], s["params"], s["workspace"],
                                  fill=s["fill"])
        return s["codes"].view(torch.float8_e4m3fn), s["scales"]
    if op == "unpack":
        zipage.zp_kv8_unpack_blocks(s["codes"], s["scales"], s["src"], s["pool"], s["dst"], s["params"], s["workspace"])
        return s["pool"]
    if op == "kv8_decode":
        zipage.zp_kv8_decode_attn(s["codes"], s["scales"], 0, s["q"], s["tables"], s["seq"], s["out"], s["params"],
                                  s["workspace"], window=case["window"], sinks=case["sinks"])
        return s["out"]
    zipage.zp_paged_window_attn(s["pool"], 0, s["q"], s["start"], s["tables"], s["seq"], s["out"], s["params"],
                                s["workspace"], case["window"], case["sinks"], s["max_new"])
    return s["out"]


# ---------------------------------------------------------------------------- 64 bits --------

def _nearest_e4m3(x):
    """The E4M3 value nearest to x (ties to even), by the grid's spacing around x."""
    size = x.abs()
    e = torch.floor(torch.log2(size.clamp(min=2.0 ** -60))).clamp(min=-6.0)
    step = torch.exp2(e - 3.0)
    return torch.copysign((torch.round(size / step) * step).clamp(max=QMAX), x)


def _least_scale(amax):
    if amax <= 0:
        return 0.0
    e = math.ceil(math.log2(amax / QMAX) - 1e-9)
    return 2.0 ** max(e, MIN_EXP)


def _exact_rope(s, case):
    rd, T = case["rotary"], case["tokens"]
    c = ROPE_SCALING[case["scaling"]]
    factor, freqs, size = c.get("factor", 1.0), [], 1.0
    base = ROPE_THETA * (factor ** (rd / (rd - 2.0)) if case["scaling"] == "base" else 1.0)
    for i in range(rd // 2):
        f = 1.0 / base ** (2.0 * i / rd)
        if case["scaling"] == "linear":
            f /= factor
        if case["scaling"] == "wavelength":
            wave = 2.0 * math.pi / f
            if wave > c["original_len"] / c["low"]:
                f /= factor
            elif wave > c["original_len"] / c["high"]:
                smooth = (c["original_len"] / wave - c["low"]) / (c["high"] - c["low"])
                f = (1.0 - smooth) * f / factor + smooth * f
        if case["scaling"] == "yarn":
            size = 0.1 * math.log(factor) + 1.0
            edge = [rd * math.log(c["original_len"] / (beta * 2.0 * math.pi)) / (2.0 * math.log(base))
                    for beta in (c["high"], c["low"])]
            lo, hi = max(math.floor(edge[0]), 0), min(math.ceil(edge[1]), rd - 1)
            ramp = min(1.0, max(0.0, (i - lo) / max(hi - lo, 0.001)))
            f = f / factor * ramp + f * (1.0 - ramp)
        freqs.append(f)
    angle = s["positions"].double()[:, None] * torch.tensor(freqs, dtype=torch.float64, device="cuda")
    wheel = torch.polar(torch.full_like(angle, size), angle)[:, None, :]
    outs = []
    for x in (s["q"], s["k"]):
        x = x.double()
        y = x.clone()
        if case["interleaved"]:
            z = torch.view_as_complex(x[..., :rd].unflatten(-1, (rd // 2, 2)).contiguous()) * wheel
            y[..., 0:rd:2], y[..., 1:rd:2] = z.real, z.imag
        else:
            z = torch.complex(x[..., :rd // 2].contiguous(), x[..., rd // 2:rd].contiguous()) * wheel
            y[..., :rd // 2], y[..., rd // 2:rd] = z.real, z.imag
        outs.append(y)
    return tuple(outs)


def _exact_append(s, case):
    Hq, Hkv, d, b = SHAPES[case["shape"]]
    codes = s["codes"].view(torch.float8_e4m3fn).double()[0]
    scales = s["scales"].double()[0].cpu()
    x = torch.stack((s["k"], s["v"]), dim=1).double()
    tables, start, cached = s["tables"].cpu().numpy(), s["start"].cpu().numpy(), s["cached"].cpu().numpy()
    if len(cached) * Hkv * 2 + x.shape[0] // b * Hkv * 2 > 12000:
        return None
    size = x.abs().amax(-1).cpu()
    for r in range(len(cached)):
        at, end, t = int(cached[r]), int(cached[r] + start[r + 1] - start[r]), int(start[r])
        while at < end:
            n = min(end, (at // b + 1) * b) - at
            block, lo = int(tables[r, at // b]), at % b
            for i in range(2):
                top = size[t:t + n, i].amax(0)
                for h in range(Hkv):
                    old = float(scales[block, i, h]) if lo else 0.0
                    new = max(old, _least_scale(float(top[h])))
                    if lo and new > old:
                        codes[block, i, h, :lo] = _nearest_e4m3(codes[block, i, h, :lo] * (old / new))
                    scales[block, i, h] = new
            sc = scales[block].to(x.device)
            codes[block, :, :, lo:lo + n] = _nearest_e4m3(x[t:t + n] / torch.where(sc > 0, sc, 1.0)[..., None]).permute(1, 2, 0, 3)
            at, t = at + n, t + n
    return codes[None], scales[None]


def _exact_pack(s, case):
    codes, scales = s["codes"].view(torch.float8_e4m3fn).double(), s["scales"].double()
    if codes.numel() > 3 << 29:
        return None
    src, dst, fill = (s[n].cpu().tolist() for n in ("src", "dst", "fill"))
    for layer in range(case["layers"]):
        x = s["pool"][layer].double()
        for rows in sorted(set(fill)):
            some = [n for n in range(len(src)) if fill[n] == rows]
            y = x[[src[n] for n in some], :, :, :rows]
            top = y.abs().flatten(3).amax(-1)
            e = torch.ceil(torch.log2(top / QMAX) - 1e-9).clamp(min=float(MIN_EXP))
            scale = torch.where(top > 0, torch.exp2(e), 0.0)
            codes[layer, [dst[n] for n in some], :, :, :rows] = _nearest_e4m3(y / torch.where(scale > 0, scale, 1.0)[..., None, None])
            scales[layer, [dst[n] for n in some]] = scale
    return codes, scales


def _exact_unpack(s, case):
    if s["pool"].numel() > 3 << 29:
        return None
    pool = s["pool"].double()
    for layer in range(case["layers"]):
        values = s["codes"][layer].view(torch.float8_e4m3fn).double() * s["scales"][layer].double()[..., None, None]
        pool[layer].index_copy_(0, s["dst"].long(), values.index_select(0, s["src"].long()))
    return pool


def _exact_attention(s, case):
    Hq, Hkv, d, b = SHAPES[case["shape"]]
    G = Hq // Hkv
    start, seq = s["start"].cpu().tolist(), s["seq"].cpu().tolist()
    out = torch.zeros((start[-1], Hq, d), dtype=torch.float64, device="cuda")
    for r, L in enumerate(seq):
        ids = s["tables"][r, :-(-L // b)].long()
        n = start[r + 1] - start[r]
        p = torch.arange(L - n, L, device="cuda")[:, None]
        t = torch.arange(L, device="cuda")[None, :]
        hidden = t > p
        if case["window"]:
            hidden = hidden | ((t <= p - case["window"]) & (t >= case["sinks"]))
        if "codes" in s:
            kv = s["codes"][0][ids].view(torch.float8_e4m3fn).double() * s["scales"][0][ids].double()[..., None, None]
        else:
            kv = s["pool"][0][ids].double()
        for h in range(Hkv):
            key, value = (kv[:, i, h].reshape(-1, d)[:L] for i in (0, 1))
            q = s["q"][start[r]:start[r + 1], h * G:(h + 1) * G].double().transpose(0, 1)
            x = torch.matmul(q, key.T) / math.sqrt(d)
            w = torch.softmax(x.masked_fill(hidden, -math.inf), dim=-1)
            out[start[r]:start[r + 1], h * G:(h + 1) * G] = torch.matmul(w, value).transpose(0, 1)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "rope":
        return _exact_rope(s, case)
    if op == "append":
        return _exact_append(s, case)
    if op == "pack":
        return _exact_pack(s, case)
    if op == "unpack":
        return _exact_unpack(s, case)
    return _exact_attention(s, case)
