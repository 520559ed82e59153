"""Measured cases of the operators that bring a step's new tokens into the paged cache and attend from them: the step's
blocks and slots made on the GPU, rotary positions with several axes, cache writes by slot, attention of whole packed prompts
that have no cache yet, and attention of a chunk of new tokens over the 8-bit cache.

A case names its operator in "op" and its sizes; head shapes and block sizes are those of the synthetic workloads (32 / 8 heads
with 16-token blocks, 28 / 4 heads with 32-token blocks, and 4 / 2 heads of 64).  `run` computes the plain form in elementary
torch operations, or, where `own` is true, makes the calls of the library.
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

# (query heads, kv heads, head size, tokens of a block)
SHAPES = {"32x8": (32, 8, 128, 16), "28x4": (28, 4, 128, 32), "4x2": (4, 2, 64, 16)}


def listed():
    return [
        # one decode step of 256 running requests: one new token each, a block for those whose last one is full
        {"name": "slots decode", "op": "slots", "shape": "32x8", "requests": 256, "cached": 2047, "new": 1, "padded": 0},
        # a step that takes in prompts of 1 to 2047 tokens, with rows left over in the step's buffers
        {"name": "slots prefill", "op": "slots", "shape": "28x4", "requests": 48, "cached": 4000, "new": 2047, "padded": 300},
        # the new token's keys and values of 250 requests, in buffers of a captured step for 256
        {"name": "append decode", "op": "append", "shape": "32x8", "requests": 250, "cached": 2047, "new": 1, "padded": 6},
        # prompts of 1 to 1024 tokens written behind what earlier chunks left
        {"name": "append prefill", "op": "append", "shape": "32x8", "requests": 16, "cached": 1000, "new": 1024, "padded": 0},
        # a decode step of a model that reads images: time, height and width in sections of a head's pairs
        {"name": "axes decode", "op": "axes", "shape": "32x8", "tokens": 256, "far": 2048, "rotary": 128, "interleaved": False,
         "layout": "sections"},
        # a prompt of text and video frames, the axes in turn along the pairs
        {"name": "axes prompt", "op": "axes", "shape": "28x4", "tokens": 8192, "far": 100000, "rotary": 128, "interleaved": False,
         "layout": "cycle"},
        # first turns of 64 conversations in one step
        {"name": "prompts short", "op": "prompt", "shape": "32x8", "requests": 64, "least": 1, "most": 127, "window": 0, "sinks": 0},
        # ragged prompts through a layer with a window of 1024
        {"name": "prompts windowed", "op": "prompt", "shape": "32x8", "requests": 8, "least": 500, "most": 4001, "window": 1024,
         "sinks": 4},
        # one long document
        {"name": "prompt long", "op": "prompt", "shape": "28x4", "requests": 1, "least": 16383, "most": 16383, "window": 0, "sinks": 0},
        # verification of three drafted tokens and one more for each of 64 requests
        {"name": "kv8 drafts", "op": "kv8_chunk", "shape": "32x8", "requests": 64, "cached_least": 1, "cached_most": 8188,
         "new_least": 4, "new_most": 4, "window": 0, "sinks": 0},
        # chunked prefill: 2048 new tokens of each of 4 requests
        {"name": "kv8 chunk", "op": "kv8_chunk", "shape": "32x8", "requests": 4, "cached_least": 0, "cached_most": 6144,
         "new_least": 2048, "new_most": 2048, "window": 0, "sinks": 0},
        # short questions about long documents that stand in the cache
        {"name": "kv8 questions", "op": "kv8_chunk", "shape": "28x4", "requests": 8, "cached_least": 60000, "cached_most": 100000,
         "new_least": 17, "new_most": 64, "window": 0, "sinks": 0},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["slots", "append", "axes", "prompt", "prompt", "kv8_chunk", "kv8_chunk"])
    shape = rng.choice(sorted(SHAPES))
    Hq, Hkv, d, b = SHAPES[shape]
    if op in ("slots", "append"):
        requests = _log(rng, 1, 256)
        most = 65536 if op == "slots" else 8192
        return {"op": op, "shape": shape, "requests": requests, "cached": _log(rng, 1, 8000),
                "new": _log(rng, 1, max(1, min(8192, most // requests))), "padded": rng.choice([0, rng.randint(1, 300)])}
    if op == "axes":
        return {"op": op, "shape": shape, "tokens": _log(rng, 1, 8192), "far": _log(rng, 100, 1000000),
                "rotary": rng.choice([d, d // 2]), "interleaved": rng.random() < 0.5,
                "layout": rng.choice(["sections", "cycle", "restart"])}
    if op == "prompt":
        most = _log(rng, 1, 8192)
        requests = _log(rng, 1, max(1, min(64, (1 << 25) // (most * most))))
        return {"op": op, "shape": shape, "requests": requests, "least": rng.randint(1, most), "most": most,
                "window": rng.choice([0, _log(rng, 1, most)]), "sinks": rng.choice([0, 4, rng.randint(1, 64)])}
    new = _log(rng, 1, 4096)
    requests = _log(rng, 1, max(1, min(64, 4096 // new)))
    cached = _log(rng, 1, min(100000, max(1, (1 << 25) // (new * requests) - new)))
    return {"op": op, "shape": shape, "requests": requests, "cached_least": rng.randint(0, cached), "cached_most": cached,
            "new_least": rng.randint(1, new), "new_most": new, "window": rng.choice([0, _log(rng, 1, cached + new)]),
            "sinks": rng.choice([0, 4, rng.randint(1, 64)])}


# ---------------------------------------------------------------------------- sizes ----------

def _spread(lo, hi, n):
    """n whole numbers from lo to hi at even steps: a ragged batch whose total is the case's own."""
    return np.rint(np.linspace(lo, hi, n)).astype(np.int64)


def _rows(case):
    """(tokens cached before the call, new tokens) of each request, the longest cache with the fewest new tokens."""
    op, n = case["op"], case["requests"]
    if op == "prompt":
        return np.zeros(n, dtype=np.int64), _spread(case["least"], case["most"], n)
    if op == "kv8_chunk":
        return _spread(case["cached_least"], case["cached_most"], n)[::-1], _spread(case["new_least"], case["new_most"], n)
    new = _spread(1, case["new"], n) if n > 1 else np.array([case["new"]])
    return _spread(0, case["cached"], n)[::-1], new


def _visible(cached, new, window, sinks):
    """Visible keys of every query of a request, and the rows of keys that any of them sees."""
    p = np.arange(cached, cached + new)
    recent = p + 1 if window == 0 else np.minimum(p + 1, window)
    seen = recent + np.minimum(sinks, p + 1 - recent)
    first = 0 if window == 0 else max(0, cached + 1 - window)
    return int(seen.sum()), cached + new - first + min(sinks, first)


def work(case):
    Hq, Hkv, d, b = SHAPES[case["shape"]]
    op = case["op"]
    if op == "axes":
        T = case["tokens"]
        axes = 2 if case["layout"] == "restart" else 3
        return {"bytes": 2 * 2 * T * (Hq + Hkv) * d + 4 * axes * T, "flops": 3 * T * (Hq + Hkv) * case["rotary"]}
    cached, new = _rows(case)
    T = int(new.sum())
    if op == "slots":
        blocks = int(((cached + new + b - 1) // b - (cached + b - 1) // b).sum())
        return {"bytes": 4 * (3 * len(new) + 2 * blocks + 2 * len(new) + 1 + 2 * (T + case["padded"])), "flops": 4 * T}
    if op == "append":
        return {"bytes": T * (2 * Hkv * d * 4 + 4), "flops": 0}
    pairs, rows = (sum(x) for x in zip(*(_visible(int(c), int(n), case["window"], case["sinks"]) for c, n in zip(cached, new))))
    return {"bytes": rows * 2 * Hkv * d * (2 if op == "prompt" else 1) + T * Hq * d * 4, "flops": 4 * pairs * Hq * d}


# ---------------------------------------------------------------------------- inputs ---------

ROPE_THETA = 1e6


def _sections(case):
    """Pairs of each axis: time, height and width; or height and width, each with frequencies of its own from 1 on."""
    pairs = case["rotary"] // 2
    if case["layout"] == "restart":
        return [pairs // 2, pairs - pairs // 2]
    side = pairs * 3 // 8 if case["layout"] == "sections" else pairs // 3 - 1
    return [pairs - 2 * side, side, side]


def _codes(g, shape):
    """E4M3 codes of normal values at a scale of 2^-6, made in pieces."""
    out = torch.empty(shape, dtype=torch.uint8, device="cuda")
    flat, step = out.view(-1), 1 << 28
    for i in range(0, flat.numel(), step):
        n = min(step, flat.numel() - i)
        x = torch.randn(n, generator=g, device="cuda").mul_(64.0).clamp_(-448.0, 448.0)
        flat[i:i + n] = x.to(torch.float8_e4m3fn).view(torch.uint8)
    return out


def _scales(g, shape):
    return torch.exp2(torch.randint(-7, -4, shape, generator=g, device="cuda").float())


def _normal(g, *shape):
    return torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16)


def _i32(x):
    return torch.as_tensor(np.ascontiguousarray(x), dtype=torch.int32).cuda()


def _params(case, max_blocks):
    Hq, Hkv, d, b = SHAPES[case["shape"]]
    return dict(num_layers=1, num_q_heads=Hq, num_kv_heads=Hkv, head_dim=d, block_size=b, n_max=max(2, max_blocks), window=1,
                alpha=0.5, beta=0.5, decay=0.9, scale=1.0 / math.sqrt(d), protect_window=1, causal=1)


def prepare(case, seed):
    Hq, Hkv, d, b = SHAPES[case["shape"]]
    g = torch.Generator(device="cuda").manual_seed(seed)
    rng = np.random.default_rng(seed)
    op = case["op"]
    s = {"case": case}
    if op == "axes":
        T = case["tokens"]
        sections = _sections(case)
        qkv = _normal(g, T, Hq + 2 * Hkv, d)  # one fused projection: queries, keys and values of a token
        s["q"], s["k"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv]
        s["positions"] = torch.randint(0, case["far"], (len(sections), T), generator=g, device="cuda", dtype=torch.int32)
        s["q_out"], s["k_out"] = (torch.empty((T, h, d), dtype=torch.bfloat16, device="cuda") for h in (Hq, Hkv))
        if own:
            from paged_kv_cache_obs_gb300 import zipage
            layouts = {"sections": zipage.ZP_AXES_SECTIONS, "cycle": zipage.ZP_AXES_CYCLE, "restart": zipage.ZP_AXES_RESTART}
            s["rope"] = zipage.zp_rope_axes_init(d, case["rotary"], ROPE_THETA, sections, layouts[case["layout"]], case["interleaved"])
        return s

    order = rng.permutation(case["requests"])
    cached, new = (x[order] for x in _rows(case))
    total = cached + new
    T, n = int(new.sum()), len(new)
    before, used = -(-cached // b), -(-total // b)
    max_blocks = int(used.max())
    start = np.concatenate([[0], np.cumsum(new)])
    workspace = 256
    if op == "slots":
        NB = int(used.sum()) + 5
        ids = rng.permutation(NB)
        held = int(before.sum())
        tables = np.zeros((n, max_blocks), dtype=np.int64)
        tables[np.arange(max_blocks)[None, :] < before[:, None]] = ids[:held]
        s["tables"], s["free"] = _i32(tables), _i32(np.sort(ids[held:]))
        s["cached"], s["new"] = _i32(cached), _i32(new)
        # positions run ahead of the cache where a compression pass has dropped tokens
        s["first"] = _i32(cached + rng.integers(0, 5000, n))
        rows = T + case["padded"]
        s["positions"], s["slots"] = (torch.empty(rows, dtype=torch.int32, device="cuda") for _ in range(2))
        s["start"], s["seq"] = (torch.empty(k, dtype=torch.int32, device="cuda") for k in (n + 1, n))
        s["blocks"] = NB
    elif op == "append":
        # the pool holds the blocks that the call writes, and one that stands behind them
        first = cached // b
        NB = int((used - first).sum()) + 2
        ids, at = rng.permutation(NB), 0
        slots = np.full(T + case["padded"], -1, dtype=np.int64)
        for r in range(n):
            pos = np.arange(cached[r], total[r])
            slots[start[r]:start[r + 1]] = ids[at + pos // b - first[r]] * b + pos % b
            at += used[r] - first[r]
        s["pool"] = _normal(g, 1, NB + 1, 2, Hkv, b, d)
        qkv = _normal(g, len(slots), Hq + 2 * Hkv, d)
        s["k"], s["v"] = _normal(g, len(slots), Hkv, d), qkv[:, Hq + Hkv:]  # keys come from the rotation, values from the projection
        s["slots"] = _i32(slots)
    else:
        s["q"] = (3.0 * torch.randn((T, Hq, d), generator=g, device="cuda")).to(torch.bfloat16)
        s["out"] = torch.empty((T, Hq, d), dtype=torch.bfloat16, device="cuda")
        s["max_new"] = int(new.max())
        s["start"], s["seq"] = _i32(start), _i32(total)
        if op == "prompt":
            s["k"], s["v"] = _normal(g, T, Hkv, d), _normal(g, T, Hq + 2 * Hkv, d)[:, Hq + Hkv:]
        else:
            NB = int(used.sum()) + 3
            tables = np.zeros((n, max_blocks), dtype=np.int64)
            tables[np.arange(max_blocks)[None, :] < used[:, None]] = rng.permutation(NB)[:used.sum()]
            s["tables"] = _i32(tables)
            s["codes"], s["scales"] = _codes(g, (1, NB, 2, Hkv, b, d)), _scales(g, (1, NB, 2, Hkv))
    if own:
        from paged_kv_cache_obs_gb300 import zipage
        p = _params(case, max_blocks)
        s["params"] = zipage.make_params(p)
        if op == "prompt":
            workspace = zipage.zp_prompt_workspace_size(p, T, n, s["max_new"], case["window"], case["sinks"])
        if op == "kv8_chunk":
            workspace = zipage.zp_kv8_window_workspace_size(p, T, n, s["max_new"], max_blocks, case["window"], case["sinks"])
        s["workspace"] = zipage.new_workspace(workspace)
    return s


# ---------------------------------------------------------------------------- plain forms ----

def _plain_slots(s):
    b = SHAPES[s["case"]["shape"]][3]
    tables, free, cached, new, first = (s[x].long() for x in ("tables", "free", "cached", "new", "first"))
    total = cached + new
    before, used = (cached + b - 1) // b, (total + b - 1) // b
    start = torch.nn.functional.pad(torch.cumsum(new, 0), (1, 0))
    taken = torch.cumsum(used - before, 0) - (used - before)
    col = torch.arange(tables.shape[1], device=tables.device)
    fresh = (col >= before[:, None]) & (col < used[:, None])
    at = (taken[:, None] + col - before[:, None]).clamp(0, len(free) - 1)
    tables = torch.where(fresh, free[at], tables)
    t = torch.arange(len(s["slots"]), device=tables.device)
    r = (torch.searchsorted(start, t, right=True) - 1).clamp(max=len(new) - 1)
    i, real = t - start[r], t < start[-1]
    at = torch.where(real, cached[r] + i, 0)
    slots = torch.where(real, tables[r, at // b] * b + at % b, -1)
    positions = torch.where(real, first[r] + i, 0)
    return tuple(x.to(torch.int32) for x in (tables, start, total, positions, slots))


def _plain_append(s):
    pool, slots = s["pool"][0], s["slots"].long()
    b = pool.shape[3]
    # rows without a slot go to the block that stands behind the others
    slots = torch.where(slots < 0, (pool.shape[0] - 1) * b, slots)
    pool[slots // b, :, :, slots % b] = torch.stack((s["k"], s["v"]), dim=1)
    return s["pool"][:, :-1]


def _angles(case, positions):
    """cos and sin [T, 1, pairs] of every pair's angle, which is taken in 64 bits."""
    pairs, sections = case["rotary"] // 2, _sections(case)
    i = torch.arange(pairs, device="cuda")
    size = torch.tensor(sections, device="cuda")
    ends = torch.cumsum(size, 0)
    axis = torch.searchsorted(ends, i, right=True)
    order, count = i, torch.full_like(i, pairs)
    if case["layout"] == "cycle":
        turn = i % len(sections)
        axis = torch.where(i < size[turn] * len(sections), turn, 0)
    if case["layout"] == "restart":
        order, count = i - (ends - size)[axis], size[axis]
    f = ROPE_THETA ** (-order.double() / count)
    angle = (positions.double()[axis].T * f)[:, None]
    return angle.cos().float(), angle.sin().float()


def _plain_axes(s):
    case, rd = s["case"], s["case"]["rotary"]
    cos, sin = _angles(case, s["positions"])

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


def _attend(q, k, v, see, scale):
    """q [B, H, G, n, d], k and v [B, H, L, d], see [B, 1, 1, n, L] -> [B, H, G, n, d] in 32 bits."""
    x = torch.einsum("bhgnd,bhld->bhgnl", q, k).mul_(scale).masked_fill_(~see, -math.inf)
    top = x.amax(-1, keepdim=True)
    x = x.sub_(torch.where(top > -math.inf, top, torch.zeros_like(top))).exp_()
    total = x.sum(-1, keepdim=True)
    return torch.einsum("bhgnl,bhld->bhgnd", x, v) / torch.where(total > 0, total, torch.ones_like(total))


def _plain_attention(s):
    case, start, seq = s["case"], s["start"].long(), s["seq"].long()
    Hq, Hkv, d, b = SHAPES[case["shape"]]
    T, B, n = s["q"].shape[0], len(seq), s["max_new"]
    t = torch.arange(T, device="cuda")
    r = torch.searchsorted(start, t, right=True) - 1
    i = t - start[r]

    def padded(x):  # [T, H, d] -> [B, n, H, d]
        y = torch.zeros((B, n) + x.shape[1:], device="cuda")
        y[r, i] = x.float()
        return y

    if case["op"] == "prompt":
        k, v = padded(s["k"]).transpose(1, 2), padded(s["v"]).transpose(1, 2)
    else:
        tables = s["tables"].long()
        codes, scales = s["codes"][0].view(torch.float8_e4m3fn), s["scales"][0]
        k, v = ((codes[tables, x].float() * scales[tables, x][..., None, None]).transpose(1, 2).flatten(2, 3) for x in (0, 1))
    q = padded(s["q"]).view(B, n, Hkv, Hq // Hkv, d).permute(0, 2, 3, 1, 4)
    p = (seq[:, None] - (start[1:] - start[:-1])[:, None] + torch.arange(n, device="cuda"))[..., None]
    key = torch.arange(k.shape[2], device="cuda")
    see = (key <= p) & ((key > p - case["window"]) | (key < case["sinks"]) | (case["window"] == 0))
    out = _attend(q, k, v, see[:, None, None], 1.0 / math.sqrt(d))
    return out.permute(0, 3, 1, 2, 4)[r, i].reshape(T, Hq, d).to(torch.bfloat16)


PLAIN = {"slots": _plain_slots, "append": _plain_append, "axes": _plain_axes, "prompt": _plain_attention, "kv8_chunk": _plain_attention}


def run(s):
    case = s["case"]
    op = case["op"]
    if not own:
        return PLAIN[op](s)
    from paged_kv_cache_obs_gb300 import zipage
    if op == "slots":
        zipage.zp_step_slots(s["cached"], s["new"], s["free"], s["tables"], s["start"], s["seq"], s["slots"], s["params"],
                             s["workspace"], num_blocks=s["blocks"], positions=s["positions"], first_pos=s["first"])
        return s["tables"], s["start"], s["seq"], s["positions"], s["slots"]
    if op == "append":
        zipage.zp_kv_append(s["pool"], 0, s["k"], s["v"], s["slots"], s["params"], s["workspace"])
        return s["pool"][:, :-1]
    if op == "axes":
        zipage.zp_rope_apply_axes(s["rope"], s["q"], s["k"], s["positions"], q_out=s["q_out"], k_out=s["k_out"])
        return s["q_out"], s["k_out"]
    if op == "prompt":
        zipage.zp_prompt_attn(s["q"], s["k"], s["v"], s["start"], s["out"], s["params"], s["workspace"], s["max_new"],
                              window=case["window"], sinks=case["sinks"])
        return s["out"]
    zipage.zp_kv8_window_attn(s["codes"], s["scales"], 0, s["q"], s["start"], s["tables"], s["seq"], s["out"], s["params"],
                              s["workspace"], case["window"], case["sinks"], s["max_new"])
    return s["out"]


# ---------------------------------------------------------------------------- 64 bits --------

def _exact_slots(s, case):
    b = SHAPES[case["shape"]][3]
    tables, free = s["tables"].cpu().numpy().copy(), s["free"].cpu().tolist()
    cached, new, first = (s[x].cpu().tolist() for x in ("cached", "new", "first"))
    positions, slots, start, seq = [], [], [0], []
    for r in range(len(new)):
        for i in range(new[r]):
            at = cached[r] + i
            if at % b == 0:
                tables[r, at // b] = free.pop(0)
            slots.append(int(tables[r, at // b]) * b + at % b)
            positions.append(first[r] + i)
        start.append(len(slots))
        seq.append(cached[r] + new[r])
    pad = case["padded"]
    return tuple(torch.tensor(np.asarray(x), dtype=torch.int32) for x in (tables, start, seq, positions + [0] * pad, slots + [-1] * pad))


def _exact_append(s, case):
    b = SHAPES[case["shape"]][3]
    pool = s["pool"].double()
    for t, slot in enumerate(s["slots"].cpu().tolist()):
        if slot >= 0:
            pool[0, slot // b, 0, :, slot % b] = s["k"][t].double()
            pool[0, slot // b, 1, :, slot % b] = s["v"][t].double()
    return pool[:, :-1]


def _exact_axes(s, case):
    rd, sections = case["rotary"], _sections(case)
    pairs, A = rd // 2, len(sections)
    positions = s["positions"].double()
    angle = torch.empty((case["tokens"], pairs), dtype=torch.float64, device="cuda")
    for i in range(pairs):
        axis, left = 0, i
        while left >= sections[axis]:
            left -= sections[axis]
            axis += 1
        share = i / pairs if case["layout"] != "restart" else left / sections[axis]
        if case["layout"] == "cycle":
            axis = i % A if i < A * sections[i % A] else 0
        angle[:, i] = positions[axis] * math.exp(-math.log(ROPE_THETA) * share)
    wheel = torch.polar(torch.ones_like(angle), angle)[:, None, :]
    outs = []
    for x in (s["q"], s["k"]):
        x = x.double()
        y = x.clone()
        if case["interleaved"]:
            z = torch.view_as_complex(x[..., :rd].unflatten(-1, (pairs, 2)).contiguous()) * wheel
            y[..., 0:rd:2], y[..., 1:rd:2] = z.real, z.imag
        else:
            z = torch.complex(x[..., :pairs].contiguous(), x[..., pairs:rd].contiguous()) * wheel
            y[..., :pairs], y[..., pairs:rd] = z.real, z.imag
        outs.append(y)
    return tuple(outs)


def _exact_attention(s, case):
    Hq, Hkv, d, b = SHAPES[case["shape"]]
    G = Hq // Hkv
    start, seq = s["start"].cpu().tolist(), s["seq"].cpu().tolist()
    out = torch.zeros((start[-1], Hq, d), dtype=torch.float64, device="cuda")
    for r, L in enumerate(seq):
        lo, hi = start[r], start[r + 1]
        p = torch.arange(L - (hi - lo), L, device="cuda")[:, None]
        t = torch.arange(L, device="cuda")[None, :]
        hidden = t > p
        if case["window"]:
            hidden = hidden | ((t <= p - case["window"]) & (t >= case["sinks"]))
        for h in range(Hkv):
            if case["op"] == "prompt":
                key, value = s["k"][lo:hi, h].double(), s["v"][lo:hi, h].double()
            else:
                ids = s["tables"][r, :-(-L // b)].long()
                key, value = ((s["codes"][0, ids, i, h].view(torch.float8_e4m3fn).double() * s["scales"][0, ids, i, h].double()[:, None, None])
                              .reshape(-1, d)[:L] for i in (0, 1))
            for g in range(h * G, (h + 1) * G):
                x = torch.matmul(s["q"][lo:hi, g].double(), key.T) / math.sqrt(d)
                w = torch.softmax(x.masked_fill(hidden, -math.inf), dim=-1)
                out[lo:hi, g] = torch.matmul(w, value)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "slots":
        return _exact_slots(s, case)
    if case["op"] == "append":
        return _exact_append(s, case)
    if case["op"] == "axes":
        return _exact_axes(s, case)
    return _exact_attention(s, case)
