"""The way of a step's tokens into the cache and out of it again, as a serving loop runs it: slots and tables on the device,
rotary positions with several axes, cache writes into both pools, attention of the prompts, then of chunks and drafts over the
8-bit cache, eagerly and as a captured step."""
import math
import os

import numpy as np
import pytest
import torch

import test_cache_attention as A
from oracle import serving_oracle as S

pytestmark = pytest.mark.gpu

Hq, Hkv, d, b, MB = 8, 2, 64, 16, 24
SECTIONS, THETA = [12, 10, 10], 1e4


@pytest.fixture(scope="module")
def zp():
    from paged_kv_cache_obs_gb300 import build
    if not os.path.exists(build.LIB):
        build.build()
    from paged_kv_cache_obs_gb300 import zipage
    return zipage


def _i32(x):
    return torch.as_tensor(np.ascontiguousarray(x), dtype=torch.int32).cuda()


def _attend(q, k, v, first, scale):
    """Rows q [n, Hq, d] at positions first, first + 1, ... over k, v [L, Hkv, d] in 64 bits: outputs and weighted magnitudes."""
    n, L = q.shape[0], k.shape[0]
    see = torch.arange(L, device="cuda")[None, :] <= first + torch.arange(n, device="cuda")[:, None]
    want, mass = (torch.empty((n, Hq, d), dtype=torch.float64, device="cuda") for _ in range(2))
    for h in range(Hq):
        key, value = k[:, h // (Hq // Hkv)], v[:, h // (Hq // Hkv)]
        w = torch.softmax((scale * (q[:, h].double() @ key.T)).masked_fill(~see, -math.inf), -1)
        want[:, h], mass[:, h] = w @ value, w @ value.abs()
    return want, mass


class Loop:
    """The state that a serving loop keeps, and one step of it."""

    def __init__(self, zp, B, T, seed):
        self.zp, self.B, self.T = zp, B, T
        rng = np.random.default_rng(seed)
        self.g = torch.Generator(device="cuda").manual_seed(seed)
        self.NB = B * MB
        self.pool = torch.zeros((1, self.NB, 2, Hkv, b, d), dtype=torch.bfloat16, device="cuda")
        self.codes = torch.zeros(self.pool.shape, dtype=torch.uint8, device="cuda")
        self.scales = torch.zeros((1, self.NB, 2, Hkv), device="cuda")
        self.tables = torch.full((B, MB), -1, dtype=torch.int32, device="cuda")
        self.free, self.at = _i32(rng.permutation(self.NB)), _i32([0])
        self.cached, self.before, self.new, self.ahead = (_i32(np.zeros(B)) for _ in range(4))
        self.start, self.pos, self.slots = _i32(np.zeros(B + 1)), _i32(np.zeros(T)), _i32(np.zeros(T))
        self.axes = torch.zeros((3, T), dtype=torch.int32, device="cuda")
        self.qkv = torch.zeros((T, Hq + 2 * Hkv, d), dtype=torch.bfloat16, device="cuda")
        self.q, self.k = (torch.zeros((T, h, d), dtype=torch.bfloat16, device="cuda") for h in (Hq, Hkv))
        self.out = torch.zeros((T, Hq, d), dtype=torch.bfloat16, device="cuda")
        self.p = zp.make_params(A._params(Hq, Hkv, d, b))
        self.scale = 1.0 / math.sqrt(d)
        self.rope = zp.zp_rope_axes_init(d, d, THETA, SECTIONS, zp.ZP_AXES_CYCLE)
        need = [zp.zp_prompt_workspace_size(self.p, T, B, n) for n in (100, 300, T)]
        need += [zp.zp_kv8_window_workspace_size(self.p, T, B, n, MB, 0, 0) for n in (3, 4, 60)]
        need += [zp.zp_paged_window_workspace_size(self.p, T, B, n, MB, 0, 0) for n in (3, 4, 60)]
        self.ws = zp.new_workspace(max(need))

    def inputs(self, new, picture=0):
        """New tokens' projections; `picture`: tokens of each request whose height and width are places in rows of 5."""
        self.new.copy_(_i32(new))
        self.qkv.copy_(torch.randn(self.qkv.shape, generator=self.g, device="cuda"))
        self.picture = picture

    def write(self):
        """Slots, positions, rotation, both caches: what may be captured."""
        zp = self.zp
        self.before.copy_(self.cached)
        first = self.before + self.ahead                         # positions run ahead where tokens were dropped
        zp.zp_step_slots(self.cached, self.new, self.free, self.tables, self.start, self.cached, self.slots, self.p, self.ws,
                         num_blocks=self.NB, positions=self.pos, first_pos=first, free_at=self.at)
        here = self.pos[None, :].expand(3, self.T)
        place = torch.stack((self.pos, self.pos // 5, self.pos % 5))
        self.axes.copy_(torch.where(self.pos[None, :] < self.picture, place, here))
        zp.zp_rope_apply_axes(self.rope, self.qkv[:, :Hq], self.qkv[:, Hq:Hq + Hkv], self.axes, q_out=self.q, k_out=self.k)
        v = self.qkv[:, Hq + Hkv:]
        zp.zp_kv_append(self.pool, 0, self.k, v, self.slots, self.p, self.ws)
        zp.zp_kv8_append(self.codes, self.scales, 0, self.k, v, self.start, self.before, self.tables, self.p, self.ws)

    def check_written(self, kept):
        """The bf16 pool holds every request's rotated keys and values in order, the 8-bit pool their codes."""
        start, L = self.start.tolist(), self.cached.tolist()
        x = self.qkv.double().cpu().numpy()
        rot = S.rope_axes(x[:, :Hq + Hkv], self.axes.cpu().numpy().astype(np.int64), d, THETA, SECTIONS, "cycle", False)
        n = start[-1]
        got = torch.cat((self.q, self.k), 1).double().cpu().numpy()
        assert (np.abs(got[:n] - rot[:n]) <= 2.0 ** -8 * np.abs(rot[:n]) + 2.0 ** -20 * np.abs(x).max()).all()
        for r in range(self.B):
            rows = slice(start[r], start[r + 1])
            if L[r] == 0:
                continue
            kept[r] = torch.cat((kept[r], torch.stack((self.k[rows], self.qkv[rows, Hq + Hkv:]))), 1)
            ids = self.tables[r, :-(-L[r] // b)].long()
            flat = lambda pool: pool.transpose(0, 1).transpose(2, 3).flatten(1, 2)[:, :L[r]]    # [2, L, H, d]
            assert kept[r].shape[1] == L[r] and torch.equal(flat(self.pool[0, ids]), kept[r])
            eight = flat(self.codes[0, ids].view(torch.float8_e4m3fn).float() * self.scales[0, ids][..., None, None])
            # E4M3 of a value under its block's scale: 2^-4 of itself, or half of the least step (2^-10 of the scale, below
            # 2^-18 of the block's largest); rounded again where a block's scale grew
            assert bool(((eight - kept[r].float()).abs() <= 2.0 ** -3 * kept[r].float().abs() + 2.0 ** -8 * kept[r].float().abs().max() / 448).all())

    def exact(self, r, pool8):
        L = self.cached[r].item()
        ids = self.tables[r, :-(-L // b)].long()
        pool = self.codes[0, ids].view(torch.float8_e4m3fn).double() * self.scales[0, ids].double()[..., None, None] if pool8 else self.pool[0, ids].double()
        return pool.transpose(0, 1).transpose(2, 3).flatten(1, 2)[:, :L]

    def check_rows(self, out, pool8, rel):
        start = self.start.tolist()
        for r in range(self.B):
            rows = slice(start[r], start[r + 1])
            if rows.start == rows.stop:
                continue
            k, v = self.exact(r, pool8)
            want, mass = _attend(self.q[rows], k, v, self.before[r].item(), self.scale)
            err = (out[rows].double() - want).abs()
            tol = 2.0 ** -8 * want.abs() + (rel + 2.0 ** -14) * mass + 2.0 ** -29 * k.shape[0] * v.abs().max() + 1e-30
            assert bool((err <= tol).all()), (r, float((err / tol).max()))


def test_prompts_chunks_and_drafts(zp):
    B, T = 6, 420
    loop, rng = Loop(zp, B, T, 1), np.random.default_rng(2)
    kept = [torch.zeros((2, 0, Hkv, d), dtype=torch.bfloat16, device="cuda") for _ in range(B)]
    for lens, picture in (([70, 1, 100, 0, 37, 64], 30), ):
        loop.inputs(lens, picture)
        loop.write()
        zp.zp_prompt_attn(loop.q, loop.k, loop.qkv[:, Hq + Hkv:], loop.start, loop.out, loop.p, loop.ws, 100)
        assert zp.zp_read_error(loop.ws) == 0
        loop.check_written(kept)
        loop.check_rows(loop.out, False, 2.0 ** -8)              # over the exact keys and values
        again = torch.zeros_like(loop.out)                        # the bf16 cache holds the same
        zp.zp_paged_window_attn(loop.pool, 0, loop.q, loop.start, loop.tables, loop.cached, again, loop.p, loop.ws, 0, 0, 100)
        loop.check_rows(again, False, 2.0 ** -8)
    for top in (60, 60, 3, 1):                                    # chunks, drafts, single tokens
        loop.inputs(rng.integers(0, top + 1, B))
        loop.write()
        zp.zp_kv8_window_attn(loop.codes, loop.scales, 0, loop.q, loop.start, loop.tables, loop.cached, loop.out, loop.p, loop.ws, 0, 0, top)
        assert zp.zp_read_error(loop.ws) == 0
        loop.check_written(kept)
        loop.check_rows(loop.out, True, 2.0 ** -10)
    # long prompts (the tiled form) beside caches that go on
    loop = Loop(zp, 3, T, 5)
    loop.inputs([300, 5, 110])
    loop.write()
    zp.zp_prompt_attn(loop.q, loop.k, loop.qkv[:, Hq + Hkv:], loop.start, loop.out, loop.p, loop.ws, 300)
    assert zp.zp_read_error(loop.ws) == 0
    loop.check_rows(loop.out, False, 2.0 ** -8)


def test_a_captured_step_of_drafts(zp):
    """One graph of a whole step, replayed: what it accepts is decided on the device, and the next replay goes on from there."""
    B, T, most = 5, 24, 4
    loop, rng = Loop(zp, B, T, 3), np.random.default_rng(4)
    loop.ahead.copy_(_i32([0, 7, 0, 1000, 0]))                    # two requests have been compressed
    loop.inputs([most] * B)
    step = lambda: (loop.write(), zp.zp_kv8_window_attn(loop.codes, loop.scales, 0, loop.q, loop.start, loop.tables, loop.cached, loop.out,
                                                        loop.p, loop.ws, 0, 0, most))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()                                                    # once as it is: every kernel is loaded
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    assert loop.cached.tolist() == [most] * B and loop.at.item() == B
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    assert loop.cached.tolist() == [most] * B
    L = [most] * B
    for _ in range(12):
        # some drafts are taken back, never those that began a block
        taken = [min(int(rng.integers(0, 3)), (n - 1) % b) for n in L]
        loop.cached.sub_(_i32(taken))
        L = [n - t for n, t in zip(L, taken)]
        new = rng.integers(0, most + 1, B)
        loop.inputs(new)
        graph.replay()
        L = [n + int(m) for n, m in zip(L, new)]
        assert loop.cached.tolist() == L and zp.zp_read_error(loop.ws) == 0
        start = np.concatenate([[0], np.cumsum(new)])
        pos = loop.pos.tolist()
        for r in range(B):
            first = L[r] - int(new[r]) + loop.ahead[r].item()
            assert pos[start[r]:start[r + 1]] == list(range(first, first + int(new[r])))
        assert loop.start.tolist() == start.tolist() and loop.slots[int(start[-1]):].tolist() == [-1] * (T - int(start[-1]))
        loop.check_rows(loop.out, True, 2.0 ** -10)
    assert loop.at.item() == sum(-(-n // b) for n in L)


def test_a_step_that_does_not_fit_writes_nothing(zp):
    """Too few free blocks: the operators behind it on the stream find a step without tokens."""
    loop = Loop(zp, 4, 60, 7)
    loop.inputs([20, 3, 17, 9])
    loop.write()
    assert zp.zp_read_error(loop.ws) == 0
    loop.at.fill_(loop.NB - 1)
    before = (loop.pool.clone(), loop.codes.clone(), loop.scales.clone(), loop.tables.clone(), loop.cached.clone())
    loop.out.fill_(7.0)
    loop.inputs([20, 20, 10, 5])
    loop.write()
    zp.zp_kv8_window_attn(loop.codes, loop.scales, 0, loop.q, loop.start, loop.tables, loop.cached, loop.out, loop.p, loop.ws, 0, 0, 20)
    zp.zp_prompt_attn(loop.q, loop.k, loop.qkv[:, Hq + Hkv:], loop.start, loop.out, loop.p, loop.ws, 20)
    assert zp.zp_read_error(loop.ws) == zp.ZP_ERR_NO_BLOCKS
    for x, y in zip(before, (loop.pool, loop.codes, loop.scales, loop.tables, loop.cached)):
        assert torch.equal(x, y)
    assert loop.start.tolist() == [0] * 5 and loop.at.item() == loop.NB - 1 and bool((loop.out == 7.0).all())
