"""The compiled part of the binding: when it is loaded, and what it refuses."""
import os
import shutil
import subprocess
import sys

import pytest
import torch


@pytest.fixture(scope="module")
def zp():
    from paged_kv_cache_obs_gb300 import build
    if not os.path.exists(build.LIB):
        build.build()
    from paged_kv_cache_obs_gb300 import zipage
    return zipage


def test_calls_that_do_not_need_the_compiled_part_run_without_it(zp, tmp_path):
    """A package whose lib/ holds libzipage.so alone: it imports, the allocator works, and a per-step
    operator says what is missing."""
    package = os.path.dirname(os.path.abspath(zp.__file__))
    copy = tmp_path / os.path.basename(package)
    shutil.copytree(package, copy, ignore=shutil.ignore_patterns("lib", "__pycache__", "csrc"))
    (copy / "lib").mkdir()
    shutil.copy(os.path.join(package, "lib", "libzipage.so"), copy / "lib")
    code = """
import torch
from paged_kv_cache_obs_gb300 import zipage as z
a = z.zp_alloc_create(4)
assert len(z.zp_alloc_blocks(a, 2)) == 2
z.zp_alloc_destroy(a)
rope = z.zp_rope_init(64, 64, 1e4)
try:
    z.zp_rope_apply(rope, torch.zeros((1, 1, 64), dtype=torch.bfloat16), None, torch.zeros(1, dtype=torch.int32))
except ImportError as e:
    assert "zp_tensors.so is not built" in str(e)
else:
    raise AssertionError("ran without its binding")
"""
    res = subprocess.run([sys.executable, "-c", code], cwd=tmp_path, capture_output=True, text=True,
                         env={**os.environ, "PYTHONPATH": str(tmp_path)})
    assert res.returncode == 0, res.stderr


def _host_args():
    bf = torch.zeros((4, 2, 64), dtype=torch.bfloat16)
    codes, scales = torch.zeros((1, 4, 2, 2, 16, 64), dtype=torch.uint8), torch.zeros((1, 4, 2, 2))
    p = dict(num_layers=1, num_q_heads=2, num_kv_heads=2, head_dim=64, block_size=16, n_max=8, window=1, alpha=0.5, beta=0.5,
             decay=0.9, scale=0.125, protect_window=1, causal=1)
    return bf, codes, scales, torch.zeros((4, 6), dtype=torch.int32), p, torch.zeros(1024, dtype=torch.uint8)


def test_index_tensors_hold_one_number_an_entry(zp):
    """Positions, lengths and block ids with further dimensions (above 1) hold more numbers than the library would read."""
    bf, codes, scales, tables, p, ws = _host_args()
    pool = torch.zeros(codes.shape, dtype=torch.bfloat16)
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)
    rope = zp.zp_rope_init(64, 64, 1e4)
    for call in (lambda: zp.zp_rope_apply(rope, bf, None, i32(4, 2)),
                 lambda: zp.zp_kv8_append(codes, scales, 0, bf, bf, i32(5, 2), i32(4), tables, p, ws),
                 lambda: zp.zp_kv8_append(codes, scales, 0, bf, bf, i32(5), i32(4, 3), tables, p, ws),
                 lambda: zp.zp_kv8_append(codes, scales, 0, bf, bf, i32(5), i32(4), i32(4, 6, 2), p, ws),
                 lambda: zp.zp_kv8_decode_attn(codes, scales, 0, bf, tables, i32(4, 2), bf, p, ws),
                 lambda: zp.zp_paged_window_attn(pool, 0, bf, i32(5), tables, i32(4, 2), bf, p, ws, 4, 1, 1),
                 lambda: zp.zp_paged_window_attn(pool, 0, bf, i32(5, 2), tables, i32(4), bf, p, ws, 4, 1, 1),
                 lambda: zp.zp_kv8_pack_blocks(pool, i32(4, 2), codes, scales, i32(4), p, ws),
                 lambda: zp.zp_kv8_pack_blocks(pool, i32(4), codes, scales, i32(4), p, ws, fill=i32(4, 2)),
                 lambda: zp.zp_kv8_unpack_blocks(codes, scales, i32(4), pool, i32(4, 2), p, ws)):
        with pytest.raises(ValueError, match="expected"):
            call()
    # a column is as good as a row of numbers
    for call in (lambda: zp.zp_rope_apply(rope, bf, None, i32(4, 1)),
                 lambda: zp.zp_kv8_append(codes, scales, 0, bf, bf, i32(5, 1), i32(4), tables, p, ws)):
        with pytest.raises(ValueError, match="current CUDA device"):
            call()


def test_codes_are_e4m3(zp):
    """Other types of one byte would be read as E4M3 and written with its codes."""
    bf, codes, scales, tables, p, ws = _host_args()
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)
    call = lambda c: zp.zp_kv8_append(c, scales, 0, bf, bf, i32(5), i32(4), tables, p, ws)
    for t in (torch.float8_e5m2, torch.float8_e4m3fnuz, torch.float8_e5m2fnuz, torch.bool):
        with pytest.raises(ValueError, match="E4M3"):
            call(codes.view(t))
    for t in (torch.uint8, torch.int8, torch.float8_e4m3fn):
        with pytest.raises(ValueError, match="current CUDA device"):
            call(codes.view(t))


def test_rows_that_are_written_do_not_overlap(zp):
    """Broadcast or overlapping rows are refused where a call writes them: on the host, before any launch."""
    ws = torch.zeros(1 << 16, dtype=torch.uint8)
    base = (ws.data_ptr() + 255) // 256 * 256
    _, _, _, _, p, _ = _host_args()
    params, bad = zp.make_params(p), zp.ZP_ERR_INVALID_ARG
    rope = zp.zp_rope_init(64, 64, 1e4)
    good, rows = zp.zp_rows(base, 128, 64), lambda t, h: zp.zp_rows(base, t, h)
    apply = lambda q, qo, T=2, H=2: zp.lib.zp_rope_apply(rope, q, qo, H, None, None, 0, base, T, None)
    for T, H, t, h in ((2, 1, 0, 64), (2, 1, 32, 64), (2, 2, 128, 0), (2, 2, 128, 63), (2, 2, 0, 64), (2, 2, -8, 64)):
        r = rows(t, h)
        assert apply(r, r, T, H) == bad and apply(good, r, T, H) == bad            # in place, and as a result
        params.num_q_heads, params.num_kv_heads = H, 1
        pool8, pool = zp.zp_kv8_pool(base, base, 4), zp.zp_kv_pool(base, 4)
        assert zp.lib.zp_kv8_decode_attn(pool8, 0, good, base, base, T, 2, 0, 0, r, params, base, 1 << 40, None) == bad
        for mq in (1, 40):
            assert zp.lib.zp_paged_window_attn(pool, 0, good, base, T, mq, base, base, 1, 2, 0, 0, r, params, base, 1 << 40, None) == bad


@pytest.mark.gpu
def test_rows_that_are_read_may_be_broadcast(zp):
    x = torch.randn((1, 1, 64), device="cuda").to(torch.bfloat16)
    pos = torch.arange(5, dtype=torch.int32, device="cuda")
    rope = zp.zp_rope_init(64, 64, 1e4)
    a, b = (torch.zeros((5, 3, 64), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    zp.zp_rope_apply(rope, x.expand(5, 3, 64), None, pos, q_out=a)
    zp.zp_rope_apply(rope, x.expand(5, 3, 64).contiguous(), None, pos, q_out=b)
    assert torch.equal(a, b) and bool((a != 0).any())
    # one row of one head has no second one to overlap
    zp.zp_rope_apply(rope, x, None, pos[:1], q_out=torch.empty(64, dtype=torch.bfloat16, device="cuda").as_strided((1, 1, 64), (0, 0, 1)))
