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
