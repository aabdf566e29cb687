"""The binding's short way (_fast.so) is a convenience: without it every call goes through the
checks in Python."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def python(code):
    r = subprocess.run([sys.executable, "-W", "always", "-c", code], cwd=ROOT, capture_output=True, text=True,
                       timeout=300)
    return r.returncode, r.stdout, r.stderr


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


def test_the_package_serves_without_it():
    """Missing, or unfit for the torch that is there: a warning that names what builds it, and
    every call keeps its checks."""
    rc, out, err = python("""
import sys
sys.modules["kv_cache_attention_fdllm_b200._fast"] = None  # importing it raises ImportError
import torch
import kv_cache_attention_fdllm_b200 as F
t = torch.zeros(2, 3, 4, 64)
i = torch.zeros(2, 3, dtype=torch.int32)
for f, n in ((F.fdllm_cache_write_fp8, 8), (F.fdllm_cache_read_fp8, 8), (F.fdllm_tree_attend, 8),
             (F.fdllm_tree_attend_fp8, 10), (F.fdllm_chain_verify, 9), (F.fdllm_tree_verify, 10)):
    for args, error in (([t] * n, ValueError), ([None] * n, TypeError)):
        try:
            f(*args)
        except error as e:
            print(f.__name__, type(e).__name__)
assert F.fdllm_fused_step_workspace_bytes(1, 64, 64, 1, 64, 1, torch.float32) > 0
""")
    assert rc == 0, err
    assert len(out.split()) == 2 * 12
    assert "RuntimeWarning" in err and "kv_cache_attention_fdllm_b200/build.py" in err


def test_it_is_used_where_it_is():
    rc, out, err = python("""
import kv_cache_attention_fdllm_b200.api as A
print(A._fast.__file__)
""")
    assert rc == 0, err
    assert out.strip().endswith("_fast.so") and "RuntimeWarning" not in err
