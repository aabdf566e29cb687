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


def test_another_torch_rebuilds_it(tmp_path, monkeypatch):
    """What was built against another torch is built again; what was not, is not."""
    import __graft_entry__
    B = __graft_entry__._build_module()
    assert not B._fast_stale()
    made = open(B.FAST_FOR).read()
    for other in (made.replace(B._torch(), "/elsewhere/torch"), made.replace("__version__ = '", "__version__ = '1"), ""):
        assert other != made
        stamp = tmp_path / "fast_for.txt"
        stamp.write_text(other)
        monkeypatch.setattr(B, "FAST_FOR", str(stamp))
        assert B._fast_stale()
    monkeypatch.setattr(B, "FAST_FOR", str(tmp_path / "none.txt"))
    assert B._fast_stale()


def test_one_of_another_torch_is_not_used():
    """It may load and still read tensors wrongly."""
    rc, out, err = python("""
import sys
import torch
import types
m = types.ModuleType("kv_cache_attention_fdllm_b200._fast")
m.torch_version = "1.0.0"
sys.modules[m.__name__] = m
import kv_cache_attention_fdllm_b200.api as A
print(A._fast)
""")
    assert rc == 0, err
    assert out.strip() == "None" and "torch 1.0.0" in err
