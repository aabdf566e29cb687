"""One attention call that runs for seconds: the limit on waits counts from when a CTA stands
still, not from when its range began."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def F():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import kv_cache_attention_fdllm_b200 as F
    return F


def test_a_call_of_several_seconds(F):
    """256 nodes of 64 heads to a kv head over 1.7 million slots of 64 kv heads, 14 GB in 8
    bits: every tile is read for 512 chunks of rows, some 3 million tiles a CTA.

    K is zero, so that a row's output is the mean of V, and V is one value a head.  A sum of
    equal products in fp32 is off by at most one step, 2^-23, an addition: 4 a tile."""
    N, Hkv, g, dh, T = 1_700_000, 64, 64, 64, 256
    free, _ = torch.cuda.mem_get_info()
    assert free > 20 * 2 ** 30
    value = (1.0 + torch.arange(Hkv, device="cuda") % 8 / 8).to(torch.float8_e4m3fn)
    k = torch.zeros((1, Hkv, N, dh), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    v = torch.empty((1, Hkv, N, dh), dtype=torch.float8_e4m3fn, device="cuda")
    v.view(torch.uint8)[:] = value.view(torch.uint8)[None, :, None, None]
    ones = torch.ones((1, Hkv, N), device="cuda")
    q = torch.randn((1, T, Hkv * g, dh), device="cuda").to(torch.bfloat16)
    lens = torch.tensor([N - T], dtype=torch.int32, device="cuda")
    out = torch.empty((1, T, Hkv * g * dh), dtype=torch.bfloat16, device="cuda")
    ws = F.alloc_workspace(F.fdllm_tree_attend_workspace_bytes(1, N, Hkv * g, Hkv, dh, T, torch.bfloat16), "cuda")
    for _ in range(2):  # the second with what the first left in the workspace
        out.zero_()
        F.fdllm_tree_attend_fp8(q, k, v, ones, ones, lens, None, None, out, ws)
        assert F.fdllm_get_status(ws) == F.OK
        want = value.float()[None, None, :, None, None]
        err = (out.reshape(1, T, Hkv, g, dh).float() / want - 1).abs().max().item()
        assert err <= 4 * ((N + 127) // 128) * 2.0 ** -23 + 2.0 ** -8, err
