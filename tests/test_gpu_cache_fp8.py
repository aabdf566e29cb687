"""8-bit cache rows on the GPU against their definition, bit by bit."""
import numpy as np
import pytest
import torch

import oracle as O

pytestmark = pytest.mark.gpu
E4M3 = torch.float8_e4m3fn
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def F():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import kv_cache_attention_fdllm_b200 as F
    return F


def _rows(B, R, H, dh, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(B, R, H, dh, generator=g) * torch.exp(2 * torch.randn(B, R, H, 1, generator=g))
    return x.to(DT[dtype])


def _empty_cache(B, N, H, dh, seed=5):
    g = torch.Generator().manual_seed(seed)
    c = torch.randint(0, 120, (B, H, N, dh), generator=g, dtype=torch.uint8)
    s = torch.rand(B, H, N, generator=g)
    return c.cuda().view(E4M3), s.cuda()


def _bits(t):
    return t.view(torch.uint8).cpu().numpy()


def _check_write(F, k, v, pos, N, stream=None):
    B, R, H, dh = k.shape
    kc, ks = _empty_cache(B, N, H, dh, 5)
    vc, vs = _empty_cache(B, N, H, dh, 6)
    before = [_bits(kc).copy(), ks.cpu().numpy().copy(), _bits(vc).copy(), vs.cpu().numpy().copy()]
    ws = F.alloc_workspace(F.fdllm_cache_fp8_workspace_bytes(B, R), "cuda")
    F.fdllm_cache_write_fp8(k.cuda(), v.cuda(), pos.cuda(), kc, vc, ks, vs, ws, stream=stream)
    torch.cuda.synchronize()
    for x, cache, scale, c0, s0 in ((k, kc, ks, before[0], before[1]), (v, vc, vs, before[2], before[3])):
        want_v, want_s = O.e4m3_to_f64(c0), s0.copy()
        q, sc = O.quantise_rows(O.to_f64(x))
        for b in range(B):
            for r in range(R):                 # in order: the last row of a slot stays
                p = int(pos[b, r])
                if 0 <= p < N:
                    want_v[b, :, p] = q[b, r]
                    want_s[b, :, p] = sc[b, r]
        np.testing.assert_array_equal(O.e4m3_to_f64(_bits(cache)), want_v)
        np.testing.assert_array_equal(scale.cpu().numpy(), want_s)
    return ws


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,N,H,dh,R", [(1, 1, 1, 64, 1), (1, 33, 1, 128, 7), (3, 50, 5, 64, 17),
                                        (2, 300, 32, 128, 41), (2, 97, 3, 128, 97), (1, 2000, 2, 64, 1500)])
def test_write(F, B, N, H, dh, R, dtype):
    g = np.random.default_rng(R)
    pos = torch.from_numpy(np.stack([g.permutation(N)[:R] for _ in range(B)]).astype(np.int32))
    _check_write(F, _rows(B, R, H, dh, dtype, R), _rows(B, R, H, dh, dtype, R + 1), pos, N)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_write_special_rows(F, dtype):
    """Zeros, denormals, the type's largest and smallest values, infinities, NaN."""
    B, R, H, dh = 1, 9, 2, 64
    x = _rows(B, R, H, dh, "f32", 3)
    x[0, 0] = 0
    x[0, 1] = 1e-39
    x[0, 2, :, ::2] = torch.finfo(DT[dtype]).max
    x[0, 3, :, 5] = float("inf")
    x[0, 4, :, 6] = float("nan")
    x[0, 5] = float("nan")
    x[0, 6] = -float("inf")
    x[0, 7] = 2.0 ** -97
    x[0, 8] = -0.0
    x = x.to(DT[dtype])
    _check_write(F, x, x.flip(1).contiguous(), torch.arange(R, dtype=torch.int32)[None], R + 1)


@pytest.mark.parametrize("R", [5, 40, 300, 2500])
def test_write_repeated_slots_and_padding(F, R):
    """Rows of one slot: the last is kept, data and scale from the same row; -1 is skipped."""
    B, N, H, dh = 2, 60, 3, 64
    g = np.random.default_rng(R)
    pos = torch.from_numpy(g.integers(-1, N, (B, R)).astype(np.int32))
    ws = _check_write(F, _rows(B, R, H, dh, "bf16", R), _rows(B, R, H, dh, "bf16", R + 1), pos, N)
    assert F.fdllm_get_status(ws) == F.OK


def test_write_bad_slots(F):
    B, N, H, dh, R = 2, 16, 2, 64, 6
    pos = torch.tensor([[0, 16, 3, -2, 2 ** 31 - 1, 5], [-2 ** 31, 1, 2, 3, 4, 15]], dtype=torch.int32)
    ws = _check_write(F, _rows(B, R, H, dh, "bf16", 1), _rows(B, R, H, dh, "bf16", 2), pos, N)
    assert F.fdllm_get_status(ws) == F.ERR_BAD_INDEX
    assert F.fdllm_get_status(ws) == F.OK


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,N,H,dh,R", [(1, 1, 1, 64, 1), (2, 40, 3, 128, 90), (3, 300, 8, 64, 33),
                                        (1, 1500, 2, 128, 1500)])
def test_read(F, B, N, H, dh, R, dtype):
    kc, ks = _empty_cache(B, N, H, dh, 7)
    vc, vs = _empty_cache(B, N, H, dh, 8)
    g = np.random.default_rng(R)
    pos = torch.from_numpy(g.integers(-1, N, (B, R)).astype(np.int32))
    rows = [torch.full((B, R, H, dh), 7.0, dtype=DT[dtype], device="cuda") for _ in range(2)]
    ws = F.alloc_workspace(F.fdllm_cache_fp8_workspace_bytes(B, R), "cuda")
    F.fdllm_cache_read_fp8(pos.cuda(), kc, vc, ks, vs, rows[0], rows[1], ws)
    assert F.fdllm_get_status(ws) == F.OK
    for got, cache, scale in ((rows[0], kc, ks), (rows[1], vc, vs)):
        val = O.e4m3_to_f64(_bits(cache)).astype(np.float32) * scale.cpu().numpy()[..., None]
        want = np.full((B, R, H, dh), 7.0)
        for b in range(B):
            for r in range(R):
                if pos[b, r] >= 0:
                    want[b, r] = O.round_to(val[b, :, int(pos[b, r])].astype(np.float64), dtype)
        np.testing.assert_array_equal(O.to_f64(got.cpu()), want)


def test_read_bad_slots(F):
    kc, ks = _empty_cache(1, 8, 2, 64)
    rows = [torch.full((1, 3, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    ws = F.alloc_workspace(256, "cuda")
    pos = torch.tensor([[8, -7, 2]], dtype=torch.int32, device="cuda")
    F.fdllm_cache_read_fp8(pos, kc, kc, ks, ks, rows[0], rows[1], ws)
    assert F.fdllm_get_status(ws) == F.ERR_BAD_INDEX
    assert (rows[0][0, :2] == 7).all() and not (rows[0][0, 2] == 7).all()


def test_write_on_another_stream(F):
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    pos = torch.arange(40, dtype=torch.int32).repeat(2, 1)
    _check_write(F, _rows(2, 40, 4, 128, "bf16", 1), _rows(2, 40, 4, 128, "bf16", 2), pos, 64, stream=s)


def test_offsets_past_32_bits(F):
    """A cache of over 2^32 bytes: the last slots of the last head."""
    B, N, H, dh = 1, 270336, 128, 128
    kc = torch.zeros((B, H, N, dh), dtype=torch.uint8, device="cuda").view(E4M3)
    ks = torch.zeros((B, H, N), device="cuda")
    assert kc.numel() > 2 ** 32
    k = _rows(B, 2, H, dh, "bf16", 4)
    pos = torch.tensor([[N - 1, N - 2]], dtype=torch.int32, device="cuda")
    ws = F.alloc_workspace(256, "cuda")
    vc, vs = torch.zeros_like(kc.view(torch.uint8)).view(E4M3), torch.zeros_like(ks)
    F.fdllm_cache_write_fp8(k.cuda(), k.cuda(), pos, kc, vc, ks, vs, ws)
    q, sc = O.quantise_rows(O.to_f64(k))
    got = O.e4m3_to_f64(_bits(kc[:, :, N - 2:].contiguous()))
    np.testing.assert_array_equal(got[0, :, 1], q[0, 0])
    np.testing.assert_array_equal(got[0, :, 0], q[0, 1])
    np.testing.assert_array_equal(ks[0, :, N - 1].cpu().numpy(), sc[0, 0])
    back = [torch.empty_like(k, device="cuda") for _ in range(2)]
    F.fdllm_cache_read_fp8(pos, kc, vc, ks, vs, back[0], back[1], ws)
    want = O.round_bf16((q.astype(np.float32) * sc[..., None]).astype(np.float64))
    np.testing.assert_array_equal(O.to_f64(back[0].cpu()), want)
    np.testing.assert_array_equal(O.to_f64(back[1].cpu()), want)
