"""CPU checks of the calls for drafted tokens: the C ABI's refusals before anything is
launched, the binding's checks, and pins of their fp64 oracle."""
import ctypes

import numpy as np
import pytest
import torch

import oracle as O

FAKE = ctypes.c_void_p(1 << 20)  # aligned, never dereferenced
ODD = ctypes.c_void_p((1 << 20) + 4)
BIG = 1 << 40
INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 6


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    __graft_entry__.build()
    from kv_cache_attention_fdllm_b200 import _native
    return _native.lib()


@pytest.mark.parametrize("name", ["fdllm_cache_write_fp8", "fdllm_cache_read_fp8"])
def test_cache_rows_refusals(lib, name):
    f = getattr(lib, name)

    def call(B=2, N=100, H=4, dh=128, R=3, dtype=1, ptrs=None, ws=FAKE, wsb=256):
        return f(B, N, H, dh, R, dtype, *(ptrs or [FAKE] * 7), ws, wsb, None)

    assert call(B=-1) == INVALID and call(N=0) == INVALID and call(H=0) == INVALID
    assert call(R=-1) == INVALID
    assert call(dh=96) == UNSUPPORTED and call(dtype=2) == UNSUPPORTED
    assert call(B=1 << 20, R=1 << 12) == UNSUPPORTED     # more rows than 32 bits count
    assert call(ws=None) == WORKSPACE and call(wsb=255) == WORKSPACE and call(ws=ODD) == WORKSPACE
    for i in range(7):
        for bad in (None, ODD):
            assert call(ptrs=[bad if i == j else FAKE for j in range(7)]) == INVALID
    assert call(B=0, ptrs=[None] * 7) == 0 and call(R=0, ptrs=[None] * 7) == 0
    assert lib.fdllm_cache_fp8_workspace_bytes(2, 3) == 256
    assert lib.fdllm_cache_fp8_workspace_bytes(-1, 3) == 0


@pytest.mark.parametrize("fp8", [False, True])
def test_tree_attend_refusals(lib, fp8):
    f = lib.fdllm_tree_attend_fp8 if fp8 else lib.fdllm_tree_attend
    n_ptr = 8 if fp8 else 6  # q, k, v, (scales), cache_len, parent, n_nodes, out

    def call(B=2, N=500, Hq=8, Hkv=2, dh=128, T=5, dtype=1, ptrs=None, ws=FAKE, wsb=BIG):
        return f(B, N, Hq, Hkv, dh, T, dtype, *(ptrs or [FAKE] * (n_ptr + 1)), ws, wsb, None)

    assert call(B=-1) == INVALID and call(N=0) == INVALID and call(T=-1) == INVALID
    assert call(Hkv=0) == INVALID and call(Hq=1) == INVALID and call(Hq=7) == INVALID
    assert call(dh=256) == UNSUPPORTED and call(dtype=3) == UNSUPPORTED
    assert call(T=257) == UNSUPPORTED and call(B=1025) == UNSUPPORTED
    assert call(Hq=130) == UNSUPPORTED                   # 65 query heads to a kv head
    if fp8:
        assert call(dtype=0) == UNSUPPORTED
    need = lib.fdllm_tree_attend_workspace_bytes(2, 500, 8, 2, 128, 5, 1)
    assert need >= 256
    assert call(wsb=need - 1) == WORKSPACE and call(ws=None) == WORKSPACE
    optional = (n_ptr - 2, n_ptr - 1)                    # parent, n_nodes
    for i in range(n_ptr + 1):
        assert call(ptrs=[ODD if i == j else FAKE for j in range(n_ptr + 1)]) == INVALID
        if i not in optional:
            assert call(ptrs=[None if i == j else FAKE for j in range(n_ptr + 1)]) == INVALID
    none = [None] * (n_ptr + 1)
    assert call(B=0, ptrs=none) == 0 and call(T=0, ptrs=none) == 0
    assert lib.fdllm_tree_attend_workspace_bytes(2, 500, 8, 3, 128, 5, 1) == 0


def test_tree_workspace_serves_smaller_calls(lib):
    w = lib.fdllm_tree_attend_workspace_bytes
    prev = 0
    for T in range(1, 257):
        now = w(8, 4096, 32, 8, 128, T, 1)
        assert now >= prev
        prev = now
    prev = 0
    for B in range(1, 300):
        now = w(B, 4096, 32, 8, 128, 40, 1)
        assert now >= prev
        prev = now


def test_draft_verify_refusals(lib):
    need = lib.fdllm_draft_verify_workspace_bytes(2, 3, 1000)
    assert need > 256
    c = lib.fdllm_chain_verify

    def chain(B=2, T=3, V=1000, ptrs=None, ws=FAKE, wsb=need):
        return c(B, T, V, *(ptrs or [FAKE] * 8), ws, wsb, None)

    assert chain(B=-1) == INVALID and chain(T=-1) == INVALID and chain(V=0) == INVALID
    assert chain(T=1025) == UNSUPPORTED and chain(B=16385) == UNSUPPORTED
    assert chain(wsb=need - 1) == WORKSPACE and chain(ws=ODD) == WORKSPACE
    for i in range(8):
        assert chain(ptrs=[ODD if i == j else FAKE for j in range(8)]) == INVALID
        if i != 3:  # n_draft may be missing
            assert chain(ptrs=[None if i == j else FAKE for j in range(8)]) == INVALID
    assert chain(B=0, ptrs=[None] * 8) == 0
    t = lib.fdllm_tree_verify

    def tree(B=2, T=3, V=1000, ptrs=None, ws=FAKE, wsb=need):
        return t(B, T, V, *(ptrs or [FAKE] * 9), ws, wsb, None)

    assert tree(T=0) == INVALID and tree(T=257) == UNSUPPORTED and tree(V=0) == INVALID
    assert tree(wsb=need - 1) == WORKSPACE
    for i in range(9):
        assert tree(ptrs=[ODD if i == j else FAKE for j in range(9)]) == INVALID
        if i != 3:  # n_nodes may be missing
            assert tree(ptrs=[None if i == j else FAKE for j in range(9)]) == INVALID
    assert lib.fdllm_draft_verify_workspace_bytes(2, 1025, 1000) == 0


def test_binding_refuses_cpu_tensors(lib):
    import kv_cache_attention_fdllm_b200 as F
    z = torch.zeros
    with pytest.raises(ValueError, match="CUDA"):
        F.fdllm_tree_attend(z(1, 1, 2, 64), z(1, 2, 8, 64), z(1, 2, 8, 64), z(1), None, None,
                            z(1, 1, 128), z(256))
    with pytest.raises(ValueError, match="CUDA"):
        F.fdllm_chain_verify(z(1, 2, 8), z(1, 1, 8), z(1, 1), None, z(1, 1), z(1), z(1), z(1), z(256))
    with pytest.raises(ValueError, match="CUDA"):
        F.fdllm_cache_write_fp8(z(1, 1, 2, 64), z(1, 1, 2, 64), z(1, 1), z(1, 2, 8, 64),
                                z(1, 2, 8, 64), z(1, 2, 8), z(1, 2, 8), z(256))


# ------------------------------------------------------------------ the oracle's pins


def test_e4m3_is_torchs():
    """Every byte's value, and rounding at random, at every tie and past the ends."""
    bits = np.arange(256, dtype=np.uint8)
    want = torch.from_numpy(bits).view(torch.float8_e4m3fn).float().numpy()
    np.testing.assert_array_equal(O.e4m3_to_f64(bits), want)
    vals = np.sort(want[np.isfinite(want)].astype(np.float64))
    ties = (vals[1:] + vals[:-1]) / 2
    x = np.concatenate([vals, ties, np.nextafter(ties, 1e9), np.nextafter(ties, -1e9),
                        np.random.default_rng(0).standard_normal(4000) * 60, [1e-9, 449.0, 1e9]])
    x = x.astype(np.float32).astype(np.float64)
    t = torch.from_numpy(x.astype(np.float32)).clamp(-448, 448).to(torch.float8_e4m3fn)
    np.testing.assert_array_equal(O.round_e4m3(x), t.float().numpy())


def test_quantised_rows():
    x = np.random.default_rng(1).standard_normal((50, 64)).astype(np.float32)
    q, s = O.quantise_rows(x)
    np.testing.assert_array_equal(np.abs(q).max(-1), 448.0)
    # a rounding is off by half a step: 2^-4 of the value, or half the subnormal step 2^-9
    err = np.abs(q * s[:, None].astype(np.float64) - x)
    assert (err <= 2.0 ** -4 * np.abs(x) * (1 + 1e-6) + 2.0 ** -10 * s[:, None] * (1 + 1e-6)).all()
    z, s0 = O.quantise_rows(np.zeros((1, 64)))
    assert (z == 0).all() and s0[0] > 0
    one = np.zeros((1, 64), np.float32)
    one[0, 3], one[0, 5] = np.inf, np.nan
    q, s = O.quantise_rows(one)
    assert q[0, 3] == 448 and np.isnan(q[0, 5]) and np.isfinite(s[0]) and (q[0, 6:] == 0).all()


def test_tree_attention_against_sdpa():
    """A chain is causal attention; a tree's node is its own path run as a sequence."""
    g = np.random.default_rng(2)
    L, T, Hq, Hkv, dh = 9, 6, 4, 2, 16
    q, k, v = g.standard_normal((T, Hq, dh)), g.standard_normal((Hkv, 20, dh)), g.standard_normal((Hkv, 20, dh))
    t64 = lambda a: torch.from_numpy(a)  # noqa: E731
    kk, vv = t64(k).repeat_interleave(2, 0), t64(v).repeat_interleave(2, 0)
    out, _, _ = O.tree_attend(q, k, v, L, None, T)
    mask = torch.ones(T, L + T).tril(L).bool()
    ref = torch.nn.functional.scaled_dot_product_attention(
        t64(q).transpose(0, 1), kk[:, :L + T], vv[:, :L + T], attn_mask=mask)
    np.testing.assert_allclose(out, ref.transpose(0, 1).numpy(), atol=1e-12)
    parent = [-1, 0, 0, 2, 1, -1]
    out, bound, _ = O.tree_attend(q, k, v, L, parent, T)
    assert (np.abs(out) <= bound + 1e-12).all()
    paths = {0: [0], 1: [0, 1], 2: [0, 2], 3: [0, 2, 3], 4: [0, 1, 4], 5: [5]}
    for t, p in paths.items():
        slots = list(range(L)) + [L + j for j in p]
        ref = torch.nn.functional.scaled_dot_product_attention(t64(q[t])[:, None], kk[:, slots], vv[:, slots])
        np.testing.assert_allclose(out[t], ref[:, 0].numpy(), atol=1e-12)


def test_draw():
    w = np.array([0.0, 0.25, 0.0, 0.5, 0.25, 0.0])
    assert [O.draw(w, r) for r in (0.0, 0.2499, 0.25, 0.7499, 0.75, 0.9999)] == [1, 1, 3, 3, 4, 4]
    assert O.draw(np.array([-1.0, np.nan, 2.0]), 0.0) == 2
    assert O.draw(np.zeros(4), 0.3) == -1


def test_chain_keeps_the_targets_distribution():
    """Over all (draft, u, r) of a fine grid, the first token is distributed as the target."""
    p = np.array([[0.5, 0.2, 0.3], [1.0, 0.0, 0.0]], np.float32)
    q = np.array([[0.2, 0.5, 0.3]], np.float32)
    got = np.zeros(3)
    n = 40
    for x in range(3):
        for i in range(n):
            for j in range(n):
                a, t = O.chain_verify(p, q, [x], 1, [(i + 0.5) / n], (j + 0.5) / n)
                got[x if a else t] += q[0, x] / n / n
    np.testing.assert_allclose(got, p[0], atol=0.02)


def test_tree_keeps_the_targets_distribution():
    p = np.array([[0.1, 0.4, 0.3, 0.2]] * 4, np.float32)
    tok, parent = [9, 2, 1, 2], [9, 0, 0, 0]             # node 3 repeats node 1's token
    got = np.zeros(4)
    n = 40
    for i in range(n):
        for j in range(n):
            path, t = O.tree_verify(p, tok, parent, 4, [(i + 0.5) / n] * 4, (j + 0.5) / n)
            assert 3 not in path
            got[tok[path[0]] if path else t] += 1.0 / n / n
    np.testing.assert_allclose(got, p[0], atol=0.02)
