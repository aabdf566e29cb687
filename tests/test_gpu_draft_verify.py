"""Sampled verification of drafted chains and trees against the fp64 oracle: whole numbers,
equal."""
import numpy as np
import pytest
import torch

import oracle as O

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def F():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import kv_cache_attention_fdllm_b200 as F
    return F


def _probs(g, *shape):
    x = np.exp(2.5 * g.standard_normal(shape))
    return (x / x.sum(-1, keepdims=True)).astype(np.float32)


def _i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, np.int32)).cuda()


def _f32(a):
    return torch.from_numpy(np.ascontiguousarray(a, np.float32)).cuda()


def _workspace(F, B, T, V):
    return F.alloc_workspace(F.fdllm_draft_verify_workspace_bytes(B, T, V), "cuda")


def run_chain(F, target, draft, tok, n, u, r, ws=None, stream=None):
    B, T, V = draft.shape
    ws = _workspace(F, B, T, V) if ws is None else ws
    na, nt = (torch.full((B,), -7, dtype=torch.int32, device="cuda") for _ in range(2))
    F.fdllm_chain_verify(_f32(target), _f32(draft), _i32(tok), None if n is None else _i32(n), _f32(u),
                         _f32(r), na, nt, ws, stream=stream)
    torch.cuda.synchronize()
    return na.cpu().numpy(), nt.cpu().numpy(), ws


def check_chain(F, target, draft, tok, n, u, r, **kw):
    na, nt, ws = run_chain(F, target, draft, tok, n, u, r, **kw)
    B, T, V = draft.shape
    for b in range(B):
        nb = T if n is None else min(max(int(n[b]), 0), T)
        assert (na[b], nt[b]) == O.chain_verify(target[b], draft[b], tok[b], nb, u[b], r[b]), b
    return na, nt, ws


def run_tree(F, target, tok, parent, n, u, r, ws=None):
    B, T, V = target.shape
    ws = _workspace(F, B, T, V) if ws is None else ws
    path = torch.full((B, T), -7, dtype=torch.int32, device="cuda")
    na, nt = (torch.full((B,), -7, dtype=torch.int32, device="cuda") for _ in range(2))
    F.fdllm_tree_verify(_f32(target), _i32(tok), _i32(parent), None if n is None else _i32(n), _f32(u),
                        _f32(r), path, na, nt, ws)
    torch.cuda.synchronize()
    return path.cpu().numpy(), na.cpu().numpy(), nt.cpu().numpy(), ws


def check_tree(F, target, tok, parent, n, u, r, **kw):
    path, na, nt, ws = run_tree(F, target, tok, parent, n, u, r, **kw)
    B, T, V = target.shape
    for b in range(B):
        nb = T if n is None else min(max(int(n[b]), 1), T)
        p, t = O.tree_verify(target[b], tok[b], parent[b], nb, u[b], r[b])
        assert na[b] == len(p) and path[b].tolist() == p + [-1] * (T - len(p)) and nt[b] == t, b
    return path, na, nt, ws


def chain_case(B, T, V, seed):
    g = np.random.default_rng(seed)
    target = _probs(g, B, T + 1, V)
    draft = target[:, :T] * np.exp(0.7 * g.standard_normal((B, T, V))).astype(np.float32)
    draft = (draft / draft.sum(-1, keepdims=True)).astype(np.float32)
    tok = np.zeros((B, T), np.int64)
    for b in range(B):
        for t in range(T):
            tok[b, t] = g.choice(V, p=draft[b, t].astype(np.float64) / draft[b, t].astype(np.float64).sum())
    return target, draft, tok, g.random((B, T), np.float32), g.random(B, np.float32)


def tree_case(B, T, V, seed, width=5):
    g = np.random.default_rng(seed)
    target = _probs(g, B, T, V)
    parent = np.stack([[-1] + [int(g.integers(max(0, t - width), t)) for t in range(1, T)] for _ in range(B)])
    tok = np.zeros((B, T), np.int64)
    for b in range(B):
        for t in range(1, T):
            best = np.argsort(-target[b, parent[b, t]])[:6]
            tok[b, t] = g.choice(best)          # siblings often repeat a token
    return target, tok, parent, (0.5 * g.random((B, T))).astype(np.float32), g.random(B, np.float32)


@pytest.mark.parametrize("B,T,V", [(1, 1, 1), (2, 1, 2), (3, 4, 5), (5, 3, 1023), (4, 7, 1025), (2, 16, 4099),
                                   (64, 4, 3000), (3, 300, 64), (1, 5, 126464), (7, 2, 50001)])
def test_chain(F, B, T, V):
    for seed in range(3):
        c = chain_case(B, T, V, seed)
        check_chain(F, c[0], c[1], c[2], None, c[3], c[4])


@pytest.mark.parametrize("B,T,V", [(1, 1, 1), (2, 1, 700), (3, 5, 9), (4, 40, 1025), (3, 64, 3001),
                                   (2, 256, 200), (64, 8, 2000), (1, 30, 126464)])
def test_tree(F, B, T, V):
    for seed in range(3):
        c = tree_case(B, T, V, seed)
        check_tree(F, c[0], c[1], c[2], None, c[3], c[4])


def test_ragged_counts(F):
    c = chain_case(6, 9, 2000, 1)
    n = np.array([0, 1, 9, 4, 8, 0])
    u = np.zeros_like(c[3])                      # everything offered is accepted
    na, nt, ws = check_chain(F, c[0], c[1], c[2], n, u, c[4])
    assert na.tolist() == n.tolist() and F.fdllm_get_status(ws) == F.OK
    c = tree_case(5, 20, 2000, 1)
    check_tree(F, c[0], c[1], c[2], np.array([1, 2, 20, 7, 13]), c[3], c[4])


def test_counts_out_of_range(F):
    c = chain_case(2, 3, 50, 1)
    _, _, ws = check_chain(F, c[0], c[1], c[2], np.array([4, -1]), c[3], c[4])
    assert F.fdllm_get_status(ws) == F.ERR_BAD_INDEX
    c = tree_case(2, 4, 50, 1)
    *_, ws = check_tree(F, c[0], c[1], c[2], np.array([0, 5]), c[3], c[4])
    assert F.fdllm_get_status(ws) == F.ERR_BAD_INDEX


def test_tokens_and_parents_out_of_range(F):
    c = list(chain_case(2, 4, 50, 2))
    c[2][0, 2], c[2][1, 0] = 50, -1
    c[3][:] = 0
    na, _, ws = check_chain(F, c[0], c[1], c[2], None, c[3], c[4])
    assert na.tolist() == [2, 0] and F.fdllm_get_status(ws) == F.ERR_BAD_INDEX
    c = list(tree_case(3, 12, 50, 2))
    c[1][0, 3], c[2][1, 4], c[2][2, 2] = 50, 4, -1
    *_, ws = check_tree(F, c[0], c[1], c[2], None, c[3], c[4])
    assert F.fdllm_get_status(ws) == F.ERR_BAD_INDEX


def test_no_drafts_at_all(F):
    """T = 0: the next token from the target's only row."""
    g = np.random.default_rng(0)
    p = _probs(g, 3, 1, 500)
    r = g.random(3, np.float32)
    na, nt, _ = run_chain(F, p, np.zeros((3, 0, 500), np.float32), np.zeros((3, 0)), None, np.zeros((3, 0)), r)
    assert na.tolist() == [0, 0, 0]
    assert nt.tolist() == [O.draw(p[b, 0].astype(np.float64), float(r[b])) for b in range(3)]


def test_empty_weights(F):
    """Draft and target alike and a refused draft: the target's row; nothing at all: -1."""
    V = 3000
    p = np.zeros((4, 2, V), np.float32)
    p[:, :, 10], p[:, :, 2990] = 0.25, 0.75
    q = p[:, :1].copy()
    p[2, 0], q[3, 0] = 0, 1                       # no target at all; a draft above the target everywhere
    tok = np.full((4, 1), 20)                     # a token with no probability is not accepted
    u = np.full((4, 1), 0.5, np.float32)
    r = np.array([0.1, 0.9, 0.5, 0.9], np.float32)
    na, nt, _ = check_chain(F, p, q, tok, None, u, r)
    assert na.tolist() == [0] * 4 and nt.tolist() == [10, 2990, -1, 2990]
    # a tree whose children hold all there is, and are not taken (u = 1)
    t = np.zeros((1, 3, V), np.float32)
    t[0, 0, 5], t[0, 0, 7] = 0.5, 0.5
    path, na, nt, _ = check_tree(F, t, np.array([[0, 5, 7]]), np.array([[-1, 0, 0]]), None,
                                 np.ones((1, 3), np.float32), np.array([0.7], np.float32))
    assert na[0] == 0 and nt[0] == 7


def test_nan_inf_and_negative_weights(F):
    V = 2100
    g = np.random.default_rng(3)
    p, q = _probs(g, 2, 2, V), _probs(g, 2, 1, V)
    p[0, :, 5], p[0, :, 1100], q[0, 0, 7] = np.nan, -3.0, np.nan
    tok = np.array([[5], [7]])                    # a NaN target is not accepted
    u, r = np.full((2, 1), 0.99, np.float32), np.array([0.3, 0.999], np.float32)
    na, nt, _ = check_chain(F, p, q, tok, None, u, r)
    assert na[0] == 0
    p[1, :, 9] = np.inf                           # whatever comes, it is a token of the row
    _, nt, _ = run_chain(F, p, q, tok, None, u, r)
    assert 0 <= nt[1] < V


def test_borders(F):
    """u q exactly equal to p is not accepted, one ulp less is; r at the ends of a step."""
    V = 1500
    p = np.zeros((3, 2, V), np.float32)
    p[:, :, 4], p[:, :, 1400] = 0.5, 0.5
    q = np.zeros((3, 1, V), np.float32)
    q[:, 0, 4] = 1.0
    u = np.array([[0.5], [np.nextafter(np.float32(0.5), np.float32(0))], [0.5]], np.float32)
    r = np.array([0.0, 0.5, np.float32(1 - 2 ** -24)], np.float32)
    na, nt, _ = check_chain(F, p, q, np.full((3, 1), 4), None, u, r)
    assert na.tolist() == [0, 1, 0] and nt.tolist() == [1400, 1400, 1400]
    _, nt, _ = run_chain(F, p, q, np.full((3, 1), 4), None, u, np.array([1.0, 2.0, np.nan], np.float32))
    assert ((0 <= nt) & (nt < V)).all()           # numbers outside [0, 1) still name a token


def test_workspace_of_many_shapes(F):
    """One workspace, sized for the largest, serves calls of every shape in turn, twice."""
    shapes = [(8, 3, 5000), (1, 2, 126464), (64, 2, 1000), (3, 4, 40000)]
    ws = max((_workspace(F, *s) for s in shapes), key=lambda w: w.numel())
    for _ in range(2):
        for s in shapes:
            c = chain_case(*s, seed=s[0])
            check_chain(F, c[0], c[1], c[2], None, c[3], c[4], ws=ws)
            c = tree_case(*s, seed=s[0])
            check_tree(F, c[0], c[1], c[2], None, c[3], c[4], ws=ws)


def test_captured_and_replayed(F):
    """A graph of the call, replayed with other numbers in the same tensors."""
    B, T, V = 4, 6, 30000
    cases = [chain_case(B, T, V, s) for s in range(3)]
    t = [_f32(cases[0][0]), _f32(cases[0][1]), _i32(cases[0][2]), _f32(cases[0][3]), _f32(cases[0][4])]
    na, nt = (torch.empty(B, dtype=torch.int32, device="cuda") for _ in range(2))
    ws = _workspace(F, B, T, V)
    call = lambda: F.fdllm_chain_verify(t[0], t[1], t[2], None, t[3], t[4], na, nt, ws)  # noqa: E731
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        call()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for c in cases:
        for x, y in zip(t, (_f32(c[0]), _f32(c[1]), _i32(c[2]), _f32(c[3]), _f32(c[4]))):
            x.copy_(y)
        graph.replay()
        torch.cuda.synchronize()
        for b in range(B):
            assert (int(na[b]), int(nt[b])) == O.chain_verify(c[0][b], c[1][b], c[2][b], T, c[3][b], c[4][b])
