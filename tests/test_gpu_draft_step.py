"""Steps of speculative decoding as a caller runs them: write the drafts' rows, attend,
verify, write what was accepted where it belongs, again and again on growing sequences.

The model is one attention layer with tables for its projections; everything between the
calls is a gather, a product and a softmax on the same stream, with no read on the host.
Tolerances of the attention are those of test_gpu_tree_attend; verification and cache are
compared bit by bit, given the probabilities that the step itself formed.
"""
import numpy as np
import pytest
import torch

import oracle as O

pytestmark = pytest.mark.gpu
B, N, HQ, HKV, DH, V = 3, 700, 8, 2, 64, 519
LENS = [0, 130, 517]
E4M3 = torch.float8_e4m3fn


@pytest.fixture(scope="module")
def F():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import kv_cache_attention_fdllm_b200 as F
    return F


class Model:
    """Tables [V, ...] of a token's q, k, v (bf16), the head, and a cache of either kind."""

    def __init__(self, F, kind, T):
        self.F, self.kind, self.T = F, kind, T
        g = torch.Generator().manual_seed(5)
        rn = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
        self.q, self.k, self.v = (rn(V, HQ, DH).bfloat16(), rn(V, HKV, DH).bfloat16(), rn(V, HKV, DH).bfloat16())
        self.dev = [x.cuda() for x in (self.q, self.k, self.v)]
        self.head = (0.5 * rn(HQ * DH, V)).cuda()
        dt = E4M3 if kind == "fp8" else torch.bfloat16
        self.cache = [torch.zeros(B, HKV, N, DH, device="cuda").to(dt) for _ in range(2)]
        self.scale = [torch.zeros(B, HKV, N, device="cuda") for _ in range(2)]
        self.len = torch.tensor(LENS, dtype=torch.int32, device="cuda")
        self.out = torch.zeros(B, T, HQ * DH, dtype=torch.bfloat16, device="cuda")
        # one workspace for all of the calls
        size = max(F.fdllm_cache_fp8_workspace_bytes(B, max(LENS)),
                   F.fdllm_tree_attend_workspace_bytes(B, N, HQ, HKV, DH, T, torch.bfloat16),
                   F.fdllm_draft_verify_workspace_bytes(B, T, V))
        self.ws = F.alloc_workspace(size, "cuda")

    def write(self, tok, pos):
        """Rows of tok [B, R] to the slots pos int32 [B, R], -1: none."""
        k, v = self.dev[1][tok], self.dev[2][tok]
        if self.kind == "fp8":
            self.F.fdllm_cache_write_fp8(k, v, pos, *self.cache, *self.scale, self.ws)
            return
        # a 16-bit cache is the caller's to write; a spare slot at the end takes the padding
        at = torch.where(pos < 0, N - 1, pos).long()[:, None, :, None].expand(B, HKV, tok.shape[1], DH)
        for c, x in zip(self.cache, (k, v)):
            c.scatter_(2, at, x.transpose(1, 2))

    def attend(self, tok, parent, nodes):
        q = self.dev[0][tok]
        if self.kind == "fp8":
            self.F.fdllm_tree_attend_fp8(q, *self.cache, *self.scale, self.len, parent, nodes, self.out, self.ws)
        else:
            self.F.fdllm_tree_attend(q, *self.cache, self.len, parent, nodes, self.out, self.ws)

    def probabilities(self):
        return torch.softmax(self.out.float() @ self.head, -1)

    # ---- on the host
    def rows64(self, toks):
        """k, v [HKV, n, DH] in 64 bits as the cache holds them, and the cache's bits."""
        res = []
        for x in (self.k, self.v):
            x = x[torch.as_tensor(toks, dtype=torch.long)].transpose(0, 1)
            if self.kind == "fp8":
                val, sc = O.quantise_rows(O.to_f64(x))
                res.append((val * sc.astype(np.float64)[..., None], val, sc))
            else:
                res.append((O.to_f64(x), O.to_f64(x), None))
        return res

    def check_attend(self, seqs, tok, parent, nodes):
        got = O.to_f64(self.out.cpu()).reshape(B, self.T, HQ, DH)
        for b in range(B):
            n, L = int(nodes[b]), len(seqs[b])
            (k, _, _), (v, _, _) = self.rows64(list(seqs[b]) + list(tok[b, :n]))
            q = O.to_f64(self.q)[tok[b]]
            out, A, S = O.tree_attend(q, k, v, L, None if parent is None else parent[b], n)
            e = 2 * ((DH + 10) * 2.0 ** -24 * S + 2.0 ** -21) + (L + n) * 2.0 ** -23 + 2.0 ** -8
            if self.kind == "fp8":
                qm = np.abs(q[:n]).reshape(n, HKV, -1).max((0, 2)).repeat(HQ // HKV)
                km = np.abs(k).max((1, 2)).repeat(HQ // HKV)
                e = e + 2 * np.sqrt(DH) * 2.0 ** -17 * qm * km
            tol = A * (np.exp(e) - 1)[..., None]
            tol = tol + 2.0 ** -8 * (np.abs(out) + tol)
            assert (np.abs(got[b, :n] - out) <= tol).all(), b

    def check_cache(self, seqs):
        assert self.len.cpu().tolist() == [len(s) for s in seqs]
        for b in range(B):
            L = len(seqs[b])
            for c, s, (_, val, sc) in zip(self.cache, self.scale, self.rows64(seqs[b])):
                assert (O.to_f64(c[b, :, :L].float().cpu()) == val).all()
                if sc is not None:
                    assert (s[b, :, :L].cpu().numpy() == sc).all()


def start(F, kind, T):
    g = np.random.default_rng(11)
    m = Model(F, kind, T)
    seqs = [g.integers(0, V, n).tolist() for n in LENS]
    R = max(LENS)
    tok, pos = np.zeros((B, R), np.int64), np.full((B, R), -1, np.int32)
    for b in range(B):
        tok[b, :LENS[b]] = seqs[b]
        pos[b, :LENS[b]] = np.arange(LENS[b])
    m.write(torch.from_numpy(tok).cuda(), torch.from_numpy(pos).cuda())
    return g, m, seqs


def no_status(F, m):
    assert F.fdllm_get_status(m.ws) == 0


@pytest.mark.parametrize("kind", ["fp8", "bf16"])
def test_steps_of_a_tree(F, kind):
    T = 11
    g, m, seqs = start(F, kind, T)
    last = torch.from_numpy(g.integers(0, V, B)).cuda()  # the token that is certain, not yet in the cache
    taken = 0
    path = torch.zeros(B, T, dtype=torch.int32, device="cuda")
    na, nt = (torch.zeros(B, dtype=torch.int32, device="cuda") for _ in range(2))
    for step in range(6):
        parent = np.stack([[-1] + [int(g.integers(max(0, t - 4), t)) for t in range(1, T)] for _ in range(B)])
        parent = parent.astype(np.int32)
        nodes = np.asarray([T, int(g.integers(1, T + 1)), T - 2], np.int32)
        tok = g.integers(0, V, (B, T))
        # small numbers take drafts that are not likely, too
        u = (2.0 ** -12 * g.random((B, T))).astype(np.float32)
        r = g.random(B, np.float32)
        d_tok, d_par, d_n = (torch.from_numpy(x).cuda() for x in (tok, parent, nodes))
        d_u, d_r = torch.from_numpy(u).cuda(), torch.from_numpy(r).cuda()
        d_tok[:, 0] = last
        t = torch.arange(T, dtype=torch.int32, device="cuda")
        old = m.len.clone()
        m.write(d_tok, torch.where(t < d_n[:, None], old[:, None] + t, -1))
        m.attend(d_tok, d_par, d_n)
        target = m.probabilities()
        F.fdllm_tree_verify(target, d_tok.int(), d_par, d_n, d_u, d_r, path, na, nt, m.ws)
        # the accepted nodes' rows to the slots behind node 0's, in order
        pos = torch.full((B, T + 1), -1, dtype=torch.int32, device="cuda")
        pos.scatter_(1, torch.where(path < 0, T, path).long(), old[:, None] + 1 + t)
        m.write(d_tok, pos[:, :T].contiguous())
        m.len += 1 + na
        last = nt.long()
        torch.cuda.synchronize()
        no_status(F, m)

        tok = d_tok.cpu().numpy()
        m.check_attend(seqs, tok, parent, nodes)
        p = target.cpu().numpy()
        for b in range(B):
            want, nxt = O.tree_verify(p[b], tok[b], parent[b], int(nodes[b]), u[b], r[b])
            assert path[b].tolist() == want + [-1] * (T - len(want))
            assert (int(na[b]), int(nt[b])) == (len(want), nxt)
            seqs[b] += [int(tok[b, 0])] + [int(tok[b, c]) for c in want]
            taken += len(want)
        m.check_cache(seqs)
    assert taken > 0  # some drafts were accepted: the second write had rows to move


@pytest.mark.parametrize("kind", ["fp8", "bf16"])
def test_steps_of_a_chain_in_a_graph(F, kind):
    """The chain's step captured once and replayed: the lengths move on the device."""
    T = 5  # drafts; the attended chain has the certain token in front
    g, m, seqs = start(F, kind, T + 1)
    z = lambda *s, dtype=torch.int32: torch.zeros(*s, dtype=dtype, device="cuda")  # noqa: E731
    tok, draft = z(B, T + 1, dtype=torch.long), z(B, T, V, dtype=torch.float32)
    u, r = z(B, T, dtype=torch.float32), z(B, dtype=torch.float32)
    n_draft, old, na, nt = z(B), z(B), z(B), z(B)
    target = z(B, T + 1, V, dtype=torch.float32)
    t = torch.arange(T + 1, dtype=torch.int32, device="cuda")
    tok[:, 0] = torch.from_numpy(g.integers(0, V, B)).cuda()

    def step():
        old.copy_(m.len)
        nodes = n_draft + 1
        m.write(tok, torch.where(t < nodes[:, None], old[:, None] + t, -1))
        m.attend(tok, None, nodes)
        target.copy_(m.probabilities())
        F.fdllm_chain_verify(target, draft, tok[:, 1:].int().contiguous(), n_draft, u, r, na, nt, m.ws)
        # accepted drafts already lie in order: only the length moves
        m.len.add_(1 + na)

    def inputs():
        d = g.dirichlet(np.ones(V), (B, T)).astype(np.float32)
        x = np.stack([[g.choice(V, p=d[b, i] / d[b, i].astype(np.float64).sum()) for i in range(T)]
                      for b in range(B)])
        draft.copy_(torch.from_numpy(d))
        tok[:, 1:] = torch.from_numpy(x).cuda()
        u.copy_(torch.from_numpy((2.0 ** -3 * g.random((B, T))).astype(np.float32)))
        r.copy_(torch.from_numpy(g.random(B, np.float32)))
        n_draft.copy_(torch.from_numpy(g.integers(0, T + 1, B).astype(np.int32)))

    inputs()
    first = m.len.clone()
    step()  # warm-up, taken back
    torch.cuda.synchronize()
    m.len.copy_(first)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    taken = 0
    for _ in range(6):
        inputs()
        graph.replay()
        torch.cuda.synchronize()
        no_status(F, m)
        x, n = tok.cpu().numpy(), n_draft.cpu().numpy()
        m.check_attend(seqs, x, None, n + 1)
        for b in range(B):
            want = O.chain_verify(target[b].cpu().numpy(), draft[b].cpu().numpy(), x[b, 1:], int(n[b]),
                                  u[b].cpu().numpy(), r[b].item())
            assert (int(na[b]), int(nt[b])) == want
            seqs[b] += x[b, :1 + want[0]].tolist()
            taken += want[0]
        m.check_cache(seqs)
        tok[:, 0] = nt.long()
    assert taken > 0


def test_one_workspace_for_every_call(F):
    """Attention's partials and verification's counters do not meet: every order of the calls
    on one workspace gives what each gives on its own."""
    g = np.random.default_rng(3)
    T = 40
    q = torch.from_numpy(g.standard_normal((2, T, HQ, DH), np.float32)).bfloat16().cuda()
    cache = [torch.from_numpy(g.standard_normal((2, HKV, 5000, DH), np.float32)).bfloat16().cuda() for _ in range(2)]
    lens = torch.tensor([4900, 1], dtype=torch.int32, device="cuda")
    target = torch.softmax(torch.from_numpy(g.standard_normal((2, T + 1, 7001), np.float32)), -1).cuda()
    draft = target[:, :T].flip(0).contiguous()
    tok = torch.from_numpy(g.integers(0, 7001, (2, T)).astype(np.int32)).cuda()
    u, r = torch.zeros(2, T, device="cuda"), torch.full((2,), 0.6, device="cuda")
    size = max(F.fdllm_tree_attend_workspace_bytes(2, 5000, HQ, HKV, DH, T, torch.bfloat16),
               F.fdllm_draft_verify_workspace_bytes(2, T, 7001))
    shared = F.alloc_workspace(size, "cuda")

    def attend(ws):
        out = torch.zeros(2, T, HQ * DH, dtype=torch.bfloat16, device="cuda")
        F.fdllm_tree_attend(q, *cache, lens, None, None, out, ws)
        return [out]

    def verify(ws):
        res = [torch.zeros(2, dtype=torch.int32, device="cuda") for _ in range(2)]
        F.fdllm_chain_verify(target, draft, tok, None, u, r, *res, ws)
        return res

    want = [f(F.alloc_workspace(size, "cuda")) for f in (attend, verify)]
    for _ in range(3):
        for f, w in ((attend, want[0]), (verify, want[1]), (verify, want[1]), (attend, want[0])):
            for a, b in zip(f(shared), w):
                assert torch.equal(a, b)
    assert F.fdllm_get_status(shared) == 0


@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_a_score_of_minus_infinity_weighs_nothing(F, kind):
    """A key whose score is -inf, the first one included, leaves the others their weights."""
    dt = torch.float32 if kind == "f32" else torch.bfloat16
    g = np.random.default_rng(4)
    L, T = 270, 3
    q = torch.from_numpy(np.abs(g.standard_normal((1, T, HQ, DH), np.float32)) + 0.1).to(dt)
    k, v = (torch.from_numpy(g.standard_normal((1, HKV, L + T, DH), np.float32)).to(dt) for _ in range(2))
    gone = [0, 1, 2, 8, 130, 269]
    k[:, :, gone, 7] = -float("inf")
    out = torch.zeros(1, T, HQ * DH, dtype=dt, device="cuda")
    ws = F.alloc_workspace(F.fdllm_tree_attend_workspace_bytes(1, L + T, HQ, HKV, DH, T, dt), "cuda")
    F.fdllm_tree_attend(q.cuda(), k.cuda(), v.cuda(), torch.tensor([L], dtype=torch.int32, device="cuda"),
                        None, None, out, ws)
    torch.cuda.synchronize()
    keep = [s for s in range(L + T) if s not in gone]
    want, A, S = O.tree_attend(O.to_f64(q)[0], O.to_f64(k[:, :, keep])[0], O.to_f64(v[:, :, keep])[0],
                               L - len(gone), None, T)
    e = 2 * ((DH + 10) * 2.0 ** -24 * S + 2.0 ** -21) + (L + T) * 2.0 ** -23 + (0 if kind == "f32" else 2.0 ** -8)
    half = 2.0 ** -24 if kind == "f32" else 2.0 ** -8
    tol = A * (np.exp(e) - 1)[..., None]
    tol = tol + half * (np.abs(want) + tol)
    got = O.to_f64(out.cpu()).reshape(T, HQ, DH)
    assert (np.abs(got - want) <= tol).all()
