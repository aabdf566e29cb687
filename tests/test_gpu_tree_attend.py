"""Attention of a drafted tree over a cache against the fp64 oracle.

The tolerance of an element is its worst case by arithmetic.  With A = sum_s p_s |v_s| and
S = max_s sum_d |q_d k_sd| / sqrt(dh):
  scores   a sum of dh products in fp32 is off by at most (dh + 10) 2^-24 S: a factor of
           1 + that on each weight, twice (weight and normaliser); 2^-21 more for exp2
  sums     n terms in fp32, rescaled as the maximum rises: n 2^-23
  weights  rounded to bf16 for the tensor cores (16- and 8-bit caches): 2^-8
  queries  kept as two e4m3 parts for an 8-bit cache: off by at most half the second
           part's smallest step, 2^-10 where the largest of the rows that share a kv head
           is at least 128, i.e. 2^-17 of it: dh 2^-17 max|q| max|k| / sqrt(dh) on a score
  output   rounded to bf16 (2^-8 of it) or fp32 (2^-24)
"""
import numpy as np
import pytest
import torch

import oracle as O

pytestmark = pytest.mark.gpu
E4M3 = torch.float8_e4m3fn
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "fp8": torch.bfloat16}
MARK = 7.0  # what the output holds where nothing may be written


@pytest.fixture(scope="module")
def F():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import kv_cache_attention_fdllm_b200 as F
    return F


def trees(g, B, T, width=6, roots=False):
    """parent [B, T]; with `roots` some nodes besides node 0 hang below the sequence itself."""
    p = np.full((B, T), -1, np.int32)
    for b in range(B):
        for t in range(1, T):
            p[b, t] = -1 if roots and g.random() < 0.2 else g.integers(max(0, t - width), t)
    return p


class Case:
    def __init__(self, kind, B, N, Hq, Hkv, dh, T, lens, parent="tree", nodes=None, seed=0, qs=2.0):
        g = np.random.default_rng(seed)
        self.kind, self.B, self.N, self.Hq, self.Hkv, self.dh, self.T = kind, B, N, Hq, Hkv, dh, T
        self.lens = np.asarray(lens, np.int32)
        self.nodes = None if nodes is None else np.asarray(nodes, np.int32)
        self.parent = None if parent is None else trees(g, B, T, roots=parent == "roots")
        dt = DT[kind]
        rn = lambda *s: torch.from_numpy(g.standard_normal(s, np.float32))  # noqa: E731
        self.q = (qs * rn(B, T, Hq, dh)).to(dt)
        self.k, self.v = rn(B, Hkv, N, dh).to(dt), rn(B, Hkv, N, dh).to(dt)
        # what no node sees holds NaN
        for b in range(B):
            n = T if nodes is None else int(self.nodes[b])
            self.k[b, :, max(0, int(self.lens[b]) + n):] = float("nan")
            self.v[b, :, max(0, int(self.lens[b]) + n):] = float("nan")
        self.scales = None
        if kind == "fp8":
            bits, self.scales = [], []
            for x in (self.k, self.v):
                val, sc = O.quantise_rows(O.to_f64(x))
                # the scales of unseen slots hold NaN too
                sc[np.isnan(O.to_f64(x)).any(-1)] = np.nan
                bits.append(torch.from_numpy(val.astype(np.float32)).to(E4M3))
                self.scales.append(torch.from_numpy(sc))
            self.k, self.v = bits
            self.k64 = O.e4m3_to_f64(self.k.view(torch.uint8).numpy()) * self.scales[0].numpy()[..., None].astype(np.float64)
            self.v64 = O.e4m3_to_f64(self.v.view(torch.uint8).numpy()) * self.scales[1].numpy()[..., None].astype(np.float64)
        else:
            self.k64, self.v64 = O.to_f64(self.k), O.to_f64(self.v)

    def dev(self, F):
        d = lambda a: None if a is None else (torch.from_numpy(a) if isinstance(a, np.ndarray) else a).cuda()  # noqa: E731
        self.t = dict(q=d(self.q), k=d(self.k), v=d(self.v), lens=d(self.lens), parent=d(self.parent),
                      nodes=d(self.nodes), scales=None if self.scales is None else [d(s) for s in self.scales])
        self.t["out"] = torch.full((self.B, self.T, self.Hq * self.dh), MARK, dtype=DT[self.kind], device="cuda")
        self.ws = F.alloc_workspace(F.fdllm_tree_attend_workspace_bytes(
            self.B, self.N, self.Hq, self.Hkv, self.dh, self.T, DT[self.kind]), "cuda")
        return self

    def call(self, F, ws=None, stream=None):
        t = self.t
        ws = self.ws if ws is None else ws
        if self.kind == "fp8":
            return F.fdllm_tree_attend_fp8(t["q"], t["k"], t["v"], t["scales"][0], t["scales"][1], t["lens"],
                                           t["parent"], t["nodes"], t["out"], ws, stream=stream)
        return F.fdllm_tree_attend(t["q"], t["k"], t["v"], t["lens"], t["parent"], t["nodes"], t["out"], ws,
                                   stream=stream)

    def check(self, seqs=None):
        torch.cuda.synchronize()
        got = O.to_f64(self.t["out"].cpu()).reshape(self.B, self.T, self.Hq, self.dh)
        q64 = O.to_f64(self.q)
        for b in range(self.B) if seqs is None else seqs:
            n = self.T if self.nodes is None else int(self.nodes[b])
            assert (got[b, n:] == MARK).all(), ("padding rows written", b)
            if n == 0:
                continue
            L = int(self.lens[b])
            par = None if self.parent is None else self.parent[b]
            out, A, S = O.tree_attend(q64[b], self.k64[b], self.v64[b], L, par, n)
            e = 2 * ((self.dh + 10) * 2.0 ** -24 * S + 2.0 ** -21) + (L + n) * 2.0 ** -23
            if self.kind == "fp8":
                g = self.Hq // self.Hkv
                qm = np.abs(q64[b, :n]).reshape(n, self.Hkv, g * self.dh).max((0, 2)).repeat(g)
                km = np.nanmax(np.abs(self.k64[b, :, :L + n]), (1, 2)).repeat(g)
                e = e + 2 * np.sqrt(self.dh) * 2.0 ** -17 * qm * km
            if self.kind != "f32":
                e = e + 2.0 ** -8
            half = 2.0 ** -24 if self.kind == "f32" else 2.0 ** -8
            tol = A * (np.exp(e) - 1)[..., None]
            tol = tol + half * (np.abs(out) + tol)
            err = np.abs(got[b, :n] - out)
            assert np.isfinite(got[b, :n]).all(), ("not finite", b)
            assert (err <= tol).all(), (b, float((err / tol).max()))


KINDS = ["f32", "bf16", "fp8"]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("B,N,Hq,Hkv,dh,T,lens", [
    (1, 1, 1, 1, 64, 1, [0]),                        # one slot, one node
    (1, 8, 2, 1, 128, 3, [0]),                       # a tree on an empty cache
    (2, 129, 4, 4, 64, 1, [127, 128]),               # single tokens around a tile's end
    (2, 300, 4, 2, 128, 5, [123, 124]),              # the tree across a tile's end
    (3, 257, 6, 2, 128, 7, [250, 0, 121]),           # groups of 3
    (2, 400, 14, 2, 64, 9, [391, 100]),              # groups of 7
    (1, 700, 8, 1, 128, 33, [600]),                  # 264 rows to one head
    (2, 600, 32, 4, 64, 16, [500, 584]),
    (1, 500, 64, 1, 64, 3, [450]),                   # 64 query heads to one
    (1, 600, 1, 1, 128, 256, [300]),                 # the largest tree
])
def test_trees(F, kind, B, N, Hq, Hkv, dh, T, lens):
    c = Case(kind, B, N, Hq, Hkv, dh, T, lens, seed=N + T).dev(F)
    c.call(F)
    assert F.fdllm_get_status(c.ws) == F.OK
    c.check()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("T,dh", [(1, 128), (2, 64), (31, 128), (65, 64), (130, 128)])
def test_chain_is_causal(F, kind, T, dh):
    c = Case(kind, 2, 300, 4, 2, dh, T, [77, 300 - T], parent=None, seed=T).dev(F)
    c.call(F)
    c.check()


@pytest.mark.parametrize("kind", KINDS)
def test_several_roots(F, kind):
    """Nodes with parent -1 see the sequence and themselves, not one another."""
    c = Case(kind, 3, 200, 4, 2, 64, 24, [50, 0, 176], parent="roots", seed=4).dev(F)
    c.call(F)
    assert F.fdllm_get_status(c.ws) == F.OK
    c.check()


@pytest.mark.parametrize("kind", KINDS)
def test_ragged_nodes_and_padding_rows(F, kind):
    c = Case(kind, 5, 260, 6, 3, 128, 12, [0, 248, 100, 128, 5], nodes=[12, 12, 0, 1, 7], seed=1).dev(F)
    c.call(F)
    assert F.fdllm_get_status(c.ws) == F.OK
    c.check()


@pytest.mark.parametrize("kind", KINDS)
def test_every_sequence_empty(F, kind):
    c = Case(kind, 3, 64, 2, 2, 64, 4, [0, 10, 64], nodes=[0, 0, 0]).dev(F)
    c.call(F)
    assert F.fdllm_get_status(c.ws) == F.OK
    c.check()


@pytest.mark.parametrize("kind", KINDS)
def test_bad_lengths_and_parents(F, kind):
    """A sequence out of range is left out, the others are computed; a bad parent counts as -1."""
    c = Case(kind, 6, 100, 4, 2, 64, 6, [10, 20, 30, 40, 50, 60], seed=2).dev(F)
    bad = np.array([10, -1, 95, 40, 50, 2 ** 31 - 1], np.int32)
    c.t["lens"] = torch.from_numpy(bad).cuda()
    c.t["nodes"] = torch.tensor([6, 6, 6, 7, -1, 6], dtype=torch.int32, device="cuda")
    c.call(F)
    assert F.fdllm_get_status(c.ws) == F.ERR_BAD_INDEX
    c.check(seqs=[0])
    assert (c.t["out"][1:] == MARK).all()
    c = Case(kind, 2, 100, 4, 2, 64, 6, [10, 20], seed=2).dev(F)
    wrong = c.parent.copy()
    wrong[0, 3], wrong[1, 5] = 3, -9
    c.t["parent"] = torch.from_numpy(wrong).cuda()
    c.parent[0, 3], c.parent[1, 5] = -1, -1
    c.call(F)
    assert F.fdllm_get_status(c.ws) == F.ERR_BAD_INDEX
    c.check()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("what", [float("nan"), float("inf"), -float("inf")])
def test_unseen_siblings_may_hold_anything(F, kind, what):
    """NaN or infinity in one node's k or v reaches that node and those below it alone."""
    c = Case(kind, 2, 300, 4, 2, 128, 12, [100, 120], seed=6).dev(F)
    bad = [5, 7]
    for b in range(2):
        slot = int(c.lens[b]) + bad[b]
        if kind == "fp8":
            for s in c.t["scales"]:
                s[b, :, slot] = what
        else:
            c.t["k"][b, 0, slot, 3] = what
            c.t["v"][b, 1, slot] = what
            c.t["v"][b, 0, slot, 9] = what
    c.call(F)
    torch.cuda.synchronize()
    got = O.to_f64(c.t["out"].cpu()).reshape(2, 12, 4, 128)
    for b in range(2):
        see = O.ancestors(c.parent[b], 12)
        hit = see[:, bad[b]]
        assert np.isfinite(got[b, ~hit]).all()
        # what sees it: v's infinity or NaN arrives as such
        if kind != "fp8":
            assert not np.isfinite(got[b, hit][:, 2:]).any()
        out, A, _ = O.tree_attend(O.to_f64(c.q)[b], c.k64[b], c.v64[b], int(c.lens[b]), c.parent[b], 12)
        assert (np.abs(got[b, ~hit] - out[~hit]) <= 0.02 * A[~hit]).all()


@pytest.mark.parametrize("kind", KINDS)
def test_one_slot_far_above_the_rest(F, kind):
    """Scores in the hundreds and rising maxima along the cache."""
    c = Case(kind, 1, 1000, 4, 2, 64, 4, [990], seed=8, qs=30.0).dev(F)
    c.call(F)
    c.check()


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
def test_a_sink_and_a_long_flat_rest(F, kind):
    """One slot e^11 above 8000 equal ones, which together still weigh a seventh of it: the
    small weights are not lost."""
    c = Case(kind, 1, 8192, 2, 1, 64, 2, [8100], parent=None, seed=9)
    c.q[:] = 0
    c.q[..., 0] = 8.0
    k = torch.zeros(1, 1, 8192, 64)
    k[:, :, 77, 0] = 11.0
    v = torch.ones(1, 1, 8192, 64) * 3.0
    v[:, :, 77] = -1.0
    if kind == "fp8":
        for i, x in enumerate((k, v)):
            val, sc = O.quantise_rows(x.numpy())
            new = torch.from_numpy(val.astype(np.float32)).to(E4M3)
            c.scales[i] = torch.from_numpy(sc)
            x64 = val * sc[..., None].astype(np.float64)
            if i == 0:
                c.k, c.k64 = new, x64
            else:
                c.v, c.v64 = new, x64
    else:
        c.k, c.v = k.to(torch.bfloat16), v.to(torch.bfloat16)
        c.k64, c.v64 = O.to_f64(c.k), O.to_f64(c.v)
    c.dev(F)
    c.call(F)
    c.check()


@pytest.mark.parametrize("kind", KINDS)
def test_same_bits_twice_and_one_workspace_for_all(F, kind):
    """Repeated calls give the same bits; a workspace sized for the largest call serves the
    others in any order."""
    cases = [Case(kind, *a, seed=3).dev(F) for a in ((3, 900, 8, 2, 128, 20, [880, 3, 500]), (1, 200, 4, 4, 64, 1, [150]),
                                                     (8, 300, 4, 1, 64, 9, [290, 0, 7, 130, 250, 128, 127, 129]))]
    ws = max((c.ws for c in cases), key=lambda w: w.numel())
    first = []
    for c in cases:
        c.call(F, ws=ws)
        c.check()
        first.append(c.t["out"].clone())
    for i in (2, 0, 1, 1, 0, 2):
        cases[i].t["out"].fill_(MARK)
        cases[i].call(F, ws=ws)
        assert torch.equal(cases[i].t["out"], first[i])


@pytest.mark.parametrize("kind", KINDS)
def test_captured_and_replayed_on_growing_lengths(F, kind):
    """One graph serves a decode whose lengths grow in place."""
    c = Case(kind, 2, 400, 4, 2, 64, 3, [100, 200], parent=None, seed=5).dev(F)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        c.call(F)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.call(F)
    for step in ([0, 1], [97, 200], [30, 126], [100, 5]):
        c.lens = np.asarray(step, np.int32)
        c.t["lens"].copy_(torch.from_numpy(c.lens))
        graph.replay()
        c.check()


@pytest.mark.parametrize("kind", KINDS)
def test_two_streams_with_their_own_workspaces(F, kind):
    cs = [Case(kind, 4, 800, 8, 2, 128, 6, [700, 10, 400, 794], seed=s).dev(F) for s in (1, 2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cs]
    for _ in range(5):
        for c, s in zip(cs, streams):
            c.call(F, stream=s)
    for c in cs:
        c.check()


def test_offsets_past_32_bits(F):
    """A cache of over 2^32 elements: the last head of the last sequence."""
    N, Hkv, dh, T = 270336, 128, 128, 2
    need = N * Hkv * dh
    assert need > 2 ** 32
    k = torch.zeros((1, Hkv, N, dh), dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    g = torch.Generator(device="cuda").manual_seed(0)
    L = 300
    small_k = torch.randn(Hkv, L + T, dh, generator=g, device="cuda").to(torch.bfloat16)
    small_v = torch.randn(Hkv, L + T, dh, generator=g, device="cuda").to(torch.bfloat16)
    k[0, :, :L + T], v[0, :, :L + T] = small_k, small_v
    q = torch.randn(1, T, Hkv, dh, generator=g, device="cuda").to(torch.bfloat16)
    lens = torch.tensor([L], dtype=torch.int32, device="cuda")
    outs = []
    for kk, vv in ((k, v), (small_k[None], small_v[None])):
        out = torch.empty((1, T, Hkv * dh), dtype=torch.bfloat16, device="cuda")
        ws = F.alloc_workspace(F.fdllm_tree_attend_workspace_bytes(1, kk.shape[2], Hkv, Hkv, dh, T, torch.bfloat16), "cuda")
        F.fdllm_tree_attend(q, kk.contiguous(), vv.contiguous(), lens, None, None, out, ws)
        assert F.fdllm_get_status(ws) == F.OK
        outs.append(out)
    assert torch.equal(outs[0], outs[1])


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dh", [64, 128])
@pytest.mark.parametrize("B,Hq,Hkv,T", [
    (1, 1, 1, 1), (4, 4, 4, 1), (4, 4, 2, 1), (4, 6, 2, 1), (4, 8, 2, 1), (4, 2, 2, 2), (4, 2, 1, 2), (4, 3, 3, 3),
    (4, 2, 2, 4), (9, 8, 8, 1), (40, 3, 3, 1), (100, 3, 3, 1), (40, 8, 2, 1)])
def test_few_rows(F, kind, dh, B, Hq, Hkv, T):
    """Up to 4 rows to a kv head, over lengths from none to several rounds of every part."""
    N = 2600
    some = [N - T, 0, 129, 1, 16, 517, 64, 255, 1024]
    lens = [some[b % len(some)] for b in range(B)]
    nodes = None if T == 1 else [T - b % 3 if T > b % 3 else 0 for b in range(B)]
    c = Case(kind, B, N, Hq, Hkv, dh, T, lens, parent="roots", nodes=nodes, seed=dh + T).dev(F)
    c.call(F)
    c.check()
    assert F.fdllm_get_status(c.ws) == F.OK


@pytest.mark.parametrize("kind", KINDS)
def test_single_tokens_captured_on_growing_lengths(F, kind):
    """One token at a time: the call is captured once, the lengths grow on the device."""
    c = Case(kind, 2, 600, 4, 2, 128, 1, [3, 500], parent=None, seed=21).dev(F)
    for t in (c.t["k"], c.t["v"]) + tuple(c.t["scales"] or ()):  # no slot is out of use for good
        x = t.view(torch.uint8) if t.element_size() == 1 else t
        x[:, :, 3:] = x[:, :, :1]
    host = lambda t: O.e4m3_to_f64(t.view(torch.uint8).cpu().numpy()) if kind == "fp8" else O.to_f64(t.cpu())  # noqa: E731
    c.k64, c.v64 = host(c.t["k"]), host(c.t["v"])
    if kind == "fp8":
        c.k64, c.v64 = (x * s.cpu().numpy()[..., None].astype(np.float64) for x, s in zip((c.k64, c.v64), c.t["scales"]))
    c.call(F)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.call(F)
        c.t["lens"] += 1
    for _ in range(40):
        graph.replay()
    c.lens = c.lens + 39
    c.check()
    assert F.fdllm_get_status(c.ws) == F.OK


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("T,Hq", [(1, 2), (1, 8), (9, 8)])
def test_same_bits_in_any_capacity(F, kind, T, Hq):
    """The cache's capacity changes no bit of the result."""
    outs = []
    for N in (300, 9000):
        c = Case(kind, 2, 300, Hq, 2, 64, T, [123, 290], parent=None, seed=8)
        if N > 300:
            grow = lambda x: torch.cat([x.view(torch.uint8) if kind == "fp8" and x.dim() == 4 else x,  # noqa: E731
                                        torch.zeros((2, 2, N - 300) + x.shape[3:], dtype=torch.uint8 if kind == "fp8" and x.dim() == 4 else x.dtype)], 2)
            back = lambda x: grow(x).view(x.dtype)  # noqa: E731
            c.k, c.v, c.N = back(c.k), back(c.v), N
            if c.scales is not None:
                c.scales = [back(s) for s in c.scales]
        c.dev(F).call(F)
        torch.cuda.synchronize()
        assert F.fdllm_get_status(c.ws) == F.OK
        outs.append(c.t["out"].cpu())
    assert torch.equal(outs[0], outs[1])


@pytest.mark.parametrize("kind,Hq,Hkv,T", [
    ("bf16", 64, 16, 4), ("bf16", 64, 16, 7), ("bf16", 48, 16, 15), ("bf16", 64, 16, 50), ("fp8", 64, 16, 3),
    ("fp8", 48, 16, 15)])
@pytest.mark.parametrize("dh", [64, 128])
def test_many_short_items_are_the_same_every_time(F, kind, Hq, Hkv, T, dh):
    """A CTA that goes through many items hands its sums over between them: the end of one
    and the first tile of the next do not meet in shared memory."""
    B, N = 32, 700
    lens = [(b * 97) % (N - T) for b in range(B)]
    c = Case(kind, B, N, Hq, Hkv, dh, T, lens, seed=4).dev(F)
    c.call(F)
    c.check(seqs=[1, 17])
    first = c.t["out"].clone()
    for _ in range(30):
        c.t["out"].fill_(MARK)
        c.call(F)
        assert torch.equal(c.t["out"].view(torch.int16), first.view(torch.int16))
