"""Attention over an 8-bit cache whose rows differ widely in magnitude, against the fp64 oracle.

The tolerance of an element is that of the other attention tests (scores, sums, weights and the
output's rounding), with two terms taken where they arise.  A row is a (node, query head) pair:
  queries  a row's two e4m3 parts lose at most 2^-17 of that row's largest element: on a score
           sqrt(dh) 2^-17 max|q| max|k|, q of this row and k of the slots that it sees
  weights  the largest product of a weight and its slot's scale that the row sees is held at
           2^8 or above in fp16 parts whose smallest step is 2^-16: half a step, 2^-17, is 2^-25
           of it, times the slot's e4m3 element, summed over the slots
"""
import numpy as np
import pytest
import torch

import oracle as O
from test_gpu_tree_attend import Case, E4M3, F, MARK  # noqa: F401

pytestmark = pytest.mark.gpu

# many items a CTA or parts of one; chunks of one node and of several; both head sizes
SHAPES = [
    (2, 300, 4, 2, 128, 12, [100, 120]),
    (1, 4000, 8, 2, 128, 12, [3900]),           # every tile its own CTA: results are merged
    (40, 200, 16, 8, 64, 9, [b * 4 for b in range(40)]),
    (2, 500, 48, 1, 64, 7, [300, 484]),         # a node's heads in two chunks
]


def from_device(c):
    """The 64-bit values of the cache as it now stands on the device."""
    val = [O.e4m3_to_f64(c.t[n].view(torch.uint8).cpu().numpy()) for n in "kv"]
    c.v_val = val[1]
    c.v_sc = c.t["scales"][1].cpu().numpy().astype(np.float64)
    with np.errstate(invalid="ignore"):
        c.k64, c.v64 = (x * s.cpu().numpy()[..., None].astype(np.float64) for x, s in zip(val, c.t["scales"]))


def check_rows(c, rows=None, seqs=None):
    """Rows [B, T] (all of them: None) against the oracle, at every element."""
    torch.cuda.synchronize()
    got = O.to_f64(c.t["out"].cpu()).reshape(c.B, c.T, c.Hq, c.dh)
    q64 = O.to_f64(c.q)
    g = c.Hq // c.Hkv
    worst = 0.0
    for b in range(c.B) if seqs is None else seqs:
        L = int(c.lens[b])
        with np.errstate(invalid="ignore", over="ignore"):
            out, A, S = O.tree_attend(q64[b], c.k64[b], c.v64[b], L, c.parent[b], c.T)
        see = O.ancestors(c.parent[b], c.T)
        for t in range(c.T):
            if rows is not None and not rows[b, t]:
                continue
            slots = np.concatenate([np.arange(L), L + np.nonzero(see[t])[0]])
            for h in range(c.Hq):
                k, q = c.k64[b, h // g, slots], q64[b, t, h]
                s = k @ q / np.sqrt(c.dh)
                p = np.exp(s - s.max())
                p /= p.sum()
                top = (p * np.abs(c.v_sc[b, h // g, slots])).max()
                lost = 2.0 ** -25 * top * np.abs(c.v_val[b, h // g, slots]).sum(0)
                e = 2 * ((c.dh + 10) * 2.0 ** -24 * S[t, h] + 2.0 ** -21) + len(slots) * 2.0 ** -23
                e += 2 * np.sqrt(c.dh) * 2.0 ** -17 * np.abs(q).max() * np.abs(k).max() + 2.0 ** -8
                with np.errstate(over="ignore"):
                    tol = A[t, h] * (np.exp(e) - 1) + lost
                tol = tol + 2.0 ** -8 * (np.abs(out[t, h]) + tol)
                assert np.isfinite(got[b, t, h]).all(), ("not finite", b, t, h)
                err = np.abs(got[b, t, h] - out[t, h])
                worst = max(worst, float((err / np.maximum(tol, 1e-300)).max()))
                assert (err <= tol).all(), (b, t, h, worst)
    return got


def write_node(c, F, node, row):
    """Writes a V row (and the K row as it was drawn) for one node of every sequence."""
    g = np.random.default_rng(77)
    k = torch.from_numpy(g.standard_normal((c.B, 1, c.Hkv, c.dh), np.float32)).to(torch.bfloat16).cuda()
    v = row.to(torch.bfloat16).expand(c.B, 1, c.Hkv, c.dh).contiguous().cuda()
    pos = (c.t["lens"] + node).to(torch.int32).reshape(c.B, 1).contiguous()
    F.fdllm_cache_write_fp8(k, v, pos, c.t["k"], c.t["v"], c.t["scales"][0], c.t["scales"][1], c.ws)
    from_device(c)


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("size", [float("inf"), -float("inf"), 2.0 ** 100, 2.0 ** 30, 2.0 ** 17])
def test_an_unseen_sibling_of_any_size(F, shape, size):
    """A drafted node whose v holds an infinity or is far above the others, as
    fdllm_cache_write_fp8 stores it, changes no node that does not see it."""
    c = Case("fp8", *shape, seed=11).dev(F)
    bad = 3
    row = torch.linspace(-1.0, 1.0, c.dh)
    row = row * size if np.isfinite(size) else torch.where(torch.arange(c.dh) == 5, size, row)
    write_node(c, F, bad, row)
    c.call(F)
    assert F.fdllm_get_status(c.ws) == F.OK
    see = np.stack([O.ancestors(p, c.T)[:, bad] for p in c.parent])
    seqs = range(0, c.B, max(1, c.B // 4))
    got = check_rows(c, ~see, seqs)
    if np.isfinite(size):
        check_rows(c, see, seqs)
    else:  # and reaches those that do
        for b in seqs:
            assert (np.sign(size) * got[b, see[b]][..., 5] > 1e20).all()


@pytest.mark.parametrize("shape", [s for s in SHAPES if s[3] < 8])
def test_a_large_row_of_little_weight(F, shape):
    """A slot of the sequence whose v is 2^40 above the others, and whose weight makes its
    share 2^-20 of theirs."""
    c = Case("fp8", *shape, seed=12, qs=0.5)
    c.q[..., 0] = 8.0
    for b in range(c.B):
        for s in (7, 77):
            k = np.zeros((c.Hkv, c.dh), np.float32)
            k[:, 0] = -60 * np.log(2) * np.sqrt(c.dh) / 8
            v = np.linspace(-1, 1, c.dh, dtype=np.float32)[None].repeat(c.Hkv, 0) * np.float32(2.0 ** 40)
            for i, x in enumerate((k, v)):
                val, sc = O.quantise_rows(x)
                (c.k, c.v)[i][b, :, s] = torch.from_numpy(val.astype(np.float32)).to(E4M3)
                c.scales[i][b, :, s] = torch.from_numpy(sc)
    c.dev(F)
    from_device(c)
    c.call(F)
    check_rows(c)


@pytest.mark.parametrize("exp", [-70, -20, 60, 110])
def test_all_rows_of_one_size(F, exp):
    """v around 2^exp throughout: nothing is lost on the way."""
    c = Case("fp8", 2, 600, 8, 2, 128, 9, [500, 33], seed=13)
    c.scales[1] = torch.ldexp(c.scales[1], torch.tensor(exp))
    c.dev(F)
    from_device(c)
    c.call(F)
    check_rows(c)


def test_rows_of_zeros(F):
    """v all zeros (the smallest scale there is) gives zeros; among others it changes nothing."""
    c = Case("fp8", 2, 600, 8, 2, 128, 9, [500, 33], seed=14)
    c.v[0] = torch.zeros(c.v[0].shape).to(E4M3)
    c.scales[1][0] = float(np.float32(2.0 ** -96) / np.float32(448))
    c.v[1, :, ::3] = torch.zeros(c.v[1, :, ::3].shape).to(E4M3)
    c.scales[1][1, :, ::3] = 0.0
    c.scales[1][1, :, 1::3] = -c.scales[1][1, :, 1::3]  # a caller's own scales may be negative
    c.dev(F)
    from_device(c)
    c.call(F)
    check_rows(c)
    assert (c.t["out"][0] == 0).all()


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("exp", [12, 20, 60])
def test_queries_of_different_size(F, shape, exp):
    """One node's queries, and one head's, far above and below the others': each row is as
    exact as if it were alone."""
    c = Case("fp8", *shape, seed=15)
    c.q[:, 4] = (c.q[:, 4].float() * 2.0 ** exp).to(torch.bfloat16)
    c.q[:, :, 1] = (c.q[:, :, 1].float() * 2.0 ** -exp).to(torch.bfloat16)
    c.dev(F)
    from_device(c)
    c.call(F)
    seqs = range(0, c.B, max(1, c.B // 4))
    rows = np.ones((c.B, c.T), bool)
    rows[:, 4] = False  # its scores are beyond what an exponent is formed from
    check_rows(c, rows, seqs)


@pytest.mark.parametrize("what", [float("nan"), float("inf")])
def test_a_query_that_is_not_finite(F, what):
    """It makes its own row NaN and no other."""
    c = Case("fp8", 2, 600, 8, 2, 128, 9, [500, 33], seed=16)
    c.q[:, 4, 3, 17] = what
    c.dev(F)
    c.q[:, 4, 3, 17] = 0.0  # for the oracle
    from_device(c)
    c.call(F)
    got = O.to_f64(c.t["out"].cpu()).reshape(c.B, c.T, c.Hq, c.dh)
    assert np.isnan(got[:, 4, 3]).all()
    got[:, 4, 3] = 0.0
    assert np.isfinite(got).all()
    rows = np.ones((c.B, c.T), bool)
    rows[:, 4] = False
    check_rows(c, rows)


@pytest.mark.parametrize("shape", SHAPES + [(2, 600, 1, 1, 128, 3, [500, 3]), (3, 400, 2, 2, 64, 4, [390, 0, 7])])
def test_single_elements_that_are_nan(F, shape):
    """An 8-bit v of a node with NaN in single elements: NaN in exactly those of the nodes that
    see it, whole items and merged ones, and every other element as it should be."""
    c = Case("fp8", *shape, seed=17)
    bad = 1
    where = [3, c.dh - 1]
    for b in range(c.B):
        slot = int(c.lens[b]) + bad
        bits = c.v.view(torch.uint8)
        bits[b, c.Hkv - 1, slot, where[0]] = 0x7f
        bits[b, c.Hkv - 1, slot, where[1]] = 0xff
    c.dev(F)
    from_device(c)
    c.call(F)
    assert F.fdllm_get_status(c.ws) == F.OK
    torch.cuda.synchronize()
    got = O.to_f64(c.t["out"].cpu()).reshape(c.B, c.T, c.Hkv, c.Hq // c.Hkv, c.dh)
    see = np.stack([O.ancestors(p, c.T)[:, bad] for p in c.parent])
    want = np.zeros(got.shape, bool)
    for d in where:
        want[:, :, c.Hkv - 1, :, d] = see[..., None]
    assert (np.isnan(got) == want).all()
    assert np.isfinite(got[~want]).all()
    # the rest: as if the elements were zeros
    out = c.t["out"]
    out[torch.isnan(out)] = 0.0
    c.v_val[np.isnan(c.v_val)] = 0.0
    c.v64[np.isnan(c.v64)] = 0.0
    seqs = range(0, c.B, max(1, c.B // 4))
    # (the oracle's zero where NaN was put to 0; other elements of those rows are compared too)
    res = O.to_f64(out.cpu()).reshape(c.B, c.T, c.Hq, c.dh)
    q64 = O.to_f64(c.q)
    for b in seqs:
        ref, _, _ = O.tree_attend(q64[b], c.k64[b], c.v64[b], int(c.lens[b]), c.parent[b], c.T)
        hit = want[b].reshape(c.T, c.Hq, c.dh)
        res[b][hit] = ref[hit]
    out.copy_(torch.from_numpy(res.reshape(out.shape)).to(out.dtype))
    check_rows(c, None, seqs)
