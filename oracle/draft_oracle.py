"""fp64 CPU oracle of the calls for drafted tokens (test infrastructure only).

8-bit cache rows, attention of a drafted tree over a cache, and the verification
of sampled drafts, each straight from its definition (include/fdllm.h).  The same
rules as in fdllm_oracle.py: nothing here is shared with the CUDA path.
"""
from __future__ import annotations

import numpy as np

E4M3_MAX = 448.0
TINY = 2.0 ** -96


# ----------------------------------------------------------------------------
# e4m3


def e4m3_to_f64(bits) -> np.ndarray:
    """Values of e4m3 bytes: sign, 4 exponent bits (bias 7), 3 mantissa bits; 0x7f is NaN."""
    b = np.asarray(bits).astype(np.int64)
    e, m = (b >> 3) & 15, b & 7
    v = np.where(e > 0, np.ldexp(1.0 + m / 8.0, e - 7), np.ldexp(m / 8.0, -6))
    v = np.where((b & 127) == 127, np.nan, v)
    return np.where(b & 128, -v, v)


def round_e4m3(x) -> np.ndarray:
    """float64 values rounded to the nearest e4m3 value, ties to even, beyond 448 to 448.

    Four significant bits: with |x| = m * 2^e, 0.5 <= m < 1, a step is 2^(e-4), at
    least the subnormal step 2^-9."""
    x = np.clip(np.asarray(x, np.float64), -E4M3_MAX, E4M3_MAX)
    with np.errstate(invalid="ignore"):
        _, e = np.frexp(x)
        step = np.ldexp(1.0, np.maximum(e - 4, -9))
        return np.rint(x / step) * step


def quantise_rows(x) -> tuple:
    """(values, scales) of the 8-bit rows of x [..., dh], the fp32 steps of the definition
    taken one by one (each numpy float32 operation rounds once)."""
    x = np.asarray(x, np.float32)
    a = np.abs(x)
    a = np.where(np.isnan(a), np.float32(0), a).max(-1)
    a = np.clip(a, np.float32(TINY), np.finfo(np.float32).max).astype(np.float32)
    inv = (np.float32(E4M3_MAX) / a).astype(np.float32)
    with np.errstate(invalid="ignore", over="ignore"):
        y = (x * inv[..., None]).astype(np.float32)
    return round_e4m3(y.astype(np.float64)), (a / np.float32(E4M3_MAX)).astype(np.float32)


# ----------------------------------------------------------------------------
# tree attention


def ancestors(parent, n) -> np.ndarray:
    """[n, n] truth values: node t sees node j (its ancestors and itself)."""
    see = np.zeros((n, n), bool)
    for t in range(n):
        j = t
        while j >= 0:
            see[t, j] = True
            j = int(parent[j]) if parent is not None else j - 1
    return see


def tree_attend(q, k, v, length, parent, n) -> tuple:
    """One sequence: q [T, Hq, dh], k and v [Hkv, N, dh] in float64.

    Returns (out [n, Hq, dh], bound [n, Hq, dh], sens [n, Hq]): the attention of nodes
    0..n-1; sum_s p_s |v_s| of each output; and max_s sum_d |q_d k_sd| / sqrt(dh), by which
    relative errors of the scores' products are scaled.  Slots a node does not see are
    never touched (they may hold anything)."""
    T, Hq, dh = q.shape
    g = Hq // k.shape[0]
    see = ancestors(parent, n)
    out = np.zeros((n, Hq, dh))
    bound = np.zeros((n, Hq, dh))
    sens = np.zeros((n, Hq))
    for t in range(n):
        slots = np.concatenate([np.arange(length), length + np.nonzero(see[t])[0]])
        for h in range(Hq):
            ks, vs = k[h // g, slots], v[h // g, slots]
            s = ks @ q[t, h] / np.sqrt(dh)
            p = np.exp(s - s.max())
            p /= p.sum()
            out[t, h] = p @ vs
            bound[t, h] = p @ np.abs(vs)
            sens[t, h] = (np.abs(ks) @ np.abs(q[t, h])).max() / np.sqrt(dh)
    return out, bound, sens


# ----------------------------------------------------------------------------
# verification


def draw(w, r) -> int:
    """The smallest v with cumsum(w)_v > r * sum(w); -1 where nothing has a weight."""
    w = np.where(np.asarray(w) > 0, w, 0.0)  # negative weights and NaN: 0
    c = np.cumsum(w)
    if not c[-1] > 0:
        return -1
    return int(np.argmax(c > r * c[-1]))


def chain_verify(target, draft, tok, n, u, r) -> tuple:
    """One sequence: (accepted, next token) of n drafts; target [T+1, V], draft [T, V]."""
    for i in range(n):
        x = int(tok[i])
        ok = 0 <= x < target.shape[1] and float(u[i]) * float(draft[i, x]) < float(target[i, x])
        if not ok:
            p, q = target[i].astype(np.float64), draft[i].astype(np.float64)
            v = draw(p - q, float(r))
            return i, v if v >= 0 else draw(p, float(r))
    return n, draw(target[n].astype(np.float64), float(r))


def tree_verify(target, tok, parent, n, u, r) -> tuple:
    """One sequence: (accepted nodes, next token) of a tree of n nodes; target [T, V]."""
    V = target.shape[1]
    kids = {t: [] for t in range(n)}
    for t in range(1, n):
        if 0 <= parent[t] < t and 0 <= tok[t] < V:
            kids[int(parent[t])].append(t)
    node, path = 0, []
    while True:
        run, seen, nxt = 0.0, set(), None
        for c in kids[node]:
            x = int(tok[c])
            if x not in seen:
                w = float(target[node, x])
                run += w if w > 0 else 0.0
                seen.add(x)
            if float(u[node]) < run:
                nxt = c
                break
        if nxt is None:
            break
        path.append(nxt)
        node = nxt
    w = target[node].astype(np.float64).copy()
    for c in kids[node]:
        w[int(tok[c])] = 0.0
    v = draw(w, float(r))
    return path, v if v >= 0 else draw(target[node].astype(np.float64), float(r))
