"""The operators of one speculative step over a KV cache, as they are measured.

  write / read      fdllm_cache_write_fp8, fdllm_cache_read_fp8: rows of k and v kept as
                    e4m3 with one fp32 scale per (sequence, head, slot), and read back
  attend            fdllm_tree_attend, fdllm_tree_attend_fp8: a tree of drafted tokens (one
                    token when T = 1) over a cache with a length per sequence and shared
                    key/value heads
  chain / tree      fdllm_chain_verify, fdllm_tree_verify: sampled acceptance of drafted
                    tokens from the target's probabilities and given random numbers

With `own` false, run() computes the operators' definitions in elementary torch operations;
with `own` true it makes the framework's calls.  exact() is the definition again, in 64 bits.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
E4M3 = torch.float8_e4m3fn
TINY = 2.0 ** -96  # the smallest absolute maximum a row's scale is made from


# ------------------------------------------------------------------------------- cases

def listed():
    return [
        # one token of one sequence: the append of a single-stream decode, where latency counts
        dict(name="write_one", op="write", B=1, N=1024, H=32, dh=128, R=1, dtype="bf16"),
        # a batch's prompt chunk: 64 sequences, 500 rows each, shared kv heads
        dict(name="write_chunk", op="write", B=64, N=4096, H=8, dh=128, R=500, dtype="bf16"),
        # the rows of one verify pass read back (8 sequences, 40 rows)
        dict(name="read_rows", op="read", B=8, N=2048, H=32, dh=128, R=40, dtype="bf16"),
        # a long cache read back whole (a migration, or a fallback to 16 bits)
        dict(name="read_long", op="read", B=1, N=16384, H=32, dh=128, R=16384, dtype="bf16"),
        # single-token decode of one sequence
        dict(name="attend_token", op="attend", B=1, N=1024, Hq=32, Hkv=32, dh=128, T=1, dtype="bf16",
             cache="bf16", low=1000, high=1000),
        # a verify batch with a drafted tree of 40 nodes, every sequence its own length
        dict(name="attend_tree", op="attend", B=8, N=2048, Hq=32, Hkv=32, dh=128, T=40, dtype="bf16",
             cache="bf16", low=1400, high=2000),
        # the largest: 64 sequences, 4096 slots, 32 nodes, no shared heads (4.3 GB of cache)
        dict(name="attend_batch", op="attend", B=64, N=4096, Hq=32, Hkv=32, dh=128, T=32, dtype="bf16",
             cache="bf16", low=4064, high=4064),
        # the long context in 8 bits, shared heads, a small tree of odd size
        dict(name="attend_long_fp8", op="attend", B=1, N=16384, Hq=32, Hkv=8, dh=128, T=13, dtype="bf16",
             cache="fp8", low=16001, high=16001),
        # a served batch in 8 bits, shared heads, ragged lengths
        dict(name="attend_batch_fp8", op="attend", B=64, N=4096, Hq=32, Hkv=8, dh=128, T=8, dtype="bf16",
             cache="fp8", low=1000, high=4080),
        # 5 drafts of a draft model for 8 sequences, full vocabulary
        dict(name="chain", op="chain", B=8, T=5, V=126464),
        # a served batch, full vocabulary
        dict(name="chain_batch", op="chain", B=64, T=4, V=126464),
        # a drafted tree of 40 nodes for 8 sequences
        dict(name="tree", op="tree", B=8, T=40, V=126464),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["write", "read", "attend", "attend", "attend", "chain", "tree"])
    if op in ("write", "read"):
        while True:
            c = dict(op=op, B=_log_int(rng, 1, 64), N=_log_int(rng, 64, 16384), H=rng.choice([1, 2, 4, 8, 12, 32]),
                     dh=rng.choice([64, 128]), R=_log_int(rng, 1, 2000), dtype=rng.choice(["bf16", "bf16", "f32"]))
            c["R"] = min(c["R"], c["N"])
            if c["B"] * c["N"] * c["H"] * c["dh"] <= 2 ** 28 and c["B"] * c["R"] * c["H"] * c["dh"] <= 2 ** 25:
                return c
    if op == "attend":
        while True:
            cache = rng.choice(["bf16", "bf16", "bf16", "fp8", "fp8", "fp8", "f32"])
            Hkv, g = rng.choice([1, 2, 4, 8, 16, 32]), rng.choice([1, 1, 2, 3, 4, 4, 7, 8])
            T = rng.choice([1, 1, _log_int(rng, 2, 128)])
            if cache == "f32":  # kept for small models and checks
                c = dict(op=op, B=_log_int(rng, 1, 4), N=_log_int(rng, 64, 1024), T=min(T, 16))
            else:
                c = dict(op=op, B=_log_int(rng, 1, 64), N=_log_int(rng, 64, 16384), T=T)
            high = c["N"] - c["T"]
            if high < 0:
                continue
            low = rng.choice([high, high // 2, 0])
            c |= dict(Hq=Hkv * g, Hkv=Hkv, dh=rng.choice([64, 128]), dtype="f32" if cache == "f32" else "bf16",
                      cache=cache, low=low, high=high)
            slots = c["B"] * c["N"] * Hkv * c["dh"]
            if slots <= 2 ** 29 and c["B"] * c["Hq"] * c["T"] * c["N"] <= 2 ** 28:
                return c
    while True:
        c = dict(op=op, B=_log_int(rng, 1, 64), T=_log_int(rng, 1, 64 if op == "tree" else 16),
                 V=_log_int(rng, 1000, 130000))
        if c["B"] * (c["T"] + 1) * c["V"] <= 2 ** 26:
            return c


def _lengths(c):
    """The sequences' lengths: spread over [low, high], the same for every seed."""
    span = c["high"] - c["low"] + 1
    return [c["low"] + (b * 2654435761 + 12345) % span for b in range(c["B"])]


def work(c):
    if c["op"] in ("write", "read"):
        rows = 2 * c["B"] * c["R"] * c["H"]
        return {"bytes": rows * (c["dh"] * (4 if c["dtype"] == "f32" else 2) + c["dh"] + 4) + 4 * c["B"] * c["R"],
                "flops": 2 * rows * c["dh"]}
    if c["op"] == "attend":
        elt = {"f32": 4, "bf16": 2, "fp8": 1}[c["cache"]]
        slots = sum(n + c["T"] for n in _lengths(c))
        qo = 2 * c["B"] * c["T"] * c["Hq"] * c["dh"] * (4 if c["dtype"] == "f32" else 2)
        row = c["dh"] * elt + (4 if c["cache"] == "fp8" else 0)
        return {"bytes": 2 * slots * c["Hkv"] * row + qo + 4 * c["B"] * (c["T"] + 1),
                "flops": 4 * slots * c["T"] * c["Hq"] * c["dh"]}
    rows = 2 if c["op"] == "chain" else 1
    return {"bytes": c["B"] * (rows * 4 * c["V"] + 20 * c["T"] + 8), "flops": c["B"] * rows * c["V"]}


# ------------------------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _trees(B, T, seed):
    """parent [B, T]: node 0 is the root; node t hangs below one of the 8 nodes before it."""
    r = np.random.default_rng(seed).random((B, T))
    t = np.arange(T)
    parent = t - 1 - np.floor(r * np.minimum(t, 8)).astype(np.int64)
    return torch.from_numpy(parent.astype(np.int32)).to(DEV)


def _rows_fp8(x):
    """The definition of the 8-bit rows: (e4m3 values, fp32 scale of each row)."""
    x = x.float()
    a = x.abs().amax(-1).clamp(TINY, torch.finfo(torch.float32).max)
    return (x * (448.0 / a)[..., None]).clamp(-448.0, 448.0).to(E4M3), a / 448.0


def prepare(c, seed):
    g = _gen(seed)
    rn = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    if c["op"] in ("write", "read"):
        B, N, H, dh, R, dt = c["B"], c["N"], c["H"], c["dh"], c["R"], DT[c["dtype"]]
        # contiguous runs of slots, each sequence at its own place, as appends come
        start = torch.randint(0, N - R + 1, (B, 1), generator=g, device=DEV)
        pos = (start + torch.arange(R, device=DEV)).to(torch.int32)
        # heads of different magnitude, as projections give them
        mag = torch.exp(rn(1, 1, H, 1))
        s = dict(c=c, pos=pos, k_rows=(rn(B, R, H, dh) * mag).to(dt), v_rows=(rn(B, R, H, dh) * mag).to(dt))
        for n in "kv":
            if c["op"] == "write":
                s[n + "_cache"] = torch.zeros((B, H, N, dh), dtype=E4M3, device=DEV)
                s[n + "_scale"] = torch.zeros((B, H, N), device=DEV)
            else:
                s[n + "_cache"] = torch.randint(-100, 101, (B, H, N, dh), generator=g, device=DEV,
                                                dtype=torch.int8).to(torch.float16).mul_(4).to(E4M3)
                s[n + "_scale"] = torch.exp(rn(B, H, N)) / 448.0
        return s
    if c["op"] == "attend":
        B, N, Hq, Hkv, dh, T = c["B"], c["N"], c["Hq"], c["Hkv"], c["dh"], c["T"]
        dt = DT[c["dtype"]]
        s = dict(c=c, q=(2.0 * rn(B, T, Hq, dh)).to(dt), parent=_trees(B, T, seed),
                 cache_len=torch.tensor(_lengths(c), dtype=torch.int32, device=DEV),
                 out=torch.empty((B, T, Hq * dh), dtype=dt, device=DEV))
        for n in "kv":
            full = torch.empty((B, Hkv, N, dh), dtype=E4M3 if c["cache"] == "fp8" else dt, device=DEV)
            scale = torch.empty((B, Hkv, N), device=DEV)
            for b in range(B):
                x = rn(Hkv, N, dh).to(dt)
                if c["cache"] == "fp8":
                    full[b], scale[b] = _rows_fp8(x)
                else:
                    full[b] = x
            s[n + "_cache"] = full
            if c["cache"] == "fp8":
                s[n + "_scale"] = scale
        return s
    B, T, V = c["B"], c["T"], c["V"]
    # peaked next-token distributions; a draft model that mostly agrees with the target
    logits = 3.0 * rn(B, T + 1 if c["op"] == "chain" else T, V)
    s = dict(c=c, target=torch.softmax(logits, -1))
    if c["op"] == "chain":
        s["draft"] = torch.softmax(logits[:, :T] + 0.5 * rn(B, T, V), -1)
        s["tok"] = torch.multinomial(s["draft"].reshape(B * T, V), 1, generator=g).reshape(B, T).to(torch.int32)
        s["u"] = torch.rand(B, T, generator=g, device=DEV)
    else:
        s["parent"] = _trees(B, T, seed)
        s["u"] = 0.2 * torch.rand(B, T, generator=g, device=DEV)
        # a node's token is one of the likeliest after its parent
        top = torch.topk(s["target"], 16 if V >= 16 else V, -1).indices
        par = s["parent"].clamp(min=0).long()
        pick = torch.arange(T, device=DEV) % top.shape[-1]
        s["tok"] = top[torch.arange(B, device=DEV)[:, None], par, pick[None, :]].to(torch.int32)
        s["path"] = torch.empty((B, T), dtype=torch.int32, device=DEV)
    s["r"] = torch.rand(B, generator=g, device=DEV)
    s["n_accept"] = torch.empty(B, dtype=torch.int32, device=DEV)
    s["next_tok"] = torch.empty(B, dtype=torch.int32, device=DEV)
    return s


# ------------------------------------------------------------------------------- one pass

def _workspace(s, nbytes):
    """Made at the first pass and kept, as a program keeps it."""
    if "ws" not in s:
        import kv_cache_attention_fdllm_b200 as F
        s["ws"] = F.alloc_workspace(nbytes(F), DEV)
    return s["ws"]


def run(s):
    if own:
        return _run_own(s)
    return {"write": _write, "read": _read, "attend": _attend, "chain": _chain, "tree": _tree}[s["c"]["op"]](s)


def _run_own(s):
    import kv_cache_attention_fdllm_b200 as F
    c = s["c"]
    if c["op"] == "write":
        ws = _workspace(s, lambda F: F.fdllm_cache_fp8_workspace_bytes(c["B"], c["R"]))
        F.fdllm_cache_write_fp8(s["k_rows"], s["v_rows"], s["pos"], s["k_cache"], s["v_cache"], s["k_scale"],
                                s["v_scale"], ws)
        return {n: s[n] for n in ("k_cache", "v_cache", "k_scale", "v_scale")}
    if c["op"] == "read":
        ws = _workspace(s, lambda F: F.fdllm_cache_fp8_workspace_bytes(c["B"], c["R"]))
        F.fdllm_cache_read_fp8(s["pos"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["k_rows"],
                               s["v_rows"], ws)
        return {"k": s["k_rows"], "v": s["v_rows"]}
    if c["op"] == "attend":
        ws = _workspace(s, lambda F: F.fdllm_tree_attend_workspace_bytes(
            c["B"], c["N"], c["Hq"], c["Hkv"], c["dh"], c["T"], DT[c["dtype"]]))
        if c["cache"] == "fp8":
            F.fdllm_tree_attend_fp8(s["q"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["cache_len"],
                                    s["parent"], None, s["out"], ws)
        else:
            F.fdllm_tree_attend(s["q"], s["k_cache"], s["v_cache"], s["cache_len"], s["parent"], None, s["out"], ws)
        return {"out": s["out"]}
    ws = _workspace(s, lambda F: F.fdllm_draft_verify_workspace_bytes(c["B"], c["T"], c["V"]))
    if c["op"] == "chain":
        F.fdllm_chain_verify(s["target"], s["draft"], s["tok"], None, s["u"], s["r"], s["n_accept"], s["next_tok"], ws)
        return {"n_accept": s["n_accept"], "next_tok": s["next_tok"]}
    F.fdllm_tree_verify(s["target"], s["tok"], s["parent"], None, s["u"], s["r"], s["path"], s["n_accept"],
                        s["next_tok"], ws)
    return {"path": s["path"], "n_accept": s["n_accept"], "next_tok": s["next_tok"]}


def _write(s):
    b = torch.arange(s["pos"].shape[0], device=DEV)[:, None]
    p = s["pos"].long()
    for n in "kv":
        q, scale = _rows_fp8(s[n + "_rows"])
        s[n + "_cache"].view(torch.uint8)[b, :, p] = q.view(torch.uint8)
        s[n + "_scale"][b, :, p] = scale
    return {n: s[n] for n in ("k_cache", "v_cache", "k_scale", "v_scale")}


def _read(s):
    b = torch.arange(s["pos"].shape[0], device=DEV)[:, None]
    p = s["pos"].long()
    got = {}
    for n in "kv":
        q = s[n + "_cache"].view(torch.uint8)[b, :, p].view(E4M3)
        got[n] = (q.float() * s[n + "_scale"][b, :, p][..., None]).to(s["k_rows"].dtype)
    return got


def _ancestors(parent):
    """[B, T, T] truth values: node t's ancestors and itself, by repeated squaring."""
    B, T = parent.shape
    t = torch.arange(T, device=DEV)
    m = ((parent[:, :, None] == t) | (t[:, None] == t)).float()
    for _ in range(max(1, (T - 1).bit_length())):
        m = (m @ m).clamp(max=1.0)
    return m > 0


def _attend(s):
    c = s["c"]
    B, N, Hq, Hkv, dh, T = c["B"], c["N"], c["Hq"], c["Hkv"], c["dh"], c["T"]
    g = Hq // Hkv
    k, v = s["k_cache"].float(), s["v_cache"].float()
    if c["cache"] == "fp8":
        k, v = k * s["k_scale"][..., None], v * s["v_scale"][..., None]
    q = s["q"].float().reshape(B, T, Hkv, g, dh).permute(0, 2, 1, 3, 4).reshape(B, Hkv, T * g, dh)
    sc = (q @ k.transpose(-1, -2)).reshape(B, Hkv, T, g, N) / math.sqrt(dh)
    slot = torch.arange(N, device=DEV)
    n = s["cache_len"].long()[:, None]
    node = slot - n                                                   # [B, N]: the tree node at a slot
    anc = torch.gather(_ancestors(s["parent"]), 2, node.clamp(0, T - 1)[:, None, :].expand(B, T, N))
    seen = (node < 0)[:, None, :] | (anc & (node < T)[:, None, :])     # [B, T, N]
    p = torch.softmax(sc.masked_fill_(~seen[:, None, :, None, :], -math.inf), -1)
    o = (p.reshape(B, Hkv, T * g, N) @ v).reshape(B, Hkv, T, g, dh).permute(0, 2, 1, 3, 4)
    return {"out": o.reshape(B, T, Hq * dh).to(s["q"].dtype)}


def _pick(w, r):
    """The smallest v with cumsum(w)_v > r * sum(w), in 64 bits."""
    cum = torch.cumsum(w, -1)
    v = torch.searchsorted(cum, (r.double() * cum[:, -1])[:, None], right=True)[:, 0]
    return v.clamp(max=w.shape[-1] - 1).to(torch.int32)


def _chain(s):
    tok = s["tok"].long()[..., None]
    B, T, V = s["draft"].shape
    p = torch.gather(s["target"][:, :T], 2, tok)[..., 0].double()
    q = torch.gather(s["draft"], 2, tok)[..., 0].double()
    n = torch.cumprod((s["u"].double() * q < p).to(torch.int32), 1).sum(1)
    b = torch.arange(B, device=DEV)
    rest = s["draft"][b, n.clamp(max=T - 1)].double() * (n < T)[:, None]
    w = (s["target"][b, n].double() - rest).clamp(min=0.0)
    return {"n_accept": n.to(torch.int32), "next_tok": _pick(w, s["r"])}


def _tree(s):
    B, T, V = s["target"].shape
    b = torch.arange(B, device=DEV)
    parent, tok = s["parent"].long(), s["tok"].long()
    t = torch.arange(T, device=DEV)
    # a sibling that repeats an earlier one's token adds nothing
    twin = (parent[:, :, None] == parent[:, None, :]) & (tok[:, :, None] == tok[:, None, :]) & (t[:, None] > t)
    p = s["target"][b[:, None], parent.clamp(min=0), tok].double() * ~twin.any(2)
    # every node's choice among its children: the first whose running sum exceeds the node's number
    child = (parent[:, None, :] == t[:, None]) & (t > 0)               # [B, node, child]
    hit = child & (s["u"].double()[..., None] < torch.cumsum(p[:, None, :] * child, 2))
    edge = hit & (torch.cumsum(hit, 2) == 1)
    # the accepted nodes are those that chosen edges join to node 0; a child's index exceeds its parent's
    m = (edge | (t[:, None] == t)).float()
    for _ in range(max(1, (T - 1).bit_length())):
        m = (m @ m).clamp(max=1.0)
    on = (m[:, 0] > 0) & (t > 0)
    n = on.sum(1)
    ranked = torch.where(on, t, T).sort(1).values
    path = torch.where(ranked < T, ranked, -1)
    node = torch.where(on, t, 0).amax(1)
    w = s["target"][b, node].double()
    kids = (parent == node[:, None]) & (t > 0)
    w[b[:, None].expand(B, T)[kids], tok[kids]] = 0.0
    return {"path": path.to(torch.int32), "n_accept": n.to(torch.int32), "next_tok": _pick(w, s["r"])}


# ------------------------------------------------------------------------------- in 64 bits

def _e4m3(x):
    """x (float64) rounded to the nearest e4m3 value, ties to even, within +-448."""
    x = x.clamp(-448.0, 448.0)
    e = torch.frexp(x.abs().clamp(min=2.0 ** -6)).exponent.double() - 1.0
    step = torch.exp2(e - 3.0)
    return torch.round(x / step) * step


def exact(c, seed):
    s = prepare(c, seed)
    if c["op"] == "write":
        got = {}
        for n in "kv":
            x = s[n + "_rows"].double()
            a = x.abs().amax(-1).clamp(TINY, float(torch.finfo(torch.float32).max))
            cache, scale = s[n + "_cache"].double(), s[n + "_scale"].double()
            for b in range(c["B"]):
                at = s["pos"][b].long()
                cache[b, :, at] = _e4m3(x[b] * (448.0 / a[b])[..., None]).transpose(0, 1)
                scale[b, :, at] = (a[b] / 448.0).transpose(0, 1)
            got[n + "_cache"], got[n + "_scale"] = cache, scale
        return got
    if c["op"] == "read":
        got = {}
        for n in "kv":
            got[n] = torch.stack([(s[n + "_cache"][b][:, s["pos"][b].long()].double()
                                   * s[n + "_scale"][b][:, s["pos"][b].long()].double()[..., None]).transpose(0, 1)
                                  for b in range(c["B"])])
        return got
    if c["op"] == "attend":
        T, Hq, Hkv, dh = c["T"], c["Hq"], c["Hkv"], c["dh"]
        parent = s["parent"].tolist()
        out = torch.empty((c["B"], T, Hq * dh), dtype=torch.float64, device=DEV)
        for b, n in enumerate(_lengths(c)):
            seen = torch.zeros((T, n + T), dtype=torch.bool)
            seen[:, :n] = True
            for t in range(T):
                a = t
                while a >= 0:
                    seen[t, n + a] = True
                    a = parent[b][a]
            k, v = s["k_cache"][b, :, :n + T].double(), s["v_cache"][b, :, :n + T].double()
            if c["cache"] == "fp8":
                k = k * s["k_scale"][b, :, :n + T, None].double()
                v = v * s["v_scale"][b, :, :n + T, None].double()
            q = s["q"][b].double().reshape(T, Hkv, Hq // Hkv, dh)
            x = torch.einsum("thgd,hsd->thgs", q, k) * dh ** -0.5
            x = x.masked_fill(~seen.to(DEV)[:, None, None, :], -math.inf)
            x = torch.exp(x - x.amax(-1, keepdim=True))
            o = torch.einsum("thgs,hsd->thgd", x, v) / x.sum(-1)[..., None]
            out[b] = o.reshape(T, Hq * dh)
        return {"out": out}
    return None  # whole numbers: the plain form's are the definition's, in 64 bits already
