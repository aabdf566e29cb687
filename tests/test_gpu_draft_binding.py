"""The binding of the calls for drafted tokens on CUDA tensors: what it refuses, and that its
short way (no stream argument) and its long one are the same call."""
import pytest
import torch

pytestmark = pytest.mark.gpu
E4M3 = torch.float8_e4m3fn


@pytest.fixture(scope="module")
def F():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import kv_cache_attention_fdllm_b200 as F
    return F


def calls(F):
    """name -> (function, arguments, names of those that may be None)."""
    g = torch.Generator(device="cuda").manual_seed(1)
    rn = lambda *s, dtype=torch.float32: torch.randn(*s, generator=g, device="cuda").to(dtype)  # noqa: E731
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")  # noqa: E731
    B, N, H, dh, T, V = 2, 40, 2, 64, 3, 50
    ws = F.alloc_workspace(max(F.fdllm_tree_attend_workspace_bytes(B, N, H, H, dh, T, torch.bfloat16),
                               F.fdllm_draft_verify_workspace_bytes(B, T, V)), "cuda")
    cache = dict(k_cache=rn(B, H, N, dh).to(E4M3), v_cache=rn(B, H, N, dh).to(E4M3),
                 k_scale=rn(B, H, N).abs(), v_scale=rn(B, H, N).abs())
    rows = dict(k_rows=rn(B, T, H, dh, dtype=torch.bfloat16), v_rows=rn(B, T, H, dh, dtype=torch.bfloat16))
    pos = torch.arange(T, dtype=torch.int32, device="cuda").repeat(B, 1)
    tree = dict(cache_len=i32(B) + 5, parent=i32(B, T) - 1, n_nodes=i32(B) + T,
                out=torch.zeros(B, T, H * dh, dtype=torch.bfloat16, device="cuda"), workspace=ws)
    q = rn(B, T, H, dh, dtype=torch.bfloat16)
    prob = torch.softmax(rn(B, T + 1, V), -1)
    draft = torch.softmax(rn(B, T, V), -1)
    end = dict(n_accept=i32(B), next_tok=i32(B), workspace=ws)
    u, r = torch.rand(B, T, generator=g, device="cuda"), torch.rand(B, generator=g, device="cuda")
    par = i32(B, T)
    return {
        "write": (F.fdllm_cache_write_fp8, dict(**rows, pos=pos, **cache, workspace=ws)),
        "read": (F.fdllm_cache_read_fp8, dict(pos=pos, **cache, **rows, workspace=ws)),
        "attend": (F.fdllm_tree_attend, dict(q=q, k_cache=rn(B, H, N, dh, dtype=torch.bfloat16),
                                             v_cache=rn(B, H, N, dh, dtype=torch.bfloat16), **tree)),
        "attend_fp8": (F.fdllm_tree_attend_fp8, dict(q=q, **cache, **tree)),
        "chain": (F.fdllm_chain_verify, dict(target=prob, draft=draft, tok=i32(B, T), n_draft=i32(B) + T, u=u, r=r, **end)),
        "tree": (F.fdllm_tree_verify, dict(target=draft, tok=i32(B, T), parent=par, n_nodes=i32(B) + T, u=u, r=r,
                                           path=i32(B, T), **end)),
    }


NAMES = ["write", "read", "attend", "attend_fp8", "chain", "tree"]
MAY_BE_NONE = {"parent", "n_nodes", "n_draft"}


@pytest.mark.parametrize("name", NAMES)
def test_every_argument_is_checked(F, name):
    f, args = calls(F)[name]
    f(**args)
    for key, t in args.items():
        for what, bad in [
                ("not a tensor", 3.5), ("no tensor", None), ("on the CPU", t.cpu()),
                ("another type", t.to(torch.float64) if t.dtype != torch.float64 else t.float()),
                ("another shape", torch.cat([t, t])), ("fewer dimensions", t.flatten()),
                ("not contiguous", torch.stack([t, t], -1)[..., 0])]:
            if what in ("no tensor",) and key in MAY_BE_NONE and not (name == "tree" and key == "parent"):
                continue
            if key == "workspace" and what in ("another shape", "fewer dimensions"):
                continue
            if t.dim() == 1 and what == "fewer dimensions":
                continue
            with pytest.raises((TypeError, ValueError)):
                f(**{**args, key: bad})
    torch.cuda.synchronize()
    assert F.fdllm_get_status(args["workspace"]) == F.OK


@pytest.mark.parametrize("name", NAMES)
def test_library_errors_are_raised(F, name):
    f, args = calls(F)[name]
    with pytest.raises(F.FdllmError) as e:
        f(**{**args, "workspace": args["workspace"][:128]})
    assert e.value.status == F.ERR_WORKSPACE
    odd = torch.zeros(args["workspace"].numel() + 1, dtype=torch.uint8, device="cuda")[1:]
    with pytest.raises(F.FdllmError) as e:
        f(**{**args, "workspace": odd})
    assert e.value.status == F.ERR_WORKSPACE


@pytest.mark.parametrize("name", NAMES)
def test_both_ways_are_the_same_call(F, name):
    """With a stream and without, and on whichever stream is the current one."""
    outs = []
    for how in ("current", "given", "made current"):
        f, args = calls(F)[name]
        torch.cuda.synchronize()
        s = torch.cuda.Stream()
        if how == "current":
            f(**args)
        elif how == "given":
            f(**args, stream=s)
        else:
            with torch.cuda.stream(s):
                graph = torch.cuda.CUDAGraph()  # only what runs on the current stream is captured
                with torch.cuda.graph(graph, stream=s):
                    f(**args)
            graph.replay()
        torch.cuda.synchronize()
        outs.append([v.view(torch.uint8).clone() for k, v in args.items() if v is not None and k != "workspace"])
    for other in outs[1:]:
        for a, b in zip(outs[0], other):
            assert torch.equal(a, b)
