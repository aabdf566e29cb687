"""Python binding of the fdllm C ABI: argument marshalling only.

Each function has the name of the C entry point it calls (include/fdllm.h),
takes torch CUDA tensors, checks their dtype, shape, device and contiguity,
passes raw pointers and the current CUDA stream, and raises FdllmError on a
non-OK status.  The library launches on the current CUDA device, so the tensors
and the stream must be on it (a ValueError otherwise).  Every step of the
computation runs in the CUDA library.  The calls for drafted tokens, where host
time counts, are checked and made in C++ when they fit (_fast); what does not
fit comes back to the checks here, which say why.  Without _fast.so all of them
go through the checks here.
"""
from __future__ import annotations

import ctypes
import warnings

import torch

from ._native import lib

try:
    from . import _fast
    if _fast.torch_version != torch.__version__.split("+")[0]:
        raise ImportError(f"it was built for torch {_fast.torch_version}")
except ImportError as e:
    # every call works without it, those for drafted tokens with 6 us more of host time
    _fast = None
    warnings.warn("_fast.so is missing or was built for another torch, calls for drafted tokens take "
                  f"the slower way: build it with `python kv_cache_attention_fdllm_b200/build.py` ({e})",
                  RuntimeWarning)

OK, ERR_INVALID_ARG, ERR_UNSUPPORTED, ERR_CUDA, ERR_BAD_INDEX, ERR_TIMEOUT, ERR_WORKSPACE = range(7)
FLAG_COMMIT, FLAG_ACCEPT, FLAG_PASS = 1, 2, 4
_DT = {torch.float32: 0, torch.bfloat16: 1}


class FdllmError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        msg = lib().fdllm_status_string(status).decode()
        super().__init__(f"{where}: {msg} (status {status})")


def _check(st: int, where: str):
    if st != OK:
        raise FdllmError(st, where)


def _p(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else ctypes.c_void_p(0)


def _stream(stream, device):
    """The stream handle to launch on.  The library launches on the current CUDA
    device, so the tensors (on `device`) and the stream must both be on it."""
    if device.type != "cuda":
        raise ValueError(f"the tensors are on {device}, not on a CUDA device")
    cur = torch.cuda.current_device()
    if device.index != cur:
        raise ValueError(f"the tensors are on {device}, but the current CUDA device is "
                         f"cuda:{cur} (use torch.cuda.set_device)")
    s = torch.cuda.current_stream(device) if stream is None else stream
    if s.device != device:
        raise ValueError(f"the stream is on {s.device}, the tensors on {device}")
    return ctypes.c_void_p(s.cuda_stream)


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream_on(stream, device):
    """_stream for calls whose host time counts: the current stream's handle, without the
    2 us that a torch.cuda.Stream object takes, where there is nothing to refuse."""
    if stream is None and _raw_stream is not None and device.index == torch.cuda.current_device():
        return _raw_stream(device.index)
    return _stream(stream, device)


def _at(t):
    """The address of a tensor's data, None for no tensor."""
    return None if t is None else t.data_ptr()


def _need(t, name, dtype=None, shape=None, device=None):
    # one look at a tensor that fits (torch.Size compares with tuples); the cause otherwise
    if (isinstance(t, torch.Tensor) and t.is_cuda and t.is_contiguous()
            and (dtype is None or t.dtype == dtype) and (shape is None or t.shape == shape)
            and (device is None or t.device == device)):
        return
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")


def _dims(t, name, n):
    if t.dim() != n:
        raise ValueError(f"{name} must have {n} dimensions, got {tuple(t.shape)}")


def _dtype_code(t):
    if t.dtype not in _DT:
        raise ValueError(f"unsupported storage dtype {t.dtype}")
    return _DT[t.dtype]


# ---------------------------------------------------------------- workspace sizes

def fdllm_fused_step_workspace_bytes(B, N, D, H, dh, nq, dtype) -> int:
    return int(lib().fdllm_fused_step_workspace_bytes(B, N, D, H, dh, nq, _DT.get(dtype, dtype)))


def fdllm_verify_step_workspace_bytes(B, N, D, H, dh, R, S_max, dtype) -> int:
    return int(lib().fdllm_verify_step_workspace_bytes(B, N, D, H, dh, R, S_max,
                                                       _DT.get(dtype, dtype)))


def fdllm_accept_workspace_bytes(B, R, V) -> int:
    return int(lib().fdllm_accept_workspace_bytes(B, R, V))


def alloc_workspace(nbytes: int, device) -> torch.Tensor:
    """A zero-filled workspace of nbytes (the library requires zeros before first use)."""
    return torch.zeros(max(int(nbytes), 256), dtype=torch.uint8, device=device)


# ---------------------------------------------------------------- fused step

def _fused_shapes(x, q_idx, w_qkv, k_cache):
    B, N, D = x.shape
    nq = q_idx.shape[1]
    H, dh = k_cache.shape[1], k_cache.shape[3]
    return B, N, D, H, dh, nq


def _check_fused(x, q_idx, w_qkv, k_cache, v_cache):
    _need(x, "x")
    B, N, D, H, dh, nq = _fused_shapes(x, q_idx, w_qkv, k_cache)
    dt, dev = x.dtype, x.device
    _need(q_idx, "q_idx", torch.int32, (B, nq), dev)
    _need(w_qkv, "w_qkv", dt, (3 * H * dh, D), dev)
    _need(k_cache, "k_cache", dt, (B, H, N, dh), dev)
    _need(v_cache, "v_cache", dt, (B, H, N, dh), dev)
    return B, N, D, H, dh, nq


def fdllm_fused_step(x, q_idx, w_qkv, k_cache, v_cache, out, workspace, rope_base=10000.0,
                     stream=None):
    """One fused KV-cache step (see include/fdllm.h); k_cache/v_cache are updated in place."""
    B, N, D, H, dh, nq = _check_fused(x, q_idx, w_qkv, k_cache, v_cache)
    _need(out, "out", x.dtype, (B, nq, H * dh), x.device)
    _need(workspace, "workspace", torch.uint8, None, x.device)
    st = lib().fdllm_fused_step(B, N, D, H, dh, nq, _dtype_code(x), _p(x), _p(q_idx), _p(w_qkv),
                                float(rope_base), _p(k_cache), _p(v_cache), _p(out),
                                _p(workspace), workspace.numel(), _stream(stream, x.device))
    _check(st, "fdllm_fused_step")
    return out


def fdllm_fused_step_rows(x_rows, q_idx, w_qkv, k_cache, v_cache, out, workspace,
                          rope_base=10000.0, stream=None):
    """fdllm_fused_step with the rows x[Q] given packed, x_rows [B, nq, D]."""
    _need(x_rows, "x_rows")
    B, nq, D = x_rows.shape
    _need(k_cache, "k_cache")
    H, N, dh = k_cache.shape[1], k_cache.shape[2], k_cache.shape[3]
    dt, dev = x_rows.dtype, x_rows.device
    _need(q_idx, "q_idx", torch.int32, (B, nq), dev)
    _need(w_qkv, "w_qkv", dt, (3 * H * dh, D), dev)
    _need(k_cache, "k_cache", dt, (B, H, N, dh), dev)
    _need(v_cache, "v_cache", dt, (B, H, N, dh), dev)
    _need(out, "out", dt, (B, nq, H * dh), dev)
    _need(workspace, "workspace", torch.uint8, None, dev)
    st = lib().fdllm_fused_step_rows(B, N, D, H, dh, nq, _dtype_code(x_rows), _p(x_rows),
                                     _p(q_idx), _p(w_qkv), float(rope_base), _p(k_cache),
                                     _p(v_cache), _p(out), _p(workspace), workspace.numel(),
                                     _stream(stream, dev))
    _check(st, "fdllm_fused_step_rows")
    return out


def fdllm_qkv_rope_scatter(x, q_idx, w_qkv, k_cache, v_cache, q_out, workspace,
                           rope_base=10000.0, stream=None):
    B, N, D, H, dh, nq = _check_fused(x, q_idx, w_qkv, k_cache, v_cache)
    _need(q_out, "q_out", x.dtype, (B, nq, H, dh), x.device)
    _need(workspace, "workspace", torch.uint8, None, x.device)
    st = lib().fdllm_qkv_rope_scatter(B, N, D, H, dh, nq, _dtype_code(x), _p(x), _p(q_idx),
                                      _p(w_qkv), float(rope_base), _p(k_cache), _p(v_cache),
                                      _p(q_out), _p(workspace), workspace.numel(),
                                      _stream(stream, x.device))
    _check(st, "fdllm_qkv_rope_scatter")
    return q_out


def fdllm_attend(q, k_cache, v_cache, out, workspace, stream=None):
    _need(q, "q")
    B, nq, H, dh = q.shape
    N = k_cache.shape[2]
    _need(k_cache, "k_cache", q.dtype, (B, H, N, dh), q.device)
    _need(v_cache, "v_cache", q.dtype, (B, H, N, dh), q.device)
    _need(out, "out", q.dtype, (B, nq, H * dh), q.device)
    _need(workspace, "workspace", torch.uint8, None, q.device)
    st = lib().fdllm_attend(B, N, H, dh, nq, _dtype_code(q), _p(q), _p(k_cache), _p(v_cache),
                            _p(out), _p(workspace), workspace.numel(), _stream(stream, q.device))
    _check(st, "fdllm_attend")
    return out


# ---------------------------------------------------------------- verify pass

def _check_verify(x_rows, pos, view, w_qkv, k_cache, v_cache, k_side, v_side):
    _need(x_rows, "x_rows")
    B, R, D = x_rows.shape
    H, N, dh = k_cache.shape[1], k_cache.shape[2], k_cache.shape[3]
    dt, dev = x_rows.dtype, x_rows.device
    _need(pos, "pos", torch.int32, (B, R), dev)
    _need(view, "view", torch.int8, (B, R), dev)
    _need(w_qkv, "w_qkv", dt, (3 * H * dh, D), dev)
    _need(k_cache, "k_cache", dt, (B, H, N, dh), dev)
    _need(v_cache, "v_cache", dt, (B, H, N, dh), dev)
    S_max = k_side.shape[2]
    _need(k_side, "k_side", dt, (B, H, S_max, dh), dev)
    _need(v_side, "v_side", dt, (B, H, S_max, dh), dev)
    return B, N, D, H, dh, R, S_max


def fdllm_verify_step(x_rows, pos, view, rank, w_qkv, k_cache, v_cache, k_side, v_side, out,
                      workspace, rope_base=10000.0, causal_cross=False, stream=None):
    """One Flash-Verify pass (see include/fdllm.h); caches and side buffers updated in place."""
    B, N, D, H, dh, R, S_max = _check_verify(x_rows, pos, view, w_qkv, k_cache, v_cache, k_side,
                                             v_side)
    _need(rank, "rank", torch.int32, (B, R), x_rows.device)
    _need(out, "out", x_rows.dtype, (B, R, H * dh), x_rows.device)
    _need(workspace, "workspace", torch.uint8, None, x_rows.device)
    st = lib().fdllm_verify_step(B, N, D, H, dh, R, S_max, _dtype_code(x_rows), _p(x_rows),
                                 _p(pos), _p(view), _p(rank), _p(w_qkv), float(rope_base),
                                 _p(k_cache), _p(v_cache), _p(k_side), _p(v_side), _p(out),
                                 int(bool(causal_cross)), _p(workspace), workspace.numel(),
                                 _stream(stream, x_rows.device))
    _check(st, "fdllm_verify_step")
    return out


def fdllm_verify_qkv_rope_scatter(x_rows, pos, view, w_qkv, k_cache, v_cache, k_side, v_side,
                                  q_out, workspace, rope_base=10000.0, stream=None):
    B, N, D, H, dh, R, S_max = _check_verify(x_rows, pos, view, w_qkv, k_cache, v_cache, k_side,
                                             v_side)
    _need(q_out, "q_out", x_rows.dtype, (B, R, H, dh), x_rows.device)
    _need(workspace, "workspace", torch.uint8, None, x_rows.device)
    st = lib().fdllm_verify_qkv_rope_scatter(B, N, D, H, dh, R, S_max, _dtype_code(x_rows),
                                             _p(x_rows), _p(pos), _p(view), _p(w_qkv),
                                             float(rope_base), _p(k_cache), _p(v_cache),
                                             _p(k_side), _p(v_side), _p(q_out), _p(workspace),
                                             workspace.numel(), _stream(stream, x_rows.device))
    _check(st, "fdllm_verify_qkv_rope_scatter")
    return q_out


def fdllm_verify_attend(q, pos, view, rank, k_cache, v_cache, k_side, v_side, out, workspace,
                        causal_cross=False, stream=None):
    _need(q, "q")
    B, R, H, dh = q.shape
    N = k_cache.shape[2]
    S_max = k_side.shape[2]
    dev, dt = q.device, q.dtype
    _need(pos, "pos", torch.int32, (B, R), dev)
    _need(view, "view", torch.int8, (B, R), dev)
    _need(rank, "rank", torch.int32, (B, R), dev)
    _need(k_cache, "k_cache", dt, (B, H, N, dh), dev)
    _need(v_cache, "v_cache", dt, (B, H, N, dh), dev)
    _need(k_side, "k_side", dt, (B, H, S_max, dh), dev)
    _need(v_side, "v_side", dt, (B, H, S_max, dh), dev)
    _need(out, "out", dt, (B, R, H * dh), dev)
    _need(workspace, "workspace", torch.uint8, None, dev)
    st = lib().fdllm_verify_attend(B, N, H, dh, R, S_max, _dtype_code(q), _p(q), _p(pos),
                                   _p(view), _p(rank), _p(k_cache), _p(v_cache), _p(k_side),
                                   _p(v_side), _p(out), int(bool(causal_cross)), _p(workspace),
                                   workspace.numel(), _stream(stream, dev))
    _check(st, "fdllm_verify_attend")
    return out


# ---------------------------------------------------------------- acceptance

def fdllm_track_select(q_masked, candidate, k_cache, track, workspace, mass=None, dtype=None,
                       stream=None):
    """The next tracked set from the last fused step on `workspace` (see include/fdllm.h).

    q_masked int8 [B, nq], candidate int8 [B, N], k_cache [B, H, N, dh] as the
    step left it, track int32 [B, beta_t] (out), mass float32 [B, N] (out, optional)."""
    _need(q_masked, "q_masked", torch.int8)
    B, nq = q_masked.shape
    _need(k_cache, "k_cache")
    _, H, N, dh = k_cache.shape
    dev = k_cache.device
    _need(q_masked, "q_masked", torch.int8, (B, nq), dev)
    _need(candidate, "candidate", torch.int8, (B, N), dev)
    _need(track, "track", torch.int32, None, dev)
    if track.dim() != 2 or track.shape[0] != B:
        raise ValueError(f"track must be [B, beta_t] with B={B}, got {tuple(track.shape)}")
    if mass is not None:
        _need(mass, "mass", torch.float32, (B, N), dev)
    _need(workspace, "workspace", torch.uint8, None, dev)
    st = lib().fdllm_track_select(B, N, H, dh, nq, _dtype_code(k_cache), _p(q_masked),
                                  _p(candidate), _p(k_cache), track.shape[1], _p(track), _p(mass),
                                  _p(workspace), workspace.numel(), _stream(stream, dev))
    _check(st, "fdllm_track_select")
    return track, mass


def fdllm_accept(logits, kind, ref_tok, rank, top1, conf, flags, n_accept, workspace, eps=0.9,
                 gamma=0.8, stream=None):
    """Top-1, confidence, epsilon split and gamma prefix acceptance (see include/fdllm.h)."""
    _need(logits, "logits", torch.float32)
    B, R, V = logits.shape
    dev = logits.device
    _need(kind, "kind", torch.int8, (B, R), dev)
    if ref_tok is not None:
        _need(ref_tok, "ref_tok", torch.int32, (B, R), dev)
    if rank is not None:
        _need(rank, "rank", torch.int32, (B, R), dev)
    _need(top1, "top1", torch.int32, (B, R), dev)
    _need(conf, "conf", torch.float32, (B, R), dev)
    _need(flags, "flags", torch.uint8, (B, R), dev)
    _need(n_accept, "n_accept", torch.int32, (B,), dev)
    _need(workspace, "workspace", torch.uint8, None, dev)
    st = lib().fdllm_accept(B, R, V, _p(logits), _p(kind), _p(ref_tok), _p(rank), float(eps),
                            float(gamma), _p(top1), _p(conf), _p(flags), _p(n_accept),
                            _p(workspace), workspace.numel(), _stream(stream, dev))
    _check(st, "fdllm_accept")
    return top1, conf, flags, n_accept


def fdllm_accept_noalloc(logits, kind, ref_tok, rank, top1, conf, flags, n_accept, eps=0.9,
                         gamma=0.8, stream=None):
    """fdllm_accept without a workspace, for callers that cannot allocate device
    memory where they call the library (see include/fdllm.h): the scratch is a
    fixed device array inside the library, shared by every call on a device."""
    _need(logits, "logits", torch.float32)
    B, R, V = logits.shape
    dev = logits.device
    _need(kind, "kind", torch.int8, (B, R), dev)
    if ref_tok is not None:
        _need(ref_tok, "ref_tok", torch.int32, (B, R), dev)
    if rank is not None:
        _need(rank, "rank", torch.int32, (B, R), dev)
    _need(top1, "top1", torch.int32, (B, R), dev)
    _need(conf, "conf", torch.float32, (B, R), dev)
    _need(flags, "flags", torch.uint8, (B, R), dev)
    _need(n_accept, "n_accept", torch.int32, (B,), dev)
    st = lib().fdllm_accept_noalloc(B, R, V, _p(logits), _p(kind), _p(ref_tok), _p(rank),
                                    float(eps), float(gamma), _p(top1), _p(conf), _p(flags),
                                    _p(n_accept), _stream(stream, dev))
    _check(st, "fdllm_accept_noalloc")
    return top1, conf, flags, n_accept


# ---------------------------------------------------------------- drafted tokens over a cache

def fdllm_cache_fp8_workspace_bytes(B, R) -> int:
    return int(lib().fdllm_cache_fp8_workspace_bytes(B, R))


def fdllm_tree_attend_workspace_bytes(B, N, Hq, Hkv, dh, T, dtype) -> int:
    return int(lib().fdllm_tree_attend_workspace_bytes(B, N, Hq, Hkv, dh, T,
                                                       _DT.get(dtype, dtype)))


def fdllm_draft_verify_workspace_bytes(B, T, V) -> int:
    return int(lib().fdllm_draft_verify_workspace_bytes(B, T, V))


def _check_fp8(k_rows, v_rows, pos, k_cache, v_cache, k_scale, v_scale, workspace):
    _need(k_rows, "k_rows")
    _dims(k_rows, "k_rows", 4)
    B, R, H, dh = k_rows.shape
    dev = k_rows.device
    _need(v_rows, "v_rows", k_rows.dtype, (B, R, H, dh), dev)
    _need(pos, "pos", torch.int32, (B, R), dev)
    _need(k_cache, "k_cache", torch.float8_e4m3fn)
    _dims(k_cache, "k_cache", 4)
    N = k_cache.shape[2]
    _need(k_cache, "k_cache", torch.float8_e4m3fn, (B, H, N, dh), dev)
    _need(v_cache, "v_cache", torch.float8_e4m3fn, (B, H, N, dh), dev)
    _need(k_scale, "k_scale", torch.float32, (B, H, N), dev)
    _need(v_scale, "v_scale", torch.float32, (B, H, N), dev)
    _need(workspace, "workspace", torch.uint8, None, dev)
    return B, N, H, dh, R


def fdllm_cache_write_fp8(k_rows, v_rows, pos, k_cache, v_cache, k_scale, v_scale, workspace,
                          stream=None):
    """Rows of k and v quantised into an 8-bit cache at pos (see include/fdllm.h).

    k_rows, v_rows [B, R, H, dh]; pos int32 [B, R], -1 skips a row; the caches
    float8_e4m3fn [B, H, N, dh] with float32 scales [B, H, N], updated in place."""
    if stream is None and _fast is not None:
        st = _fast.cache_write_fp8(k_rows, v_rows, pos, k_cache, v_cache, k_scale, v_scale, workspace)
        if st >= 0:
            _check(st, "fdllm_cache_write_fp8")
            return
    B, N, H, dh, R = _check_fp8(k_rows, v_rows, pos, k_cache, v_cache, k_scale, v_scale, workspace)
    st = lib().fdllm_cache_write_fp8(B, N, H, dh, R, _dtype_code(k_rows), _at(k_rows), _at(v_rows),
                                     _at(pos), _at(k_cache), _at(v_cache), _at(k_scale), _at(v_scale),
                                     _at(workspace), workspace.numel(),
                                     _stream_on(stream, k_rows.device))
    _check(st, "fdllm_cache_write_fp8")


def fdllm_cache_read_fp8(pos, k_cache, v_cache, k_scale, v_scale, k_rows, v_rows, workspace,
                         stream=None):
    """Rows of an 8-bit cache read back into k_rows, v_rows [B, R, H, dh] (see include/fdllm.h)."""
    if stream is None and _fast is not None:
        st = _fast.cache_read_fp8(k_rows, v_rows, pos, k_cache, v_cache, k_scale, v_scale, workspace)
        if st >= 0:
            _check(st, "fdllm_cache_read_fp8")
            return k_rows, v_rows
    B, N, H, dh, R = _check_fp8(k_rows, v_rows, pos, k_cache, v_cache, k_scale, v_scale, workspace)
    st = lib().fdllm_cache_read_fp8(B, N, H, dh, R, _dtype_code(k_rows), _at(pos), _at(k_cache),
                                    _at(v_cache), _at(k_scale), _at(v_scale), _at(k_rows), _at(v_rows),
                                    _at(workspace), workspace.numel(),
                                    _stream_on(stream, k_rows.device))
    _check(st, "fdllm_cache_read_fp8")
    return k_rows, v_rows


def _check_tree(q, k_cache, v_cache, cache_dtype, cache_len, parent, n_nodes, out, workspace):
    _need(q, "q")
    _dims(q, "q", 4)
    B, T, Hq, dh = q.shape
    dev = q.device
    _need(k_cache, "k_cache", cache_dtype)
    _dims(k_cache, "k_cache", 4)
    Hkv, N = k_cache.shape[1], k_cache.shape[2]
    _need(k_cache, "k_cache", cache_dtype, (B, Hkv, N, dh), dev)
    _need(v_cache, "v_cache", cache_dtype, (B, Hkv, N, dh), dev)
    _need(cache_len, "cache_len", torch.int32, (B,), dev)
    if parent is not None:
        _need(parent, "parent", torch.int32, (B, T), dev)
    if n_nodes is not None:
        _need(n_nodes, "n_nodes", torch.int32, (B,), dev)
    _need(out, "out", q.dtype, (B, T, Hq * dh), dev)
    _need(workspace, "workspace", torch.uint8, None, dev)
    return B, N, Hq, Hkv, dh, T


def fdllm_tree_attend(q, k_cache, v_cache, cache_len, parent, n_nodes, out, workspace,
                      stream=None):
    """Attention of a tree of drafted tokens over a cache (see include/fdllm.h).

    q [B, T, Hq, dh]; caches [B, Hkv, N, dh]; cache_len int32 [B]; parent int32
    [B, T] or None (a chain); n_nodes int32 [B] or None (T); out [B, T, Hq*dh]."""
    if stream is None and _fast is not None:
        st = _fast.tree_attend(q, k_cache, v_cache, cache_len, parent, n_nodes, out, workspace)
        if st >= 0:
            _check(st, "fdllm_tree_attend")
            return out
    B, N, Hq, Hkv, dh, T = _check_tree(q, k_cache, v_cache, getattr(q, "dtype", None), cache_len,
                                       parent, n_nodes, out, workspace)
    st = lib().fdllm_tree_attend(B, N, Hq, Hkv, dh, T, _dtype_code(q), _at(q), _at(k_cache),
                                 _at(v_cache), _at(cache_len), _at(parent), _at(n_nodes), _at(out),
                                 _at(workspace), workspace.numel(), _stream_on(stream, q.device))
    _check(st, "fdllm_tree_attend")
    return out


def fdllm_tree_attend_fp8(q, k_cache, v_cache, k_scale, v_scale, cache_len, parent, n_nodes, out,
                          workspace, stream=None):
    """fdllm_tree_attend over an 8-bit cache (float8_e4m3fn, float32 scales [B, Hkv, N])."""
    if stream is None and _fast is not None:
        st = _fast.tree_attend_fp8(q, k_cache, v_cache, k_scale, v_scale, cache_len, parent,
                    n_nodes, out, workspace)
        if st >= 0:
            _check(st, "fdllm_tree_attend_fp8")
            return out
    B, N, Hq, Hkv, dh, T = _check_tree(q, k_cache, v_cache, torch.float8_e4m3fn, cache_len, parent,
                                       n_nodes, out, workspace)
    _need(k_scale, "k_scale", torch.float32, (B, Hkv, N), q.device)
    _need(v_scale, "v_scale", torch.float32, (B, Hkv, N), q.device)
    st = lib().fdllm_tree_attend_fp8(B, N, Hq, Hkv, dh, T, _dtype_code(q), _at(q), _at(k_cache),
                                     _at(v_cache), _at(k_scale), _at(v_scale), _at(cache_len),
                                     _at(parent), _at(n_nodes), _at(out), _at(workspace),
                                     workspace.numel(), _stream_on(stream, q.device))
    _check(st, "fdllm_tree_attend_fp8")
    return out


def fdllm_chain_verify(target, draft, tok, n_draft, u, r, n_accept, next_tok, workspace,
                       stream=None):
    """Sampled acceptance of a drafted chain (see include/fdllm.h).

    target float32 [B, T+1, V], draft float32 [B, T, V], tok int32 [B, T], n_draft
    int32 [B] or None (T), u float32 [B, T], r float32 [B]; n_accept, next_tok
    int32 [B] (out)."""
    if stream is None and _fast is not None:
        st = _fast.chain_verify(target, draft, tok, n_draft, u, r, n_accept, next_tok, workspace)
        if st >= 0:
            _check(st, "fdllm_chain_verify")
            return n_accept, next_tok
    _need(target, "target", torch.float32)
    _dims(target, "target", 3)
    _need(draft, "draft", torch.float32)
    _dims(draft, "draft", 3)
    B, T, V = draft.shape
    dev = target.device
    _need(target, "target", torch.float32, (B, T + 1, V))
    _need(draft, "draft", torch.float32, (B, T, V), dev)
    _need(tok, "tok", torch.int32, (B, T), dev)
    if n_draft is not None:
        _need(n_draft, "n_draft", torch.int32, (B,), dev)
    _need(u, "u", torch.float32, (B, T), dev)
    _need(r, "r", torch.float32, (B,), dev)
    _need(n_accept, "n_accept", torch.int32, (B,), dev)
    _need(next_tok, "next_tok", torch.int32, (B,), dev)
    _need(workspace, "workspace", torch.uint8, None, dev)
    st = lib().fdllm_chain_verify(B, T, V, _at(target), _at(draft), _at(tok), _at(n_draft), _at(u),
                                  _at(r), _at(n_accept), _at(next_tok), _at(workspace),
                                  workspace.numel(), _stream_on(stream, dev))
    _check(st, "fdllm_chain_verify")
    return n_accept, next_tok


def fdllm_tree_verify(target, tok, parent, n_nodes, u, r, path, n_accept, next_tok, workspace,
                      stream=None):
    """Sampled acceptance along a drafted tree (see include/fdllm.h).

    target float32 [B, T, V], tok and parent int32 [B, T], n_nodes int32 [B] or
    None (T), u float32 [B, T], r float32 [B]; path int32 [B, T], n_accept and
    next_tok int32 [B] (out)."""
    if stream is None and _fast is not None:
        st = _fast.tree_verify(target, tok, parent, n_nodes, u, r, path, n_accept, next_tok,
                    workspace)
        if st >= 0:
            _check(st, "fdllm_tree_verify")
            return path, n_accept, next_tok
    _need(target, "target", torch.float32)
    _dims(target, "target", 3)
    B, T, V = target.shape
    dev = target.device
    _need(tok, "tok", torch.int32, (B, T), dev)
    _need(parent, "parent", torch.int32, (B, T), dev)
    if n_nodes is not None:
        _need(n_nodes, "n_nodes", torch.int32, (B,), dev)
    _need(u, "u", torch.float32, (B, T), dev)
    _need(r, "r", torch.float32, (B,), dev)
    _need(path, "path", torch.int32, (B, T), dev)
    _need(n_accept, "n_accept", torch.int32, (B,), dev)
    _need(next_tok, "next_tok", torch.int32, (B,), dev)
    _need(workspace, "workspace", torch.uint8, None, dev)
    st = lib().fdllm_tree_verify(B, T, V, _at(target), _at(tok), _at(parent), _at(n_nodes), _at(u),
                                 _at(r), _at(path), _at(n_accept), _at(next_tok), _at(workspace),
                                 workspace.numel(), _stream_on(stream, dev))
    _check(st, "fdllm_tree_verify")
    return path, n_accept, next_tok


SPLIT_STREAM_K, SPLIT_WHOLE_ITEMS, SPLIT_CLUSTERS = 1, 2, 3


def fdllm_attention_split(B, N, H, dh, rows, S_max=0, verify=False):
    """(split, cluster_size): how the bf16 attention spreads these shapes over the
    current device (SPLIT_STREAM_K, SPLIT_WHOLE_ITEMS or SPLIT_CLUSTERS; -1 if
    it does not run them).  A diagnostic: launches nothing."""
    cs = ctypes.c_int(0)
    mode = lib().fdllm_attention_split(B, N, H, dh, rows, S_max, int(bool(verify)),
                                       ctypes.byref(cs))
    return int(mode), int(cs.value)


def fdllm_bounded_wait_selftest(limit_ns, workspace, stream=None):
    """Runs the kernels' bounded mbarrier wait against a barrier nothing completes
    (see include/fdllm.h).  Returns the four result words (first wait completed,
    its ns, second wait completed, its ns) after synchronising the stream; the
    status word is left for fdllm_get_status."""
    _need(workspace, "workspace", torch.uint8, None, None)
    st = lib().fdllm_bounded_wait_selftest(int(limit_ns), _p(workspace), workspace.numel(),
                                           _stream(stream, workspace.device))
    _check(st, "fdllm_bounded_wait_selftest")
    torch.cuda.current_stream(workspace.device).synchronize() if stream is None else \
        stream.synchronize()
    return [int(v) for v in workspace[256:288].view(torch.int64).cpu().tolist()]


def fdllm_get_status(workspace, stream=None) -> int:
    """Synchronises the stream and returns (and clears) the device status word."""
    return int(lib().fdllm_get_status(_p(workspace), _stream(stream, workspace.device)))
