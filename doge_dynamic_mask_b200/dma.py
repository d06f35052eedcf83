"""Thin Python binding of libdma (argument marshalling only).

Every function here forwards to the C entry point of the same name in
``libdma.so`` (declared in include/dma.h) with device pointers taken from torch
tensors and the current torch CUDA stream.  No step of the computation runs in
Python, and there is no fallback: importing this module fails loudly if the
library has not been built.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

import torch

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libdma.so")
if not os.path.exists(_LIB_PATH):
    raise ImportError(
        f"libdma.so is not built ({_LIB_PATH}); run `python -m doge_dynamic_mask_b200.build` (needs nvcc)")
_lib = ctypes.CDLL(_LIB_PATH)

DMA_OK = 0
STATUS = {0: "DMA_OK", 1: "DMA_ERR_INVALID_ARG", 2: "DMA_ERR_UNSUPPORTED", 3: "DMA_ERR_WORKSPACE",
          4: "DMA_ERR_CUDA", 5: "DMA_ERR_TIMEOUT", 6: "DMA_ERR_BAD_LENGTH", 7: "DMA_ERR_BAD_POSITION",
          8: "DMA_ERR_BAD_PAGE"}

_vp, _i, _f, _sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
_i64 = ctypes.c_int64
_lib.dma_workspace_size.restype = _sz
_lib.dma_workspace_size.argtypes = [_i] * 7
_lib.dma_dt_scores.restype = _i
_lib.dma_dt_scores.argtypes = [_vp, _vp, _vp, _i, _i, _i, _i, _vp, _vp]
_lib.dma_build_mask.restype = _i
_lib.dma_build_mask.argtypes = [_vp, _vp, _i, _i, _i, _i, _i, _vp, _vp, _vp, _sz, _vp]
_lib.dma_forward_prefill.restype = _i
_lib.dma_forward_prefill.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _f, _vp, _vp, _vp, _sz,
                                     _vp]
_lib.dma_forward_prefill_lse.restype = _i
_lib.dma_forward_prefill_lse.argtypes = [_vp] * 6 + [_i] * 6 + [_f] + [_vp] * 4 + [_sz, _vp]
_lib.dma_decode_step.restype = _i
_lib.dma_decode_step.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _f, _vp, _vp, _vp, _sz, _vp]
_lib.dma_decode_state_size.restype = _sz
_lib.dma_decode_state_size.argtypes = [_i] * 6
_lib.dma_decode_state_init.restype = _i
_lib.dma_decode_state_init.argtypes = [_vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _vp, _sz, _vp]
_lib.dma_decode_step_cached.restype = _i
_lib.dma_decode_step_cached.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _f, _vp, _vp, _sz, _vp]
_lib.dma_prologue.restype = _i
_lib.dma_prologue.argtypes = [_vp] * 5 + [_f, _f, _vp] + [_i] * 6 + [_vp] * 4 + [_sz, _vp]
_lib.dma_cdmoe_workspace_size.restype = _sz
_lib.dma_cdmoe_workspace_size.argtypes = [_i, _i]
_lib.dma_cdmoe_forward.restype = _i
_lib.dma_cdmoe_forward.argtypes = [_vp] * 4 + [_i] * 4 + [_vp] * 5 + [_sz, _vp]
_lib.dma_backward_workspace_size.restype = _sz
_lib.dma_backward_workspace_size.argtypes = [_i] * 6
_lib.dma_backward_prefill.restype = _i
_lib.dma_backward_prefill.argtypes = [_vp] * 6 + [_i] * 6 + [_f] + [_vp] * 11 + [_sz, _vp]
_lib.dma_append_paged.restype = _i
_lib.dma_append_paged.argtypes = [_vp] * 3 + [_i64] * 3 + [_vp] * 2 + [_f] * 2 + [_vp] * 5 + [_i] * 5 + [_i64] + [
    _i] * 3 + [_vp] * 6 + [_sz, _vp]
_lib.dma_decode_paged_workspace_size.restype = _sz
_lib.dma_decode_paged_workspace_size.argtypes = [_i] * 9
_lib.dma_decode_paged.restype = _i
_lib.dma_decode_paged.argtypes = [_vp] * 6 + [_i] * 4 + [_i64] + [_i] * 6 + [_f] + [_vp] * 2 + [_sz, _vp]
_lib.dma_prologue_backward_workspace_size.restype = _sz
_lib.dma_prologue_backward_workspace_size.argtypes = [_i] * 5
_lib.dma_prologue_backward.restype = _i
_lib.dma_prologue_backward.argtypes = [_vp] * 2 + [_i64] * 2 + [_vp] * 2 + [_f] * 2 + [_vp] * 3 + [_i] * 5 + [
    _vp] * 2 + [_i64] * 2 + [_vp] * 3 + [_sz, _vp]
_lib.dma_selftest_wait.restype = _i
_lib.dma_selftest_wait.argtypes = [_vp, _vp]
_lib.dma_check.restype = _i
_lib.dma_check.argtypes = [_vp, _i, _vp]
_lib.dma_status_string.restype = ctypes.c_char_p
_lib.dma_status_string.argtypes = [_i]
_lib.dma_last_cuda_error.restype = _i
_lib.dma_last_cuda_error.argtypes = []
_lib.dma_set_stage_events.restype = _i
_lib.dma_set_stage_events.argtypes = [_vp, _i]


class DMAError(RuntimeError):
    def __init__(self, status: int, where: str):
        name = _lib.dma_status_string(status).decode()
        extra = f" (cudaError {_lib.dma_last_cuda_error()})" if status == 4 else ""
        super().__init__(f"{where}: {name}{extra}")
        self.status = status


def _ok(status: int, where: str):
    if status != DMA_OK:
        raise DMAError(status, where)


def _ptr(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if not t.is_contiguous():
        raise ValueError("tensors passed to libdma must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def lib_path() -> str:
    return _LIB_PATH


def dma_workspace_size(B, Lq, Lk, Hq, Hkv, d, keep_window_size) -> int:
    return int(_lib.dma_workspace_size(B, Lq, Lk, Hq, Hkv, d, keep_window_size))


def new_workspace(nbytes: int, device=None) -> torch.Tensor:
    """A zeroed device workspace (the status word must start at zero)."""
    return torch.zeros(int(nbytes), dtype=torch.uint8, device=device or "cuda")


def _scratch(nbytes: int, device) -> torch.Tensor:
    """A workspace of which only the header is zeroed, for the calls that need no more."""
    ws = torch.empty(nbytes, dtype=torch.uint8, device=device)
    ws[:256].zero_()
    return ws


def dma_dt_scores(v, W_dt, A, dt_out=None, stream=None):
    B, L, Hkv, d = v.shape
    if dt_out is None:
        dt_out = torch.empty((B, Hkv, L), dtype=torch.float32, device=v.device)
    _ok(_lib.dma_dt_scores(_ptr(v), _ptr(W_dt), _ptr(A), B, L, Hkv, d, _ptr(dt_out), _stream(stream)),
        "dma_dt_scores")
    return dt_out


def dma_build_mask(dt, lengths, Lq, keep_window_size, workspace=None, tau_out=None, bitmask_out=None,
                   stream=None):
    B, Hkv, Lk = dt.shape
    if workspace is None:
        workspace = new_workspace(dma_workspace_size(B, Lq, Lk, Hkv, Hkv, 64, keep_window_size), dt.device)
    _ok(_lib.dma_build_mask(_ptr(dt), _ptr(lengths), B, Hkv, Lq, Lk, keep_window_size, _ptr(tau_out),
                            _ptr(bitmask_out), _ptr(workspace), workspace.numel(), _stream(stream)),
        "dma_build_mask")
    return workspace


def dma_forward_prefill(q, k, v, W_dt, A, lengths, keep_window_size, scale=None, dt_in=None, out=None,
                        workspace=None, stream=None, lse_out=None):
    """With lse_out ([B, Hq, L] float32) the rows' normalisers are written too
    (dma_forward_prefill_lse), for dma_backward_prefill(lse_in=...)."""
    B, L, Hq, d = q.shape
    Hkv = k.shape[2]
    if scale is None:
        scale = d ** -0.5
    if out is None:
        out = torch.empty_like(q)
    if workspace is None:
        workspace = new_workspace(dma_workspace_size(B, L, L, Hq, Hkv, d, keep_window_size), q.device)
    if lse_out is None:
        _ok(_lib.dma_forward_prefill(_ptr(q), _ptr(k), _ptr(v), _ptr(W_dt), _ptr(A), _ptr(lengths), B, L, Hq, Hkv,
                                     d, keep_window_size, float(scale), _ptr(dt_in), _ptr(out), _ptr(workspace),
                                     workspace.numel(), _stream(stream)),
            "dma_forward_prefill")
    else:
        _ok(_lib.dma_forward_prefill_lse(_ptr(q), _ptr(k), _ptr(v), _ptr(W_dt), _ptr(A), _ptr(lengths), B, L, Hq,
                                         Hkv, d, keep_window_size, float(scale), _ptr(dt_in), _ptr(out),
                                         _ptr(lse_out), _ptr(workspace), workspace.numel(), _stream(stream)),
            "dma_forward_prefill_lse")
    return out


def dma_decode_step(q, k_cache, v_cache, W_dt, A, lengths, keep_window_size, scale=None, dt_in=None, out=None,
                    workspace=None, stream=None):
    B, Hq, d = q.shape
    Lk, Hkv = k_cache.shape[1], k_cache.shape[2]
    if scale is None:
        scale = d ** -0.5
    if out is None:
        out = torch.empty_like(q)
    if workspace is None:
        workspace = new_workspace(dma_workspace_size(B, 1, Lk, Hq, Hkv, d, keep_window_size), q.device)
    _ok(_lib.dma_decode_step(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(W_dt), _ptr(A), _ptr(lengths), B, Lk, Hq,
                             Hkv, d, keep_window_size, float(scale), _ptr(dt_in), _ptr(out), _ptr(workspace),
                             workspace.numel(), _stream(stream)),
        "dma_decode_step")
    return out


def dma_prologue(q, k, v, q_norm_w, k_norm_w, positions, k_cache, v_cache, eps=1e-6, rope_theta=10000.0,
                 q_out=None, workspace=None, stream=None):
    """q/k RMSNorm over head_dim, rotary embedding, and the KV-cache append of
    L new tokens per sequence (token t of sequence b at cache row positions[b] + t).
    Returns q_out; k_cache and v_cache are written in place."""
    B, L, Hq, d = q.shape
    Hkv = k.shape[2]
    Lmax = k_cache.shape[1]
    if q_out is None:
        q_out = torch.empty_like(q)
    if workspace is None:
        workspace = new_workspace(256, q.device)
    _ok(_lib.dma_prologue(_ptr(q), _ptr(k), _ptr(v), _ptr(q_norm_w), _ptr(k_norm_w), float(eps), float(rope_theta),
                          _ptr(positions), B, L, Lmax, Hq, Hkv, d, _ptr(q_out), _ptr(k_cache), _ptr(v_cache),
                          _ptr(workspace), workspace.numel(), _stream(stream)),
        "dma_prologue")
    return q_out


def dma_backward_workspace_size(B, L, Hq, Hkv, d, keep_window_size) -> int:
    return int(_lib.dma_backward_workspace_size(B, L, Hq, Hkv, d, keep_window_size))


def dma_backward_prefill(q, k, v, W_dt, A, lengths, keep_window_size, out, dout, scale=None, dt_in=None,
                         workspace=None, want_d_dt=False, stream=None, lse_in=None):
    """Gradients of sum(out * dout) with the selection held fixed: returns
    (dq, dk, dv) bf16, dW_dt and dA float32, and d_dt [B, Hkv, L] float32 when
    want_d_dt.  lse_in: the forward's row normalisers (dma_forward_prefill with
    lse_out), else they are recomputed."""
    B, L, Hq, d = q.shape
    Hkv = k.shape[2]
    if scale is None:
        scale = d ** -0.5
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    dW = torch.empty_like(W_dt)
    dA = torch.empty_like(A)
    d_dt = torch.empty((B, Hkv, L), dtype=torch.float32, device=q.device) if want_d_dt else None
    if workspace is None:
        workspace = new_workspace(dma_backward_workspace_size(B, L, Hq, Hkv, d, keep_window_size), q.device)
    _ok(_lib.dma_backward_prefill(_ptr(q), _ptr(k), _ptr(v), _ptr(W_dt), _ptr(A), _ptr(lengths), B, L, Hq, Hkv, d,
                                  keep_window_size, float(scale), _ptr(dt_in), _ptr(out), _ptr(dout),
                                  _ptr(lse_in), _ptr(dq),
                                  _ptr(dk), _ptr(dv), _ptr(d_dt), _ptr(dW), _ptr(dA), _ptr(workspace),
                                  workspace.numel(), _stream(stream)),
        "dma_backward_prefill")
    return (dq, dk, dv, dW, dA, d_dt) if want_d_dt else (dq, dk, dv, dW, dA)


def dma_cdmoe_workspace_size(T, num_experts) -> int:
    return int(_lib.dma_cdmoe_workspace_size(T, num_experts))


def dma_cdmoe_forward(h, W_router, down_embed, up_embed, top_k, logits_in=None, out=None, experts_out=None,
                      scores_out=None, workspace=None, stream=None):
    """Routed CDMoE output [T, hidden] (bf16).  With experts_out / scores_out
    ([T, top_k] int32 / float32) the kept experts are written too, best first."""
    T, hidden = h.shape
    num_experts = down_embed.shape[0]
    if out is None:
        out = torch.empty_like(h)
    if workspace is None:
        size = dma_cdmoe_workspace_size(T, num_experts)
        if size == 0:
            raise ValueError("unsupported CDMoE geometry")
        workspace = new_workspace(size, h.device)
    _ok(_lib.dma_cdmoe_forward(_ptr(h), _ptr(W_router), _ptr(down_embed), _ptr(up_embed), T, hidden, num_experts,
                               top_k, _ptr(logits_in), _ptr(out), _ptr(experts_out), _ptr(scores_out),
                               _ptr(workspace), workspace.numel(), _stream(stream)),
        "dma_cdmoe_forward")
    return out


def dma_decode_state_size(B, Lk, Hq, Hkv, d, keep_window_size) -> int:
    return int(_lib.dma_decode_state_size(B, Lk, Hq, Hkv, d, keep_window_size))


def dma_decode_state_init(v_cache, W_dt, A, lengths, keep_window_size, Hq, state=None, stream=None):
    """Decode state for incremental steps: dt of every cached token and each
    (batch, kv head)'s kept set.  Returns the state (a uint8 device tensor)."""
    B, Lk, Hkv, d = v_cache.shape
    size = dma_decode_state_size(B, Lk, Hq, Hkv, d, keep_window_size)
    if size == 0:
        raise ValueError("unsupported decode geometry")
    if state is None:
        state = torch.empty(size, dtype=torch.uint8, device=v_cache.device)
    _ok(_lib.dma_decode_state_init(_ptr(v_cache), _ptr(W_dt), _ptr(A), _ptr(lengths), B, Lk, Hq, Hkv, d,
                                   keep_window_size, _ptr(state), state.numel(), _stream(stream)),
        "dma_decode_state_init")
    return state


def dma_decode_step_cached(q, k_cache, v_cache, W_dt, A, lengths, keep_window_size, state, scale=None, out=None,
                           stream=None):
    """One decode step that takes in only the tokens cached since the previous step."""
    B, Hq, d = q.shape
    Lk, Hkv = k_cache.shape[1], k_cache.shape[2]
    if scale is None:
        scale = d ** -0.5
    if out is None:
        out = torch.empty_like(q)
    _ok(_lib.dma_decode_step_cached(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(W_dt), _ptr(A), _ptr(lengths), B,
                                    Lk, Hq, Hkv, d, keep_window_size, float(scale), _ptr(out), _ptr(state),
                                    state.numel(), _stream(stream)),
        "dma_decode_step_cached")
    return out


# the current device and its current stream's handle, without building torch objects for them
_current_device = torch._C._cuda_getDevice
_current_stream = torch._C._cuda_getCurrentRawStream


def _elsewhere(call, device, stream, *args, **kw):
    """The call with the stream it names, or its tensors' device, made current: what the binding allocates then
    belongs to the stream that uses it."""
    if device.type != "cuda":
        raise ValueError("tensors passed to libdma must be CUDA tensors")
    with torch.cuda.device(device) if stream is None else torch.cuda.stream(stream):
        if _current_device() != device.index:
            raise ValueError("the stream belongs to another device than the tensors")
        return call(*args, **kw)


def _refuse(device, *wanted):
    """Names the argument that keeps a call from being made: (name, tensor, dtype, shape, may be strided)."""
    for name, t, dtype, shape, strided in wanted:
        if t is None:
            continue
        if t.dtype is not dtype or t.get_device() != device or tuple(t.shape) != tuple(shape):
            raise ValueError(f"{name}: {dtype} {tuple(shape)} on cuda:{device} is wanted, "
                             f"got {t.dtype} {tuple(t.shape)} on {t.device}")
        if not strided and not t.is_contiguous():
            raise ValueError(f"{name}: must be contiguous")
    raise ValueError("unsupported arguments")


def _token_stride(name, t):
    """Elements between tokens of [.., H, d] whose head rows are dense (a slice of a wider projection's output)."""
    shape = t.shape
    d = shape[-1]
    if t.is_contiguous():
        return shape[-2] * d
    st = t.stride()
    if st[-1] != 1 or (shape[-2] > 1 and st[-2] != d):
        raise ValueError(f"{name}: its heads must be dense")
    if len(st) == 3:
        return st[0] if shape[0] > 1 else shape[1] * d
    if shape[0] > 1 and shape[1] > 1 and st[0] != st[1] * shape[1]:
        raise ValueError(f"{name}: its tokens must be evenly spaced")
    return st[1] if shape[1] > 1 else st[0] if shape[0] > 1 else shape[2] * d


def _page_stride(k_pages, v_pages):
    """Elements between the pages of both pools (the rest of a page is dense)."""
    _, page_size, Hkv, d = shape = k_pages.shape
    if k_pages.is_contiguous() and v_pages.is_contiguous() and v_pages.shape == shape:
        return page_size * Hkv * d
    st = k_pages.stride()
    if (v_pages.shape != shape or v_pages.stride() != st or st[3] != 1 or (Hkv > 1 and st[2] != d)
            or (page_size > 1 and st[1] != Hkv * d)):
        raise ValueError("k_pages and v_pages must have one shape and stride, with dense pages")
    return st[0] if shape[0] > 1 else page_size * Hkv * d


def dma_append_paged(q, k, v, q_norm_w, k_norm_w, W_dt, A, cu_tokens, positions, page_table, k_pages, v_pages,
                     dt_pages, eps=1e-6, rope_theta=10000.0, q_out=None, k_out=None, workspace=None, stream=None):
    """q/k RMSNorm and rotary embedding of a ragged batch's new tokens (packed [T, H, d]; sequence b owns tokens
    cu_tokens[b] .. cu_tokens[b + 1] - 1, at positions from positions[b] on), K and V to their pages, dt to
    dt_pages.  q, k and v may be slices of one projection's output.  Returns q_out; with k_out ([T, Hkv, d]) the
    rotated K rows are written there too."""
    dev = q.get_device()
    if dev < 0 or stream is not None or dev != _current_device():
        return _elsewhere(dma_append_paged, q.device, stream, q, k, v, q_norm_w, k_norm_w, W_dt, A, cu_tokens,
                          positions, page_table, k_pages, v_pages, dt_pages, eps, rope_theta, q_out, k_out, workspace)
    T, Hq, d = q.shape
    N, page_size, Hkv, _ = k_pages.shape
    B, max_pages = page_table.shape
    bf, f32, i32 = torch.bfloat16, torch.float32, torch.int32
    if q_out is None:
        q_out = torch.empty(T, Hq, d, dtype=bf, device=q.device)
    if workspace is None:
        workspace = new_workspace(256, q.device)
    kv = (T, Hkv, d)
    if not (q.dtype is bf and k.dtype is bf and v.dtype is bf and k_pages.dtype is bf and v_pages.dtype is bf
            and q_out.dtype is bf and q_norm_w.dtype is f32 and k_norm_w.dtype is f32 and W_dt.dtype is f32
            and A.dtype is f32 and dt_pages.dtype is f32 and cu_tokens.dtype is i32 and positions.dtype is i32
            and page_table.dtype is i32 and k.shape == kv and v.shape == kv and q_out.shape == (T, Hq, d)
            and k_pages.shape[3] == d and dt_pages.shape == (N, Hkv, page_size) and W_dt.shape == (Hkv * d, Hkv)
            and q_norm_w.shape == k_norm_w.shape == (d,) and A.shape == (Hkv,) and cu_tokens.shape == (B + 1,)
            and positions.shape == (B,)
            and k.get_device() == v.get_device() == q_norm_w.get_device() == k_norm_w.get_device()
            == W_dt.get_device() == A.get_device() == cu_tokens.get_device() == positions.get_device()
            == page_table.get_device() == k_pages.get_device() == v_pages.get_device() == dt_pages.get_device()
            == q_out.get_device() == workspace.get_device() == dev
            and q_norm_w.is_contiguous() and k_norm_w.is_contiguous() and W_dt.is_contiguous() and A.is_contiguous()
            and cu_tokens.is_contiguous() and positions.is_contiguous() and page_table.is_contiguous()
            and dt_pages.is_contiguous() and q_out.is_contiguous() and workspace.is_contiguous()
            and (k_out is None or (k_out.dtype is bf and k_out.shape == kv and k_out.get_device() == dev
                                   and k_out.is_contiguous()))):
        _refuse(dev, ("q", q, bf, (T, Hq, d), True), ("k", k, bf, kv, True), ("v", v, bf, kv, True),
                ("q_norm_w", q_norm_w, f32, (d,), False), ("k_norm_w", k_norm_w, f32, (d,), False),
                ("W_dt", W_dt, f32, (Hkv * d, Hkv), False), ("A", A, f32, (Hkv,), False),
                ("cu_tokens", cu_tokens, i32, (B + 1,), False), ("positions", positions, i32, (B,), False),
                ("page_table", page_table, i32, (B, max_pages), False),
                ("k_pages", k_pages, bf, (N, page_size, Hkv, d), True),
                ("v_pages", v_pages, bf, (N, page_size, Hkv, d), True),
                ("dt_pages", dt_pages, f32, (N, Hkv, page_size), False), ("q_out", q_out, bf, (T, Hq, d), False),
                ("k_out", k_out, bf, kv, False),
                ("workspace", workspace, workspace.dtype, workspace.shape, False))
    _ok(_lib.dma_append_paged(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), _token_stride("q", q), _token_stride("k", k),
        _token_stride("v", v), q_norm_w.data_ptr(), k_norm_w.data_ptr(), eps, rope_theta, W_dt.data_ptr(),
        A.data_ptr(), cu_tokens.data_ptr(), positions.data_ptr(), page_table.data_ptr(), T, B, max_pages, N,
        page_size, _page_stride(k_pages, v_pages), Hq, Hkv, d, q_out.data_ptr(),
        None if k_out is None else k_out.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(), dt_pages.data_ptr(),
        workspace.data_ptr(), workspace.nbytes, _current_stream(dev)), "dma_append_paged")
    return q_out


def dma_decode_paged_workspace_size(B, max_pages, page_size, Hq, Hkv, d, keep_window_size, window=0, sinks=0) -> int:
    if (B | max_pages | page_size | Hq | Hkv | d | keep_window_size | window | sinks) >> 31:
        return 0   # ctypes would take them modulo 2^32
    return int(_lib.dma_decode_paged_workspace_size(B, max_pages, page_size, Hq, Hkv, d, keep_window_size, window,
                                                    sinks))


def dma_decode_paged(q, k_pages, v_pages, dt_pages, page_table, lengths, keep_window_size, window=0, sinks=0,
                     scale=None, out=None, workspace=None, stream=None):
    """One new query per sequence ([B, Hq, d]) over a paged cache: of the keys a sequence of lengths[b] tokens
    sees (all, or the last `window` and the first `sinks`) the keep_window_size best by dt_pages, with dt as an
    additive bias.  A length of 0 gives a zero row."""
    if (keep_window_size | window | sinks) >> 31:
        raise ValueError("keep_window_size, window and sinks must lie in [0, 2^31)")
    dev = q.get_device()
    if dev < 0 or stream is not None or dev != _current_device():
        return _elsewhere(dma_decode_paged, q.device, stream, q, k_pages, v_pages, dt_pages, page_table, lengths,
                          keep_window_size, window, sinks, scale, out, workspace)
    B, Hq, d = q.shape
    N, page_size, Hkv, _ = k_pages.shape
    max_pages = page_table.shape[1]
    bf, i32 = torch.bfloat16, torch.int32
    if out is None:
        out = torch.empty(B, Hq, d, dtype=bf, device=q.device)
    if workspace is None:
        size = dma_decode_paged_workspace_size(B, max_pages, page_size, Hq, Hkv, d, keep_window_size, window, sinks)
        if size == 0:
            raise ValueError("unsupported paged decode geometry")
        workspace = _scratch(size, q.device)
    if not (q.dtype is bf and k_pages.dtype is bf and v_pages.dtype is bf and out.dtype is bf
            and dt_pages.dtype is torch.float32 and page_table.dtype is i32 and lengths.dtype is i32
            and out.shape == (B, Hq, d) and k_pages.shape[3] == d and dt_pages.shape == (N, Hkv, page_size)
            and page_table.shape == (B, max_pages) and lengths.shape == (B,)
            and k_pages.get_device() == v_pages.get_device() == dt_pages.get_device() == page_table.get_device()
            == lengths.get_device() == out.get_device() == workspace.get_device() == dev
            and q.is_contiguous() and dt_pages.is_contiguous() and page_table.is_contiguous()
            and lengths.is_contiguous() and out.is_contiguous() and workspace.is_contiguous()):
        _refuse(dev, ("q", q, bf, (B, Hq, d), False), ("k_pages", k_pages, bf, (N, page_size, Hkv, d), True),
                ("v_pages", v_pages, bf, (N, page_size, Hkv, d), True),
                ("dt_pages", dt_pages, torch.float32, (N, Hkv, page_size), False),
                ("page_table", page_table, i32, (B, max_pages), False), ("lengths", lengths, i32, (B,), False),
                ("out", out, bf, (B, Hq, d), False),
                ("workspace", workspace, workspace.dtype, workspace.shape, False))
    if out.data_ptr() == q.data_ptr():
        raise ValueError("out must not be q: blocks that share a row read q until the last one has joined it")
    _ok(_lib.dma_decode_paged(
        q.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(), dt_pages.data_ptr(), page_table.data_ptr(),
        lengths.data_ptr(), B, max_pages, N, page_size, _page_stride(k_pages, v_pages), Hq, Hkv, d,
        keep_window_size, window, sinks, d ** -0.5 if scale is None else scale, out.data_ptr(),
        workspace.data_ptr(), workspace.nbytes, _current_stream(dev)), "dma_decode_paged")
    return out


def dma_prologue_backward_workspace_size(B, L, Hq, Hkv, d) -> int:
    if (B | L | Hq | Hkv | d) >> 31:
        return 0   # ctypes would take them modulo 2^32
    return int(_lib.dma_prologue_backward_workspace_size(B, L, Hq, Hkv, d))


def dma_prologue_backward(q, k, q_norm_w, k_norm_w, positions, dq_out, dk_out, eps=1e-6, rope_theta=10000.0, dq=None,
                          dk=None, dq_norm_w=None, dk_norm_w=None, workspace=None, stream=None):
    """Gradients of dma_prologue's norms and rotation from those of its rotated q and k ([B, L, H, d]): returns
    (dq, dk) bf16 and (dq_norm_w, dk_norm_w) float32.  q, k, dq and dk may be slices of a projection's buffers."""
    dev = q.get_device()
    if dev < 0 or stream is not None or dev != _current_device():
        return _elsewhere(dma_prologue_backward, q.device, stream, q, k, q_norm_w, k_norm_w, positions, dq_out,
                          dk_out, eps, rope_theta, dq, dk, dq_norm_w, dk_norm_w, workspace)
    B, L, Hq, d = qs = q.shape
    Hkv = k.shape[2]
    ks = (B, L, Hkv, d)
    bf, f32 = torch.bfloat16, torch.float32
    if dq is None:
        dq = torch.empty(B, L, Hq, d, dtype=bf, device=q.device)
    if dk is None:
        dk = torch.empty(B, L, Hkv, d, dtype=bf, device=q.device)
    if dq_norm_w is None and dk_norm_w is None:
        dq_norm_w, dk_norm_w = torch.empty_like(q_norm_w), torch.empty_like(k_norm_w)
    elif dq_norm_w is None or dk_norm_w is None:
        raise ValueError("dq_norm_w and dk_norm_w: give both or neither")
    if workspace is None:
        size = dma_prologue_backward_workspace_size(B, L, Hq, Hkv, d)
        if size == 0:
            raise ValueError("unsupported prologue geometry")
        workspace = _scratch(size, q.device)
    if not (q.dtype is bf and k.dtype is bf and dq_out.dtype is bf and dk_out.dtype is bf and dq.dtype is bf
            and dk.dtype is bf and q_norm_w.dtype is f32 and k_norm_w.dtype is f32 and dq_norm_w.dtype is f32
            and dk_norm_w.dtype is f32 and positions.dtype is torch.int32
            and k.shape == dk_out.shape == dk.shape == ks and dq_out.shape == dq.shape == qs
            and q_norm_w.shape == k_norm_w.shape == dq_norm_w.shape == dk_norm_w.shape == (d,)
            and positions.shape == (B,)
            and k.get_device() == dq_out.get_device() == dk_out.get_device() == dq.get_device() == dk.get_device()
            == q_norm_w.get_device() == k_norm_w.get_device() == dq_norm_w.get_device() == dk_norm_w.get_device()
            == positions.get_device() == workspace.get_device() == dev
            and dq_out.is_contiguous() and dk_out.is_contiguous() and q_norm_w.is_contiguous()
            and k_norm_w.is_contiguous() and dq_norm_w.is_contiguous() and dk_norm_w.is_contiguous()
            and positions.is_contiguous() and workspace.is_contiguous()):
        _refuse(dev, ("q", q, bf, qs, True), ("k", k, bf, ks, True), ("dq_out", dq_out, bf, qs, False),
                ("dk_out", dk_out, bf, ks, False), ("dq", dq, bf, qs, True), ("dk", dk, bf, ks, True),
                ("q_norm_w", q_norm_w, f32, (d,), False), ("k_norm_w", k_norm_w, f32, (d,), False),
                ("dq_norm_w", dq_norm_w, f32, (d,), False), ("dk_norm_w", dk_norm_w, f32, (d,), False),
                ("positions", positions, torch.int32, (B,), False),
                ("workspace", workspace, workspace.dtype, workspace.shape, False))
    _ok(_lib.dma_prologue_backward(
        q.data_ptr(), k.data_ptr(), _token_stride("q", q), _token_stride("k", k), q_norm_w.data_ptr(),
        k_norm_w.data_ptr(), eps, rope_theta, positions.data_ptr(), dq_out.data_ptr(), dk_out.data_ptr(), B, L, Hq,
        Hkv, d, dq.data_ptr(), dk.data_ptr(), _token_stride("dq", dq), _token_stride("dk", dk),
        dq_norm_w.data_ptr(), dk_norm_w.data_ptr(), workspace.data_ptr(), workspace.nbytes,
        _current_stream(dev)), "dma_prologue_backward")
    return dq, dk, dq_norm_w, dk_norm_w


# keys per split of the decode attention: the kept lists are padded to a
# multiple of it (the library's layout of a decode workspace)
DECODE_CHUNK = 128


def decode_state_views(state, B, Lk, Hq, Hkv, d, keep_window_size):
    """(dt [B, Hkv, Lk] float32, kept count [B, Hkv] int32, kept key lists [B, Hkv, cap] int32) views of a
    decode state, for tests: the layout is that of a decode workspace."""
    bg = B * Hkv
    cap = -(-min(Lk, keep_window_size) // DECODE_CHUNK) * DECODE_CHUNK
    def up(x):
        return -(-x // 256) * 256
    off = 256
    dt = state[off:off + bg * Lk * 4].view(torch.float32).view(B, Hkv, Lk)
    off = up(off + bg * Lk * 4)
    off = up(off + bg * 8)                   # tau
    idx = state[off:off + bg * cap * 4].view(torch.int32).view(B, Hkv, cap)
    off = up(off + bg * cap * 4)
    off = up(off + bg * cap * 4)             # bias
    count = state[off:off + bg * 4].view(torch.int32).view(B, Hkv)
    return dt, count, idx


def paged_list_views(workspace, B, Hq, Hkv, d, keep_window_size):
    """(positions [B, Hkv, w] int32, bias [B, Hkv, w] float32) of a paged decode workspace with kept lists, for tests:
    a kept key's position in its sequence (-1: no key), and its dt.  Written for the rows that see more than w keys.
    They are the workspace's last two parts, each rounded up to 256 bytes; what lies before them depends on the head
    shapes alone, so the size for the shortest table with lists tells where they begin."""
    n = B * Hkv * keep_window_size * 4
    part = -(-n // 256) * 256
    bias = dma_decode_paged_workspace_size(B, keep_window_size + 1, 1, Hq, Hkv, d, keep_window_size) - part
    shape = (B, Hkv, keep_window_size)
    return (workspace[bias - part:bias - part + n].view(torch.int32).view(shape),
            workspace[bias:bias + n].view(torch.float32).view(shape))


def dma_selftest_wait(workspace, stream=None):
    """Launch the bounded-wait diagnostic: its wait runs out (about one second)
    and records a timeout that dma_check then reports."""
    _ok(_lib.dma_selftest_wait(_ptr(workspace), _stream(stream)), "dma_selftest_wait")


def dma_check(workspace, clear=True, stream=None) -> int:
    """Synchronises the stream and returns the device-recorded status (0 = DMA_OK)."""
    return int(_lib.dma_check(_ptr(workspace), 1 if clear else 0, _stream(stream)))


class StageEvents:
    """Context manager: while active, prefill/decode calls on this thread record
    4 torch CUDA events (before S1, after S1, after S2, after the attention)."""

    def __init__(self):
        self.events = [torch.cuda.Event(enable_timing=True) for _ in range(4)]
        for e in self.events:          # materialise the underlying cudaEvent_t
            e.record()
        self._arr = (ctypes.c_void_p * 4)(*[ctypes.c_void_p(e.cuda_event) for e in self.events])

    def __enter__(self):
        _ok(_lib.dma_set_stage_events(self._arr, 4), "dma_set_stage_events")
        return self

    def __exit__(self, *exc):
        _lib.dma_set_stage_events(None, 0)

    def stage_ms(self):
        """(S1, S2, attention) milliseconds of the last recorded call."""
        e = self.events
        return (e[0].elapsed_time(e[1]), e[1].elapsed_time(e[2]), e[2].elapsed_time(e[3]))


def dma_status_string(status: int) -> str:
    return _lib.dma_status_string(status).decode()


def raw():
    """The ctypes handle (for tests that call the C ABI with raw pointers)."""
    return _lib
