"""Python binding of libgdr (the C ABI in include/gdr.h): argument marshalling only.

The attention-layer operators go through a compiled binding (_gdr_bind, csrc/gdr_bind.cpp), the other
calls through ctypes.

Each function checks tensor devices, dtypes, shapes and contiguity, allocates outputs the
caller did not pass (memory of the launch stream: plumbing, no arithmetic), hands raw device pointers
and the current CUDA stream, or the one given, to the library and raises ``GdrError`` on a non-OK status. Every
step of the computation runs in the library's kernels; there is no CPU fallback: if
``libgdr.so`` is missing this module raises instead of computing anything. No call is recorded by
autograd: gradients are calls of their own.
"""
from __future__ import annotations

import ctypes
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libgdr.so")

GDR_OK, GDR_ERR_INVALID_ARG, GDR_ERR_UNSUPPORTED, GDR_ERR_CUDA, GDR_ERR_DEVICE_INDEX, GDR_ERR_TIMEOUT, \
    GDR_ERR_NO_PAGES = range(7)
GDR_F32, GDR_BF16 = 0, 1
D = 128

EXPORTS = ["gdr_chunk_workspace_bytes", "gdr_chunk_fwd", "gdr_chunk_fwd_varlen", "gdr_chunk_fwd_gated",
           "gdr_chunk_fwd_noalloc", "gdr_chunk_fwd_prologue_workspace_bytes", "gdr_chunk_fwd_prologue",
           "gdr_fork_workspace_bytes",
           "gdr_fork_fwd", "gdr_decode_step", "gdr_prologue", "gdr_gated_rmsnorm",
           "gdr_backward_workspace_bytes", "gdr_backward",
           "gdr_backward_chunked_workspace_bytes", "gdr_backward_chunked",
           "gdr_chunk_fwd_save", "gdr_backward_chunked_saved",
           "gdr_qk_norm_rope", "gdr_qk_norm_rope_append", "gdr_qk_norm_rope_backward_workspace_bytes",
           "gdr_qk_norm_rope_backward", "gdr_tree_attn_workspace_bytes", "gdr_tree_attn", "gdr_verify_draft",
           "gdr_cache_workspace_bytes", "gdr_cache_reserve", "gdr_cache_fork", "gdr_cache_free", "gdr_cache_compact",
           "gdr_sync_status", "gdr_status_string", "gdr_last_error_message",
           "gdr_stage_timer_enable", "gdr_stage_timer_collect", "gdr_kernel_name", "gdr_debug_set_wait_budget"]


class GdrError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(message)
        self.status = status


_lib = None


def lib() -> ctypes.CDLL:
    """Load libgdr.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is missing: build it with __graft_entry__.build() "
                           "or python -m gated_deltanet_rule_gb300.build")
    L = ctypes.CDLL(LIB_PATH)
    vp, fp, i, sz = ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
    L.gdr_chunk_workspace_bytes.argtypes = [i, i, i, i, i, i]
    L.gdr_chunk_workspace_bytes.restype = sz
    L.gdr_chunk_fwd.argtypes = [vp, vp, vp, fp, fp, fp, vp, fp, i, i, i, i, i, i, vp, sz, vp]
    L.gdr_chunk_fwd.restype = i
    L.gdr_chunk_fwd_varlen.argtypes = [vp, vp, vp, fp, fp, fp, vp, vp, fp, i, i, i, i, i, i, vp, sz, vp]
    L.gdr_chunk_fwd_varlen.restype = i
    L.gdr_chunk_fwd_gated.argtypes = [vp, vp, vp, fp, fp, fp, vp, fp, ctypes.c_float, vp, fp, i, i, i, i, i, i, vp, sz, vp]
    L.gdr_chunk_fwd_gated.restype = i
    L.gdr_chunk_fwd_noalloc.argtypes = [vp, vp, vp, fp, fp, fp, vp, fp, i, i, i, i, i, i, vp]
    L.gdr_chunk_fwd_noalloc.restype = i
    L.gdr_fork_workspace_bytes.argtypes = [i, i, i, i, i, i]
    L.gdr_fork_workspace_bytes.restype = sz
    L.gdr_fork_fwd.argtypes = [vp, vp, vp, fp, fp, fp, vp, i, vp, fp, i, i, i, i, i, i, vp, sz, vp]
    L.gdr_fork_fwd.restype = i
    L.gdr_decode_step.argtypes = [vp, vp, vp, fp, fp, fp, vp, i, i, i, i, i, vp]
    L.gdr_decode_step.restype = i
    L.gdr_prologue.argtypes = [vp, vp, fp, fp, fp, fp, fp, vp, vp, vp, vp, fp, fp, vp, i, i, i, i, i, i, vp]
    L.gdr_prologue.restype = i
    L.gdr_chunk_fwd_prologue_workspace_bytes.argtypes = [i, i, i, i, i, i]
    L.gdr_chunk_fwd_prologue_workspace_bytes.restype = sz
    L.gdr_chunk_fwd_prologue.argtypes = [vp, vp, fp, fp, fp, fp, fp, fp, vp, fp, vp, i, i, i, i, i, i, vp, sz, vp]
    L.gdr_chunk_fwd_prologue.restype = i
    L.gdr_gated_rmsnorm.argtypes = [vp, vp, fp, ctypes.c_float, vp, ctypes.c_longlong, i, vp]
    L.gdr_gated_rmsnorm.restype = i
    L.gdr_backward_workspace_bytes.argtypes = [i, i, i, i, i]
    L.gdr_backward_workspace_bytes.restype = sz
    L.gdr_backward.argtypes = [vp, vp, vp, fp, fp, fp, vp, fp, fp, fp, fp, fp, fp, fp, i, i, i, i, i, i, vp, sz, vp]
    L.gdr_backward.restype = i
    L.gdr_backward_chunked_workspace_bytes.argtypes = [i, i, i, i, i]
    L.gdr_backward_chunked_workspace_bytes.restype = sz
    L.gdr_backward_chunked.argtypes = [vp, vp, vp, fp, fp, fp, vp, fp, fp, fp, fp, fp, fp, fp, i, i, i, i, i, i, vp, sz,
                                       vp]
    L.gdr_backward_chunked.restype = i
    L.gdr_backward_chunked_saved.argtypes = L.gdr_backward_chunked.argtypes
    L.gdr_backward_chunked_saved.restype = i
    L.gdr_chunk_fwd_save.argtypes = [vp, vp, vp, fp, fp, fp, vp, fp, i, i, i, i, i, i, vp, sz, vp]
    L.gdr_chunk_fwd_save.restype = i
    ll, f32 = ctypes.c_longlong, ctypes.c_float
    L.gdr_qk_norm_rope.argtypes = [vp, vp, fp, fp, vp, vp, f32, i, vp, vp, i, i, i, i, i, i, ll, ll, ll, ll, i, vp]
    L.gdr_qk_norm_rope.restype = i
    L.gdr_qk_norm_rope_append.argtypes = [vp, vp, vp, fp, fp, vp, vp, f32, i, vp, vp, vp, vp, vp, vp, i, i, i, i, i, i,
                                          i, i, i, ll, ll, ll, ll, ll, ll, i, vp]
    L.gdr_qk_norm_rope_append.restype = i
    L.gdr_qk_norm_rope_backward_workspace_bytes.argtypes = [i]
    L.gdr_qk_norm_rope_backward_workspace_bytes.restype = sz
    L.gdr_qk_norm_rope_backward.argtypes = [vp, vp, fp, fp, vp, vp, vp, vp, f32, i, fp, fp, fp, fp, i, i, i, i, i, i, ll,
                                            ll, ll, ll, i, vp, sz, vp]
    L.gdr_qk_norm_rope_backward.restype = i
    L.gdr_tree_attn_workspace_bytes.argtypes = [i]
    L.gdr_tree_attn_workspace_bytes.restype = sz
    L.gdr_tree_attn.argtypes = [vp, vp, vp, vp, vp, vp, vp, f32, vp, fp, i, i, i, i, i, i, i, i, i, vp, sz, vp]
    L.gdr_tree_attn.restype = i
    L.gdr_verify_draft.argtypes = [vp, vp, vp, vp, vp, fp, fp, vp, vp, vp, i, i, i, i, vp]
    L.gdr_verify_draft.restype = i
    L.gdr_cache_workspace_bytes.argtypes = [i, i]
    L.gdr_cache_workspace_bytes.restype = sz
    L.gdr_cache_reserve.argtypes = [vp, vp, vp, vp, i, i, i, i, i, i, vp, sz, vp]
    L.gdr_cache_reserve.restype = i
    L.gdr_cache_fork.argtypes = [vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, ll, vp, sz, vp]
    L.gdr_cache_fork.restype = i
    L.gdr_cache_free.argtypes = [vp, vp, vp, vp, i, i, i, i, vp]
    L.gdr_cache_free.restype = i
    L.gdr_cache_compact.argtypes = [vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, ll, vp]
    L.gdr_cache_compact.restype = i
    L.gdr_sync_status.argtypes = [vp]
    L.gdr_sync_status.restype = i
    L.gdr_status_string.argtypes = [i]
    L.gdr_status_string.restype = ctypes.c_char_p
    L.gdr_last_error_message.argtypes = []
    L.gdr_last_error_message.restype = ctypes.c_char_p
    L.gdr_stage_timer_enable.argtypes = [i, i]
    L.gdr_stage_timer_enable.restype = i
    L.gdr_stage_timer_collect.argtypes = [ctypes.POINTER(ctypes.c_double), ctypes.POINTER(ctypes.c_int), i]
    L.gdr_stage_timer_collect.restype = i
    L.gdr_debug_set_wait_budget.argtypes = [ctypes.c_longlong]
    L.gdr_debug_set_wait_budget.restype = i
    L.gdr_kernel_name.argtypes = [i]
    L.gdr_kernel_name.restype = ctypes.c_char_p
    _lib = L
    return L


def _check(status: int) -> None:
    if status != GDR_OK:
        L = lib()
        name = L.gdr_status_string(status).decode()
        msg = L.gdr_last_error_message().decode()
        raise GdrError(status, f"{name}: {msg}")


def _p(t):
    return None if t is None else t.data_ptr()


def _stream(stream) -> int:
    if stream is None:   # the raw handle: building a Stream object costs more than a small kernel
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
    return stream.cuda_stream


def _empty(shape, dtype, device, stream) -> torch.Tensor:
    """A new output or workspace, of the launch stream's memory: the allocator hands memory out again in
    the order of the stream it was taken for, so what is dropped while the kernels run goes to nobody
    whose work does not come after them. The current stream may read it too."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if not isinstance(stream, torch.cuda.Stream):   # any object with the raw handle
        raw = stream.cuda_stream
        stream = torch.cuda.ExternalStream(raw, device) if raw else torch.cuda.default_stream(device)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=device)
    t.record_stream(torch.cuda.current_stream())
    return t


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return GDR_F32
    if t.dtype == torch.bfloat16:
        return GDR_BF16
    raise TypeError(f"q/k/v must be float32 or bfloat16, got {t.dtype}")


def _need(cond: bool, msg: str) -> None:
    if not cond:
        raise ValueError(msg)


def _check_inputs(q, k, v, g, beta, device_check=True):
    for name, t in (("q", q), ("k", k), ("v", v), ("g", g), ("beta", beta)):
        _need(isinstance(t, torch.Tensor), f"{name} must be a tensor")
        if device_check:
            _need(t.is_cuda, f"{name} must be a CUDA tensor")
        _need(t.is_contiguous(), f"{name} must be contiguous")
    _need(q.dtype == k.dtype == v.dtype, "q, k, v must share one dtype")
    _need(g.dtype == torch.float32 and beta.dtype == torch.float32, "g and beta must be float32")
    _need(q.dim() == 4 and k.shape == q.shape and v.dim() == 4, "q, k [B,L,Hk,D] and v [B,L,Hv,D]")
    B, L, Hk, Dk = q.shape
    _need(v.shape[0] == B and v.shape[1] == L, "v must be [B, L, Hv, D]")
    Hv = v.shape[2]
    _need(g.shape == (B, L, Hv) and beta.shape == (B, L, Hv), "g and beta must be [B, L, Hv]")
    return B, L, Hk, Hv, Dk


def workspace_bytes(B: int, L: int, Hk: int, Hv: int, D: int = D, dtype=torch.bfloat16) -> int:
    code = GDR_BF16 if dtype == torch.bfloat16 else GDR_F32
    return int(lib().gdr_chunk_workspace_bytes(B, L, Hk, Hv, D, code))


def gdr_chunk_fwd(q, k, v, g, beta, S0=None, o=None, S_T=None, ws=None, stream=None,
                  final_state: bool = True, lengths=None):
    """Prefill of B rows: returns (o [B,L,Hv,D] in v's dtype, S_T [B,Hv,D,D] float32 or None).

    lengths: optional CUDA int32 [B], each row's valid tokens (gdr_chunk_fwd_varlen): positions past
    a row's length are pads, not run, and their o is left as it was (pass o to control it)."""
    B, L, Hk, Hv, Dk = _check_inputs(q, k, v, g, beta)
    dt = _dtype_code(q)
    if o is None:
        o = _empty(v.shape, v.dtype, v.device, stream)
    if S_T is None and final_state:
        S_T = _empty((B, Hv, Dk, v.shape[3]), torch.float32, v.device, stream)
    for name, t in (("S0", S0), ("S_T", S_T)):
        if t is not None:
            _need(t.dtype == torch.float32 and t.is_contiguous() and t.is_cuda, f"{name} must be contiguous CUDA float32")
    need = workspace_bytes(B, L, Hk, Hv, Dk, q.dtype)
    if need and ws is None:
        ws = _empty(need, torch.uint8, q.device, stream)
    ws_bytes = 0 if ws is None else ws.numel() * ws.element_size()
    if lengths is None:
        _check(lib().gdr_chunk_fwd(_p(q), _p(k), _p(v), _p(g), _p(beta), _p(S0), _p(o), _p(S_T),
                                   B, L, Hk, Hv, Dk, dt, _p(ws), ws_bytes, _stream(stream)))
    else:
        _need(lengths.is_cuda and lengths.dtype == torch.int32 and lengths.shape == (B,) and lengths.is_contiguous(),
              "lengths must be a contiguous CUDA int32 tensor of shape [B]")
        _check(lib().gdr_chunk_fwd_varlen(_p(q), _p(k), _p(v), _p(g), _p(beta), _p(S0), _p(lengths), _p(o),
                                          _p(S_T), B, L, Hk, Hv, Dk, dt, _p(ws), ws_bytes, _stream(stream)))
    return o, S_T


def gdr_chunk_fwd_gated(q, k, v, g, beta, S0, z, w, eps: float, out=None, S_T=None, ws=None, stream=None,
                        final_state: bool = True):
    """Prefill with the gated RMSNorm fused into its output: returns (out [B,L,Hv,D] bf16 =
    w * o / rms(o) * silu(z), S_T [B,Hv,D,D] float32 or None)."""
    B, L, Hk, Hv, Dk = _check_inputs(q, k, v, g, beta)
    dt = _dtype_code(q)
    _need(z.is_cuda and z.dtype == torch.bfloat16 and z.shape == v.shape and z.is_contiguous(), "z: contiguous CUDA bf16 like v")
    _need(w.is_cuda and w.dtype == torch.float32 and w.shape == (Dk,) and w.is_contiguous(), "w: contiguous CUDA float32 [D]")
    if out is None:
        out = _empty(v.shape, v.dtype, v.device, stream)
    if S_T is None and final_state:
        S_T = _empty((B, Hv, Dk, v.shape[3]), torch.float32, v.device, stream)
    need = workspace_bytes(B, L, Hk, Hv, Dk, q.dtype)
    if need and ws is None:
        ws = _empty(need, torch.uint8, q.device, stream)
    ws_bytes = 0 if ws is None else ws.numel() * ws.element_size()
    _check(lib().gdr_chunk_fwd_gated(_p(q), _p(k), _p(v), _p(g), _p(beta), _p(S0), _p(z), _p(w), float(eps), _p(out),
                                     _p(S_T), B, L, Hk, Hv, Dk, dt, _p(ws), ws_bytes, _stream(stream)))
    return out, S_T


def fork_workspace_bytes(F: int, L_pad: int, Hk: int, Hv: int, D: int = D, dtype=torch.bfloat16) -> int:
    code = GDR_BF16 if dtype == torch.bfloat16 else GDR_F32
    return int(lib().gdr_fork_workspace_bytes(F, L_pad, Hk, Hv, D, code))


def gdr_fork_fwd(q, k, v, g, beta, trunk, trunk_idx, o=None, states_out=None, stream=None,
                 keep: bool = True, ws=None):
    """Fork batch: returns (o [F,L_pad,Hv,D], states_out [F,Hv,D,D] or None)."""
    F, L, Hk, Hv, Dk = _check_inputs(q, k, v, g, beta)
    dt = _dtype_code(q)
    _need(trunk.is_cuda and trunk.dtype == torch.float32 and trunk.is_contiguous(), "trunk: CUDA float32")
    _need(trunk_idx.is_cuda and trunk_idx.dtype == torch.int64 and trunk_idx.shape == (F,), "trunk_idx: CUDA int64 [F]")
    if o is None:
        o = _empty(v.shape, v.dtype, v.device, stream)
    if states_out is None and keep:
        states_out = _empty((F, Hv, Dk, v.shape[3]), torch.float32, v.device, stream)
    need = fork_workspace_bytes(F, L, Hk, Hv, Dk, q.dtype)
    if need and ws is None:
        ws = _empty(need, torch.uint8, q.device, stream)
    ws_bytes = 0 if ws is None else ws.numel() * ws.element_size()
    _check(lib().gdr_fork_fwd(_p(q), _p(k), _p(v), _p(g), _p(beta), _p(trunk), _p(trunk_idx),
                              trunk.shape[0], _p(o), _p(states_out), F, L, Hk, Hv, Dk, dt,
                              _p(ws), ws_bytes, _stream(stream)))
    return o, states_out


def gdr_decode_step(q, k, v, g, beta, states, o=None, stream=None):
    """One token per row; ``states`` [F,Hv,D,D] float32 is updated in place. Returns o [F,1,Hv,D]."""
    F, L, Hk, Hv, Dk = _check_inputs(q, k, v, g, beta)
    _need(L == 1, "decode takes one token per row")
    dt = _dtype_code(q)
    _need(states.is_cuda and states.dtype == torch.float32 and states.is_contiguous(), "states: CUDA float32")
    if o is None:
        o = _empty(v.shape, v.dtype, v.device, stream)
    _check(lib().gdr_decode_step(_p(q), _p(k), _p(v), _p(g), _p(beta), _p(states), _p(o),
                                 F, Hk, Hv, Dk, dt, _stream(stream)))
    return o


def gdr_prologue(mixed, conv_w, a, b, A_log, dt_bias, Hk: int, Hv: int, tail=None, lengths=None,
                 q=None, k=None, v=None, g=None, beta=None, new_tail=None, stream=None,
                 keep_tail: bool = True):
    """GDN prologue: conv + SiLU of ``mixed`` [B,L,C] bf16 (with the carry ``tail`` [B,K-1,C]),
    gates from ``a``, ``b`` [B,L,Hv]. Returns (q, k, v, g, beta, new_tail or None)."""
    for name, t in (("mixed", mixed), ("conv_w", conv_w), ("a", a), ("b", b), ("A_log", A_log), ("dt_bias", dt_bias)):
        _need(isinstance(t, torch.Tensor) and t.is_cuda and t.is_contiguous(), f"{name} must be a contiguous CUDA tensor")
    _need(mixed.dtype == torch.bfloat16 and mixed.dim() == 3, "mixed must be bfloat16 [B, L, C]")
    B, L, C = mixed.shape
    _need(C == (2 * Hk + Hv) * D, f"mixed has {C} channels, expected (2 Hk + Hv) D = {(2 * Hk + Hv) * D}")
    _need(conv_w.dtype == torch.float32 and conv_w.dim() == 2 and conv_w.shape[0] == C, "conv_w must be float32 [C, K]")
    K = conv_w.shape[1]
    for name, t in (("a", a), ("b", b)):
        _need(t.dtype == torch.float32 and t.shape == (B, L, Hv), f"{name} must be float32 [B, L, Hv]")
    for name, t in (("A_log", A_log), ("dt_bias", dt_bias)):
        _need(t.dtype == torch.float32 and t.shape == (Hv,), f"{name} must be float32 [Hv]")
    if tail is not None:
        _need(tail.is_cuda and tail.is_contiguous() and tail.dtype == torch.bfloat16 and tail.shape == (B, K - 1, C),
              "tail must be contiguous CUDA bfloat16 [B, K-1, C]")
    if lengths is not None:
        _need(lengths.is_cuda and lengths.dtype == torch.int32 and lengths.shape == (B,), "lengths must be CUDA int32 [B]")
    dev = mixed.device
    if q is None:
        q = _empty((B, L, Hk, D), torch.bfloat16, dev, stream)
    if k is None:
        k = _empty((B, L, Hk, D), torch.bfloat16, dev, stream)
    if v is None:
        v = _empty((B, L, Hv, D), torch.bfloat16, dev, stream)
    if g is None:
        g = _empty((B, L, Hv), torch.float32, dev, stream)
    if beta is None:
        beta = _empty((B, L, Hv), torch.float32, dev, stream)
    if new_tail is None and keep_tail and K > 1:
        new_tail = _empty((B, K - 1, C), torch.bfloat16, dev, stream)
    _check(lib().gdr_prologue(_p(mixed), _p(tail), _p(conv_w), _p(a), _p(b), _p(A_log), _p(dt_bias), _p(lengths),
                              _p(q), _p(k), _p(v), _p(g), _p(beta), _p(new_tail), B, L, Hk, Hv, D, K,
                              _stream(stream)))
    return q, k, v, g, beta, new_tail


def prologue_workspace_bytes(B: int, L: int, Hk: int, Hv: int, K: int = 4, D: int = D) -> int:
    return int(lib().gdr_chunk_fwd_prologue_workspace_bytes(B, L, Hk, Hv, D, K))


def gdr_chunk_fwd_prologue(mixed, conv_w, a, b, A_log, dt_bias, Hk: int, Hv: int, S0=None, tail=None,
                           o=None, S_T=None, new_tail=None, ws=None, stream=None, final_state: bool = True,
                           keep_tail: bool = True):
    """The GDN prologue fused into the bf16 prefill: gdr_prologue(mixed, ...) then gdr_chunk_fwd on its
    outputs, in one pass. Returns (o [B,L,Hv,D] bf16, S_T [B,Hv,D,D] float32 or None, new_tail
    [B,3,C] bf16 or None)."""
    for name, t in (("mixed", mixed), ("conv_w", conv_w), ("a", a), ("b", b), ("A_log", A_log), ("dt_bias", dt_bias)):
        _need(isinstance(t, torch.Tensor) and t.is_cuda and t.is_contiguous(), f"{name} must be a contiguous CUDA tensor")
    _need(mixed.dtype == torch.bfloat16 and mixed.dim() == 3, "mixed must be bfloat16 [B, L, C]")
    B, L, C = mixed.shape
    _need(C == (2 * Hk + Hv) * D, f"mixed has {C} channels, expected (2 Hk + Hv) D = {(2 * Hk + Hv) * D}")
    _need(conv_w.dtype == torch.float32 and conv_w.dim() == 2 and conv_w.shape[0] == C, "conv_w must be float32 [C, K]")
    K = conv_w.shape[1]
    for name, t in (("a", a), ("b", b)):
        _need(t.dtype == torch.float32 and t.shape == (B, L, Hv), f"{name} must be float32 [B, L, Hv]")
    for name, t in (("A_log", A_log), ("dt_bias", dt_bias)):
        _need(t.dtype == torch.float32 and t.shape == (Hv,), f"{name} must be float32 [Hv]")
    if tail is not None:
        _need(tail.is_cuda and tail.is_contiguous() and tail.dtype == torch.bfloat16 and tail.shape == (B, K - 1, C),
              "tail must be contiguous CUDA bfloat16 [B, K-1, C]")
    for name, t in (("S0", S0), ("S_T", S_T)):
        if t is not None:
            _need(t.dtype == torch.float32 and t.is_contiguous() and t.is_cuda and t.shape == (B, Hv, D, D),
                  f"{name} must be contiguous CUDA float32 [B, Hv, D, D]")
    dev = mixed.device
    if o is None:
        o = _empty((B, L, Hv, D), torch.bfloat16, dev, stream)
    if S_T is None and final_state:
        S_T = _empty((B, Hv, D, D), torch.float32, dev, stream)
    if new_tail is None and keep_tail and K > 1:
        new_tail = _empty((B, K - 1, C), torch.bfloat16, dev, stream)
    need = prologue_workspace_bytes(B, L, Hk, Hv, K)
    if ws is None and need:
        ws = _empty(need, torch.uint8, dev, stream)
    ws_bytes = 0 if ws is None else ws.numel() * ws.element_size()
    _check(lib().gdr_chunk_fwd_prologue(_p(mixed), _p(tail), _p(conv_w), _p(a), _p(b), _p(A_log), _p(dt_bias),
                                        _p(S0), _p(o), _p(S_T), _p(new_tail), B, L, Hk, Hv, D, K, _p(ws), ws_bytes,
                                        _stream(stream)))
    return o, S_T, new_tail


def gdr_gated_rmsnorm(x, z, w, eps: float = 1e-6, out=None, stream=None):
    """Gated RMSNorm over the last dimension (D = 128) of ``x`` with gate ``z`` (both bf16, same
    shape, e.g. o [B, L, Hv, D]) and weight ``w`` [D] float32; returns ``out`` (x's shape, bf16)."""
    for name, t in (("x", x), ("z", z), ("w", w)):
        _need(isinstance(t, torch.Tensor) and t.is_cuda and t.is_contiguous(), f"{name} must be a contiguous CUDA tensor")
    _need(x.dtype == torch.bfloat16 and z.dtype == torch.bfloat16 and z.shape == x.shape, "x and z: bfloat16, same shape")
    _need(w.dtype == torch.float32 and w.shape == (x.shape[-1],), "w must be float32 [D]")
    if out is None:
        out = _empty(x.shape, x.dtype, x.device, stream)
    rows = x.numel() // x.shape[-1]
    _check(lib().gdr_gated_rmsnorm(_p(x), _p(z), _p(w), float(eps), _p(out), rows, x.shape[-1], _stream(stream)))
    return out


def backward_workspace_bytes(B: int, L: int, Hk: int, Hv: int, D: int = D) -> int:
    return int(lib().gdr_backward_workspace_bytes(B, L, Hk, Hv, D))


def gdr_backward(q, k, v, g, beta, S0, dO, dS_T=None, ws=None, stream=None, want_dS0: bool = True):
    """Gradients of gdr_chunk_fwd: returns (dq, dk [B,L,Hk,D], dv [B,L,Hv,D], dg, dbeta [B,L,Hv],
    dS0 [B,Hv,D,D] or None), all float32, given dO (o's shape, q's dtype) and dS_T (None = 0)."""
    B, L, Hk, Hv, Dk = _check_inputs(q, k, v, g, beta)
    dt = _dtype_code(q)
    _need(isinstance(dO, torch.Tensor) and dO.is_cuda and dO.is_contiguous() and dO.dtype == q.dtype
          and dO.shape == v.shape, "dO must be a contiguous CUDA tensor of v's shape and q's dtype")
    for name, t in (("S0", S0), ("dS_T", dS_T)):
        if t is not None:
            _need(t.dtype == torch.float32 and t.is_contiguous() and t.is_cuda and t.shape == (B, Hv, Dk, v.shape[3]),
                  f"{name} must be contiguous CUDA float32 [B, Hv, D, D]")
    f32 = torch.float32, q.device, stream
    dq = _empty(q.shape, *f32)
    dk = _empty(k.shape, *f32)
    dv = _empty(v.shape, *f32)
    dg = _empty(g.shape, *f32)
    dbeta = _empty(beta.shape, *f32)
    dS0 = _empty((B, Hv, Dk, v.shape[3]), *f32) if want_dS0 else None
    need = backward_workspace_bytes(B, L, Hk, Hv, Dk)
    if ws is None:
        ws = _empty(max(need, 1), torch.uint8, q.device, stream)
    ws_bytes = ws.numel() * ws.element_size()
    _check(lib().gdr_backward(_p(q), _p(k), _p(v), _p(g), _p(beta), _p(S0), _p(dO), _p(dS_T), _p(dq), _p(dk),
                              _p(dv), _p(dg), _p(dbeta), _p(dS0), B, L, Hk, Hv, Dk, dt, _p(ws), ws_bytes,
                              _stream(stream)))
    return dq, dk, dv, dg, dbeta, dS0


def backward_chunked_workspace_bytes(B: int, L: int, Hk: int, Hv: int, D: int = 128) -> int:
    return int(lib().gdr_backward_chunked_workspace_bytes(B, L, Hk, Hv, D))


def gdr_chunk_fwd_save(q, k, v, g, beta, S0=None, saved=None, o=None, S_T=None, stream=None,
                       final_state: bool = True):
    """gdr_chunk_fwd for bf16 rows that also keeps, in ``saved`` (a uint8 CUDA buffer of
    backward_chunked_workspace_bytes; allocated if None), what gdr_backward_chunked would recompute.
    Returns (o, S_T or None, saved); pass saved to gdr_backward_chunked(..., saved=saved)."""
    B, L, Hk, Hv, Dk = _check_inputs(q, k, v, g, beta)
    _need(q.dtype == torch.bfloat16, "gdr_chunk_fwd_save takes bf16 q, k, v")
    if o is None:
        o = _empty(v.shape, v.dtype, v.device, stream)
    if S_T is None and final_state:
        S_T = _empty((B, Hv, Dk, v.shape[3]), torch.float32, v.device, stream)
    for name, t in (("S0", S0), ("S_T", S_T)):
        if t is not None:
            _need(t.dtype == torch.float32 and t.is_contiguous() and t.is_cuda, f"{name} must be contiguous CUDA float32")
    need = backward_chunked_workspace_bytes(B, L, Hk, Hv, Dk)
    if saved is None:
        saved = _empty(max(need, 1), torch.uint8, q.device, stream)
    _check(lib().gdr_chunk_fwd_save(_p(q), _p(k), _p(v), _p(g), _p(beta), _p(S0), _p(o), _p(S_T), B, L, Hk, Hv, Dk,
                                    _dtype_code(q), _p(saved), saved.numel() * saved.element_size(), _stream(stream)))
    return o, S_T, saved


def gdr_backward_chunked(q, k, v, g, beta, S0, dO, dS_T=None, ws=None, stream=None, want_dS0: bool = True,
                         saved=None):
    """gdr_backward's gradients for bf16 q, k, v, dO, computed chunk by chunk on the tensor cores
    (bf16-path accuracy); same arguments and results. With ``saved`` (the buffer gdr_chunk_fwd_save
    filled on the same q, k, v, g, beta, S0) the forward passes are not run again
    (gdr_backward_chunked_saved)."""
    B, L, Hk, Hv, Dk = _check_inputs(q, k, v, g, beta)
    _need(q.dtype == torch.bfloat16, "gdr_backward_chunked takes bf16 q, k, v, dO (float32: gdr_backward)")
    _need(isinstance(dO, torch.Tensor) and dO.is_cuda and dO.is_contiguous() and dO.dtype == q.dtype
          and dO.shape == v.shape, "dO must be a contiguous CUDA tensor of v's shape and q's dtype")
    for name, t in (("S0", S0), ("dS_T", dS_T)):
        if t is not None:
            _need(t.dtype == torch.float32 and t.is_contiguous() and t.is_cuda and t.shape == (B, Hv, Dk, v.shape[3]),
                  f"{name} must be contiguous CUDA float32 [B, Hv, D, D]")
    f32 = torch.float32, q.device, stream
    dq = _empty(q.shape, *f32)
    dk = _empty(k.shape, *f32)
    dv = _empty(v.shape, *f32)
    dg = _empty(g.shape, *f32)
    dbeta = _empty(beta.shape, *f32)
    dS0 = _empty((B, Hv, Dk, v.shape[3]), *f32) if want_dS0 else None
    need = backward_chunked_workspace_bytes(B, L, Hk, Hv, Dk)
    if saved is not None:
        _need(ws is None, "pass either ws or saved")
        ws = saved
    if ws is None:
        ws = _empty(max(need, 1), torch.uint8, q.device, stream)
    ws_bytes = ws.numel() * ws.element_size()
    fn = lib().gdr_backward_chunked_saved if saved is not None else lib().gdr_backward_chunked
    _check(fn(_p(q), _p(k), _p(v), _p(g), _p(beta), _p(S0), _p(dO), _p(dS_T), _p(dq), _p(dk), _p(dv), _p(dg),
              _p(dbeta), _p(dS0), B, L, Hk, Hv, Dk, _dtype_code(q), _p(ws), ws_bytes, _stream(stream)))
    return dq, dk, dv, dg, dbeta, dS0


# --------------------------------------------------------------------------------------------------
# softmax-attention layers: drafted tokens over a cache of pages
#
# A decoding step makes these calls once a layer, on kernels of a few microseconds: their checks and
# marshalling are compiled (csrc/gdr_bind.cpp) and raise ValueError for a tensor of the wrong device (all
# of them are on the current one), dtype, shape or layout, GdrError for what the library refuses.
# --------------------------------------------------------------------------------------------------
_bind_mod = None


def _bind():
    global _bind_mod
    if _bind_mod is None:
        lib()
        try:
            from . import _gdr_bind
        except ImportError as e:
            raise RuntimeError("the compiled binding _gdr_bind is missing: build it with __graft_entry__.build() "
                               f"or python -m gated_deltanet_rule_gb300.build ({e})") from e
        _bind_mod = _gdr_bind
    return _bind_mod


def _raw(stream):
    return None if stream is None else stream.cuda_stream


def gdr_qk_norm_rope(q, k, q_w, k_w, inv_freq, pos, eps: float = 1e-6, interleaved: bool = False, q_out=None,
                     k_out=None, stream=None):
    """RMS norm of every head of q [B,N,Hq,D] and k [B,N,Hk,D] (views of one projection are read in
    place) and the rotation of its first R = 2 len(inv_freq) elements by pos [B,N] int32 times inv_freq
    (float64). Returns (q_out, k_out), contiguous, in q's dtype."""
    return _bind().norm_rope(q, k, q_w, k_w, inv_freq, pos, eps, interleaved, q_out, k_out, _raw(stream))


def gdr_qk_norm_rope_append(q, k, v, q_w, k_w, inv_freq, pos, k_pages, v_pages, table, ctx, lengths=None,
                            eps: float = 1e-6, interleaved: bool = False, q_out=None, stream=None):
    """gdr_qk_norm_rope that leaves the keys, and v as it is, in the pages of table [B,M] at positions
    ctx[b] + i (i < lengths[b] where given). Returns q_out."""
    return _bind().norm_rope_append(q, k, q_w, k_w, inv_freq, pos, v, k_pages, v_pages, table, ctx, lengths, eps,
                                    interleaved, q_out, _raw(stream))


def gdr_qk_norm_rope_backward(q, k, q_w, k_w, inv_freq, pos, dq_out, dk_out, eps: float = 1e-6,
                              interleaved: bool = False, ws=None, stream=None):
    """Gradients of gdr_qk_norm_rope from dq_out, dk_out (contiguous, q's dtype): (dq, dk, dq_w, dk_w),
    all float32."""
    return _bind().norm_rope_backward(q, k, q_w, k_w, inv_freq, pos, dq_out, dk_out, eps, interleaved, ws, _raw(stream))


def tree_attn_workspace_bytes(D: int = D) -> int:
    return int(lib().gdr_tree_attn_workspace_bytes(D))


def gdr_tree_attn(q, k_pages, v_pages, table, ctx, lengths=None, mask=None, scale: float | None = None, o=None,
                  lse=None, want_lse: bool = False, ws=None, stream=None):
    """Attention of the nodes q [B,N,Hq,D] bf16 over each row's ctx[b] positions and the nodes that
    mask [B,N,ceil(N/64)] int64 (bit j: node i sees node j; None: nodes 0 .. i) lets them see, the pages
    already holding the nodes' keys and values. scale defaults to D^-1/2. Returns o, or (o, lse [B,N,Hq]
    float32) with want_lse or lse given."""
    return _bind().tree_attn(q, k_pages, v_pages, table, ctx, lengths, mask, scale, o, lse, want_lse, ws, _raw(stream))


def gdr_verify_draft(tokens, parents, lengths, p, q, u, u_next, path=None, n_path=None, next_token=None, stream=None):
    """Walks each row's tree of drafted tokens (tokens, parents [B,N] int32, lengths [B]) against the
    target's probabilities p [B,N,V] and the drafts' q [B,N,V] (None: given drafts) with the uniform
    numbers u [B,N], u_next [B]. Returns (path [B,N] of accepted nodes, root first, -1 after them;
    n_path [B]; next_token [B])."""
    return _bind().verify(tokens, parents, lengths, p, q, u, u_next, path, n_path, next_token, _raw(stream))


def cache_workspace_bytes(F: int, M: int) -> int:
    return int(lib().gdr_cache_workspace_bytes(F, M))


def gdr_cache_reserve(table, ctx, refs, rows, extra: int, page: int, ws=None, stream=None) -> None:
    """Gives rows (int32 [F]) pages so that ctx + extra positions of each fit; table, refs in place."""
    _bind().cache_reserve(table, ctx, refs, rows, extra, page, ws, _raw(stream))


def gdr_cache_fork(k_cache, v_cache, table, ctx, refs, src, dst, ws=None, stream=None) -> None:
    """Row dst[f] becomes a copy of row src[f]: full pages shared, the last one copied. In place."""
    _bind().cache_fork(k_cache, v_cache, table, ctx, refs, src, dst, ws, _raw(stream))


def gdr_cache_free(table, ctx, refs, rows, stream=None) -> None:
    """Gives the pages of rows (int32 [F]) back; table, ctx, refs in place."""
    _bind().cache_free(table, ctx, refs, rows, _raw(stream))


def gdr_cache_compact(k_cache, v_cache, table, ctx, path, n_path, new_ctx=None, stream=None):
    """Moves the entries of the accepted paths (gdr_verify_draft's path, n_path) to the front of their
    rows in every layer; returns new_ctx = ctx + n_path (which may not be ctx itself)."""
    return _bind().cache_compact(k_cache, v_cache, table, ctx, path, n_path, new_ctx, _raw(stream))


def gdr_sync_status(stream=None) -> None:
    """Synchronise the stream and raise if a kernel recorded a device-side error."""
    _check(lib().gdr_sync_status(_stream(stream)))


def kernel_names() -> list[str]:
    names, i = [], 0
    while True:
        n = lib().gdr_kernel_name(i)
        if n is None:
            return names
        names.append(n.decode())
        i += 1


def debug_set_wait_budget(cycles: int) -> None:
    """Testing aid: cycles a kernel wait may take before it gives up (0: at once; < 0: default)."""
    _check(lib().gdr_debug_set_wait_budget(int(cycles)))


def stage_timer_enable(on: bool = True, capacity: int = 8192) -> None:
    _check(lib().gdr_stage_timer_enable(int(on), int(capacity)))


def stage_timer_collect() -> dict:
    """{kernel name: (total ms, launches)} for the launches recorded since the last collect."""
    names = kernel_names()
    n = len(names)
    ms = (ctypes.c_double * n)()
    cnt = (ctypes.c_int * n)()
    _check(lib().gdr_stage_timer_collect(ms, cnt, n))
    return {names[i]: (ms[i], cnt[i]) for i in range(n)}
