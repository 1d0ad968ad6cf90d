"""GB300 gated delta rule: thin Python binding over libgdr.so (include/gdr.h).

Argument marshalling only -- every step of the computation runs in the CUDA
kernels behind the C ABI.  Tensors are torch CUDA tensors, contiguous, in the
layouts of the header; the current torch stream is passed as the stream.  If
the library is missing or fails to load, every call raises: there is no CPU
or PyTorch fallback.

    out, final = chunk_fwd(q, k, v, g, beta, a_min, init_state=None, chunk=64)
    out        = decode_step(q, k, v, g, beta, a_min, state)   # state in place

chunk_fwd and chunk_fwd_varlen take the two-kernel path (a parallel chunk
preparation into a workspace, then the state chain) when it applies, with the
workspace from torch's caching allocator; workspace=None selects the
single-launch path, a uint8 CUDA tensor supplies the workspace.
"""
from __future__ import annotations

import contextlib
import ctypes
import os

import torch

from . import build as _build

__all__ = ["GdrError", "load", "chunk_fwd", "decode_step", "chunk_decay", "chunk_wy",
           "chunk_state", "chunk_output", "chunk_fwd_kernels", "chunk_fwd_path", "chunk_fwd_varlen",
           "chunk_fwd_workspace_size", "chunk_fwd_varlen_workspace_size", "last_device_error",
           "status_string", "version", "library_path", "STATUS", "PATHS", "OPTIONS",
           "set_option", "get_option", "option", "mla_decode", "mla_decode_workspace_size",
           "chunk_bwd", "chunk_bwd_workspace_size", "chunk_saved_size", "chunk_fwd_train",
           "chunk_bwd_saved", "page_plan", "kv8_append", "kv8_attn", "kv8_attn_workspace_size",
           "KV8", "kv8_shared_plan", "kv8_attn_shared", "kv8_attn_shared_workspace_size",
           "qk_norm_rope", "qk_norm_rope_bwd", "qk_norm_rope_bwd_workspace_size", "NORM", "PAIRS"]

DECAY = {"affine": 0, "log": 1}   # gdr_decay_t
STATUS = {0: "GDR_OK", 1: "GDR_ERR_INVALID_ARG", 2: "GDR_ERR_UNSUPPORTED", 3: "GDR_ERR_RANGE",
          4: "GDR_ERR_CUDA", 5: "GDR_ERR_TIMEOUT"}
DTYPE = {torch.float32: 0, torch.bfloat16: 1}
KV8 = {torch.float8_e4m3fn: 0, torch.int8: 1}   # gdr_kv8_t
NORM = {None: 0, "none": 0, "rms": 1, "l2": 2}  # gdr_norm_t
PAIRS = {"half": 0, "adjacent": 1}              # gdr_rope_t
# gdr_option_t
OPTIONS = {"wait_limit_ns": 0, "fused_variant": 1, "chain_split": 2, "segments": 3,
           "bwd_variant": 4, "shared_least": 5}

_lib = None


class GdrError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        self.name = STATUS.get(code, str(code))
        msg = status_string(code) if _lib is not None else self.name
        super().__init__(f"{where}: {self.name} ({msg})")


def library_path() -> str:
    return _build.LIB


def load(build_if_missing: bool = False) -> ctypes.CDLL:
    """Load libgdr.so (optionally building it first).  Raises if unavailable."""
    global _lib
    if _lib is not None:
        return _lib
    path = _build.LIB
    if not os.path.exists(path):
        if not build_if_missing:
            raise RuntimeError(f"libgdr.so not built ({path}); run __graft_entry__.build() or "
                               "python -m gated_delta_rule_gdr_gb300.build")
        _build.build()
    lib = ctypes.CDLL(path)
    vp, i, f, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
    i64 = ctypes.c_int64
    sig = {
        "gdr_chunk_fwd": [vp, vp, vp, vp, vp, f, vp, vp, vp, i, i, i, i, i, i, i, vp],
        "gdr_chunk_fwd_ws": [vp, vp, vp, vp, vp, f, vp, vp, vp, i, i, i, i, i, i, i, vp, sz, vp],
        "gdr_chunk_fwd_varlen_ws": [vp, vp, vp, vp, vp, f, vp, vp, vp, vp, i, i, i, i, i, i, i, vp,
                                    sz, vp],
        "gdr_chunk_fwd_ws_path": [i, i, i, i, i, i, f, i],
        "gdr_chunk_fwd_ex": [vp, vp, vp, vp, vp, i, f, vp, vp, vp, i, i, i, i, i, i, i, vp, sz, vp],
        "gdr_decode_step_ex": [vp, vp, vp, vp, vp, i, f, vp, vp, i, i, i, i, i, vp],
        "gdr_chunk_fwd_host": [vp, vp, vp, vp, vp, f, vp, vp, vp, i, i, i, i, i, i, i, vp, sz, vp],
        "gdr_chunk_bwd": [vp, vp, vp, vp, vp, i, f, vp, vp, vp, vp, vp, vp, vp, vp, vp,
                          i, i, i, i, i, i, i, vp, sz, vp],
        "gdr_chunk_fwd_train": [vp, vp, vp, vp, vp, i, f, vp, vp, vp, i, i, i, i, i, i, i, vp, sz,
                                vp, sz, vp],
        "gdr_chunk_bwd_saved": [vp, vp, vp, vp, vp, i, f, vp, vp, vp, vp, vp, vp, vp, vp, vp,
                                i, i, i, i, i, i, i, vp, sz, vp, sz, vp],
        "gdr_chunk_fwd_varlen": [vp, vp, vp, vp, vp, f, vp, vp, vp, vp, i, i, i, i, i, i, i, vp],
        "gdr_chunk_fwd_static": [vp, vp, vp, vp, vp, f, vp, vp, vp, i, i, i, i, i, i, i, vp],
        "gdr_decode_step": [vp, vp, vp, vp, vp, f, vp, vp, i, i, i, i, i, vp],
        "gdr_chunk_decay": [vp, f, vp, i, i, i, vp],
        "gdr_chunk_wy": [vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, vp],
        "gdr_chunk_state": [vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, vp],
        "gdr_chunk_output": [vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, vp],
        "gdr_last_device_error": [vp],
        "gdr_chunk_fwd_kernels": [i, i, i, i, i, i, f, i],
        "gdr_chunk_fwd_path": [i, i, i, i, i, i, f, i],
        "gdr_status_string": [i],
        "gdr_version": [],
        "gdr_set_option": [i, ctypes.c_int64],
        "gdr_mla_decode": [vp, vp, vp, vp, vp, f, vp, i, i, i, i, i, vp, sz, vp],
        "gdr_page_plan": [vp] * 11 + [i] * 5 + [vp],
        "gdr_page_plan_ex": [vp] * 13 + [i] * 5 + [vp],
        "gdr_kv8_append": [vp, vp, i64, i64, vp, vp, vp, vp, vp, i, i, i, i, i, i, i, vp],
        "gdr_kv8_shared_plan": [vp] * 6 + [i] * 4 + [vp],
        "gdr_kv8_attn_shared": [vp, i64] + [vp] * 10 + [f, vp, vp] + [i] * 13 + [vp, sz, vp],
        "gdr_qk_norm_rope": [vp, i64, vp, i64, vp, vp, f, i, vp, vp, i, i, vp, i64, vp, i64] + [i] * 5 + [vp],
        "gdr_qk_norm_rope_bwd": [vp, i64, vp, i64, vp, vp, f, i, vp, vp, i, i, vp, i64, vp, i64, vp, i64, vp,
                                 i64, vp, vp] + [i] * 5 + [vp, sz, vp],
        "gdr_kv8_attn": [vp, i64, vp, vp, vp, vp, vp, vp, vp, f, vp, vp] + [i] * 11 + [vp, sz, vp],
    }
    for name, args in sig.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = ctypes.c_int
    for name in ("gdr_chunk_fwd_workspace_size", "gdr_chunk_fwd_varlen_workspace_size",
                 "gdr_chunk_bwd_workspace_size", "gdr_chunk_fwd_host_buffer_size",
                 "gdr_chunk_saved_size"):
        fn = getattr(lib, name)
        fn.argtypes = [i, i, i, i, i, i, i]
        fn.restype = sz
    lib.gdr_mla_decode_workspace_size.argtypes = [i, i, i, i, i]
    lib.gdr_mla_decode_workspace_size.restype = sz
    lib.gdr_kv8_attn_workspace_size.argtypes = [i] * 7
    lib.gdr_kv8_attn_workspace_size.restype = sz
    lib.gdr_kv8_attn_shared_workspace_size.argtypes = [i] * 9
    lib.gdr_kv8_attn_shared_workspace_size.restype = sz
    lib.gdr_qk_norm_rope_bwd_workspace_size.argtypes = [i]
    lib.gdr_qk_norm_rope_bwd_workspace_size.restype = sz
    lib.gdr_get_option.argtypes = [i]
    lib.gdr_get_option.restype = ctypes.c_int64
    lib.gdr_status_string.restype = ctypes.c_char_p
    lib.gdr_version.restype = ctypes.c_char_p
    _lib = lib
    return lib


def status_string(code: int) -> str:
    return load().gdr_status_string(int(code)).decode()


def version() -> str:
    return load().gdr_version().decode()


def set_option(name: str, value: int) -> None:
    """Set a process-wide option of the library (gdr_set_option): "wait_limit_ns"
    (0 = every device-side wait gives up at once), "fused_variant" (0 auto, 1 one CTA
    per head, 2 cluster pair), "chain_split" (0 auto, 1, 2), "segments" (0 auto, else
    the sequence segments of the two-kernel path), "shared_least" (common tokens from which
    kv8_attn_shared reads them in a pass of their own; 0 by a cost model)."""
    _check(load().gdr_set_option(OPTIONS[name], int(value)), "gdr_set_option")


def get_option(name: str) -> int:
    return int(load().gdr_get_option(OPTIONS[name]))


@contextlib.contextmanager
def option(**values):
    """Set options for the duration of a with-block, then restore them."""
    old = {n: get_option(n) for n in values}
    try:
        for n, val in values.items():
            set_option(n, val)
        yield
    finally:
        for n, val in old.items():
            set_option(n, val)


def _ptr(t):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("libgdr takes CUDA tensors")
    if not t.is_contiguous():
        raise ValueError("libgdr takes contiguous tensors")
    return ctypes.c_void_p(t.data_ptr())


def _stream(device) -> ctypes.c_void_p:
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _check(code: int, where: str):
    if code != 0:
        raise GdrError(code, where)


def _f32(t, name):
    if t is not None and t.dtype != torch.float32:
        raise TypeError(f"{name} must be float32")
    return t


def _workspace(nbytes: int, workspace, device):
    """The workspace to pass: None for the single-launch path, else a uint8 CUDA
    tensor of at least nbytes ("auto": from torch's caching allocator)."""
    if workspace is None or nbytes == 0:
        return None
    if isinstance(workspace, str):
        if workspace != "auto":
            raise ValueError('workspace must be "auto", None or a uint8 CUDA tensor')
        return torch.empty(nbytes, dtype=torch.uint8, device=device)
    if workspace.dtype != torch.uint8 or workspace.numel() < nbytes:
        raise ValueError(f"workspace must be a uint8 tensor of at least {nbytes} bytes")
    return workspace


def chunk_fwd_workspace_size(B, H, T, dk, dv, chunk=64, dtype=torch.bfloat16) -> int:
    """Bytes of workspace the two-kernel path needs (0 where it does not apply)."""
    return int(load().gdr_chunk_fwd_workspace_size(B, H, T, dk, dv, chunk, DTYPE[dtype]))


def chunk_fwd_varlen_workspace_size(S, H, total_T, dk, dv, chunk=64, dtype=torch.bfloat16) -> int:
    """Bytes of workspace the packed two-kernel path needs (0 where it does not apply)."""
    return int(load().gdr_chunk_fwd_varlen_workspace_size(S, H, total_T, dk, dv, chunk, DTYPE[dtype]))


def chunk_fwd(q, k, v, g, beta, a_min: float, init_state=None, *, chunk: int = 64,
              out=None, final_state=None, want_final: bool = True, workspace="auto",
              decay: str = "affine"):
    """Chunked prefill.  q,k [B,H,T,dk], v [B,H,T,dv] (fp32 or bf16), g,beta [B,H,T]
    fp32, init_state [B,H,dk,dv] fp32 or None.  Returns (out, final_state).
    decay "log": a_min is the log-domain floor g_min <= 0, log alpha = g_min sigmoid(g)."""
    lib = load()
    B, H, T, dk = q.shape
    dv = v.shape[-1]
    if q.dtype not in DTYPE or k.dtype != q.dtype or v.dtype != q.dtype:
        raise TypeError("q, k, v must share one dtype, float32 or bfloat16")
    _f32(g, "g"), _f32(beta, "beta"), _f32(init_state, "init_state")
    if out is None:
        out = torch.empty((B, H, T, dv), dtype=q.dtype, device=q.device)
    if final_state is None and want_final:
        final_state = torch.empty((B, H, dk, dv), dtype=torch.float32, device=q.device)
    ws = _workspace(chunk_fwd_workspace_size(B, H, T, dk, dv, chunk, q.dtype), workspace, q.device)
    if decay != "affine":
        if decay not in DECAY:
            raise ValueError(f"unknown decay {decay!r}")
        _check(lib.gdr_chunk_fwd_ex(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), DECAY[decay],
                                    float(a_min), _ptr(init_state), _ptr(out), _ptr(final_state),
                                    B, H, T, dk, dv, int(chunk), DTYPE[q.dtype], _ptr(ws),
                                    0 if ws is None else ws.numel(), _stream(q.device)),
               "gdr_chunk_fwd_ex")
    elif ws is None:
        _check(lib.gdr_chunk_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), float(a_min),
                                 _ptr(init_state), _ptr(out), _ptr(final_state), B, H, T, dk, dv,
                                 int(chunk), DTYPE[q.dtype], _stream(q.device)), "gdr_chunk_fwd")
    else:
        _check(lib.gdr_chunk_fwd_ws(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), float(a_min),
                                    _ptr(init_state), _ptr(out), _ptr(final_state), B, H, T, dk,
                                    dv, int(chunk), DTYPE[q.dtype], _ptr(ws), ws.numel(),
                                    _stream(q.device)), "gdr_chunk_fwd_ws")
    return out, final_state


def chunk_fwd_varlen(q, k, v, g, beta, a_min: float, cu_seqlens, init_state=None, *,
                     chunk: int = 64, out=None, final_state=None, want_final: bool = True,
                     workspace="auto"):
    """Chunked prefill over packed sequences.  q,k [total_T,H,dk], v [total_T,H,dv] bf16,
    g,beta [total_T,H] fp32, cu_seqlens int32 [S+1] on the device, init_state [S,H,dk,dv]
    fp32 or None.  Returns (out [total_T,H,dv], final_state [S,H,dk,dv])."""
    lib = load()
    total_T, H, dk = q.shape
    dv = v.shape[-1]
    S = cu_seqlens.numel() - 1
    if q.dtype not in DTYPE or k.dtype != q.dtype or v.dtype != q.dtype:
        raise TypeError("q, k, v must share one dtype")
    if cu_seqlens.dtype != torch.int32 or not cu_seqlens.is_contiguous():
        raise TypeError("cu_seqlens must be a contiguous int32 tensor")
    _f32(g, "g"), _f32(beta, "beta"), _f32(init_state, "init_state")
    if out is None:
        out = torch.empty((total_T, H, dv), dtype=q.dtype, device=q.device)
    if final_state is None and want_final:
        final_state = torch.empty((S, H, dk, dv), dtype=torch.float32, device=q.device)
    ws = _workspace(chunk_fwd_varlen_workspace_size(S, H, total_T, dk, dv, chunk, q.dtype),
                    workspace, q.device)
    if ws is None:
        _check(lib.gdr_chunk_fwd_varlen(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta),
                                        float(a_min), _ptr(init_state), _ptr(out),
                                        _ptr(final_state), _ptr(cu_seqlens), S, H, total_T, dk, dv,
                                        int(chunk), DTYPE[q.dtype], _stream(q.device)),
               "gdr_chunk_fwd_varlen")
    else:
        _check(lib.gdr_chunk_fwd_varlen_ws(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta),
                                           float(a_min), _ptr(init_state), _ptr(out),
                                           _ptr(final_state), _ptr(cu_seqlens), S, H, total_T, dk,
                                           dv, int(chunk), DTYPE[q.dtype], _ptr(ws), ws.numel(),
                                           _stream(q.device)), "gdr_chunk_fwd_varlen_ws")
    return out, final_state


def chunk_fwd_host_buffer_size(B, H, T, dk, dv, chunk=64, dtype=torch.bfloat16) -> int:
    """Bytes of device memory chunk_fwd_host needs (inputs, outputs, workspace)."""
    return int(load().gdr_chunk_fwd_host_buffer_size(B, H, T, dk, dv, chunk, DTYPE[dtype]))


def _host_ptr(t):
    if t is None:
        return None
    if t.is_cuda or not t.is_contiguous():
        raise ValueError("chunk_fwd_host takes contiguous CPU tensors")
    return ctypes.c_void_p(t.data_ptr())


def chunk_fwd_host(q, k, v, g, beta, a_min: float, init_state, out, final_state, device_buffer,
                   *, chunk: int = 64, stream=None):
    """Prefill from host tensors to host tensors (pinned memory for overlap): copies in,
    computes and copies out on ``stream`` (default: the current stream of the buffer's
    device).  ``device_buffer`` is a uint8 CUDA tensor of chunk_fwd_host_buffer_size
    bytes; ``out`` [B,H,T,dv] and ``final_state`` [B,H,dk,dv] (or None) are CPU tensors
    written when the stream reaches the end of the call."""
    lib = load()
    B, H, T, dk = q.shape
    dv = v.shape[-1]
    if q.dtype not in DTYPE or k.dtype != q.dtype or v.dtype != q.dtype or out.dtype != q.dtype:
        raise TypeError("q, k, v, out must share one dtype, float32 or bfloat16")
    _f32(g, "g"), _f32(beta, "beta"), _f32(init_state, "init_state"), _f32(final_state, "final_state")
    if device_buffer.dtype != torch.uint8 or not device_buffer.is_cuda:
        raise ValueError("device_buffer must be a uint8 CUDA tensor")
    st = stream if stream is not None else torch.cuda.current_stream(device_buffer.device)
    _check(lib.gdr_chunk_fwd_host(_host_ptr(q), _host_ptr(k), _host_ptr(v), _host_ptr(g),
                                  _host_ptr(beta), float(a_min), _host_ptr(init_state),
                                  _host_ptr(out), _host_ptr(final_state), B, H, T, dk, dv,
                                  int(chunk), DTYPE[q.dtype], _ptr(device_buffer),
                                  device_buffer.numel(), ctypes.c_void_p(st.cuda_stream)),
           "gdr_chunk_fwd_host")
    return out, final_state


def chunk_bwd_workspace_size(B, H, T, dk, dv, chunk=64, dtype=torch.bfloat16) -> int:
    """Bytes of workspace the backward needs (0 for empty work or unsupported shapes)."""
    return int(load().gdr_chunk_bwd_workspace_size(B, H, T, dk, dv, chunk, DTYPE[dtype]))


def chunk_bwd(q, k, v, g, beta, a_min: float, init_state, d_out, d_final=None, *,
              chunk: int = 64, want_dinit: bool = True, workspace=None, decay: str = "affine"):
    """Gradients of a loss through chunk_fwd: given d_out [B,H,T,dv] (q's dtype) and
    d_final [B,H,dk,dv] fp32 or None, returns (dq, dk, dv, dg, dbeta, dinit) for the
    forward with the same arguments (dinit None unless want_dinit).  workspace: None
    (allocated here) or a uint8 CUDA tensor of at least chunk_bwd_workspace_size bytes."""
    lib = load()
    B, H, T, dk = q.shape
    dv = v.shape[-1]
    if q.dtype not in DTYPE or k.dtype != q.dtype or v.dtype != q.dtype or d_out.dtype != q.dtype:
        raise TypeError("q, k, v, d_out must share one dtype, float32 or bfloat16")
    _f32(g, "g"), _f32(beta, "beta"), _f32(init_state, "init_state"), _f32(d_final, "d_final")
    if decay not in DECAY:
        raise ValueError(f"unknown decay {decay!r}")
    dq, dk_, dv_ = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    dg, db = torch.empty_like(g), torch.empty_like(beta)
    dinit = torch.empty((B, H, dk, dv), dtype=torch.float32, device=q.device) if want_dinit else None
    need = chunk_bwd_workspace_size(B, H, T, dk, dv, chunk, q.dtype)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=q.device)
    elif workspace.dtype != torch.uint8 or workspace.numel() < need:
        raise ValueError(f"workspace must be a uint8 tensor of at least {need} bytes")
    _check(lib.gdr_chunk_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), DECAY[decay],
                             float(a_min), _ptr(init_state), _ptr(d_out), _ptr(d_final),
                             _ptr(dq), _ptr(dk_), _ptr(dv_), _ptr(dg), _ptr(db), _ptr(dinit),
                             B, H, T, dk, dv, int(chunk), DTYPE[q.dtype], _ptr(workspace),
                             workspace.numel(), _stream(q.device)), "gdr_chunk_bwd")
    return dq, dk_, dv_, dg, db, dinit


def chunk_saved_size(B, H, T, dk, dv, chunk=64, dtype=torch.bfloat16) -> int:
    """Bytes of the buffer chunk_fwd_train fills for chunk_bwd_saved (0: not supported)."""
    return int(load().gdr_chunk_saved_size(B, H, T, dk, dv, chunk, DTYPE[dtype]))


def chunk_fwd_train(q, k, v, g, beta, a_min: float, init_state=None, *, chunk: int = 64,
                    out=None, final_state=None, want_final: bool = True, workspace=None,
                    saved=None, decay: str = "affine"):
    """chunk_fwd (bf16, d = 128, chunk 64, two-kernel path) that also keeps every chunk's
    state and W tile for chunk_bwd_saved.  workspace / saved: None (allocated here) or
    uint8 CUDA tensors of at least chunk_fwd_workspace_size / chunk_saved_size bytes.
    Returns (out, final_state, saved)."""
    lib = load()
    B, H, T, dk = q.shape
    dv = v.shape[-1]
    if q.dtype not in DTYPE or k.dtype != q.dtype or v.dtype != q.dtype:
        raise TypeError("q, k, v must share one dtype")
    _f32(g, "g"), _f32(beta, "beta"), _f32(init_state, "init_state")
    if decay not in DECAY:
        raise ValueError(f"unknown decay {decay!r}")
    if out is None:
        out = torch.empty((B, H, T, dv), dtype=q.dtype, device=q.device)
    if final_state is None and want_final:
        final_state = torch.empty((B, H, dk, dv), dtype=torch.float32, device=q.device)
    need_ws = chunk_fwd_workspace_size(B, H, T, dk, dv, chunk, q.dtype)
    need_sv = chunk_saved_size(B, H, T, dk, dv, chunk, q.dtype)
    if workspace is None:
        workspace = torch.empty(max(need_ws, 16), dtype=torch.uint8, device=q.device)
    if saved is None:
        saved = torch.empty(max(need_sv, 16), dtype=torch.uint8, device=q.device)
    for name, t, need in (("workspace", workspace, need_ws), ("saved", saved, need_sv)):
        if t.dtype != torch.uint8 or t.numel() < need:
            raise ValueError(f"{name} must be a uint8 tensor of at least {need} bytes")
    _check(lib.gdr_chunk_fwd_train(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), DECAY[decay],
                                   float(a_min), _ptr(init_state), _ptr(out), _ptr(final_state),
                                   B, H, T, dk, dv, int(chunk), DTYPE[q.dtype], _ptr(workspace),
                                   workspace.numel(), _ptr(saved), saved.numel(),
                                   _stream(q.device)), "gdr_chunk_fwd_train")
    return out, final_state, saved


def chunk_bwd_saved(q, k, v, g, beta, a_min: float, init_state, d_out, saved, d_final=None, *,
                    chunk: int = 64, want_dinit: bool = True, workspace=None,
                    decay: str = "affine"):
    """chunk_bwd reading the states chunk_fwd_train saved (same arguments as that
    forward) instead of recomputing them.  Returns (dq, dk, dv, dg, dbeta, dinit)."""
    lib = load()
    B, H, T, dk = q.shape
    dv = v.shape[-1]
    if q.dtype not in DTYPE or k.dtype != q.dtype or v.dtype != q.dtype or d_out.dtype != q.dtype:
        raise TypeError("q, k, v, d_out must share one dtype")
    _f32(g, "g"), _f32(beta, "beta"), _f32(init_state, "init_state"), _f32(d_final, "d_final")
    if decay not in DECAY:
        raise ValueError(f"unknown decay {decay!r}")
    if saved.dtype != torch.uint8 or not saved.is_cuda:
        raise ValueError("saved must be the uint8 CUDA tensor chunk_fwd_train filled")
    dq, dk_, dv_ = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    dg, db = torch.empty_like(g), torch.empty_like(beta)
    dinit = torch.empty((B, H, dk, dv), dtype=torch.float32, device=q.device) if want_dinit else None
    need = chunk_bwd_workspace_size(B, H, T, dk, dv, chunk, q.dtype)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=q.device)
    elif workspace.dtype != torch.uint8 or workspace.numel() < need:
        raise ValueError(f"workspace must be a uint8 tensor of at least {need} bytes")
    _check(lib.gdr_chunk_bwd_saved(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), DECAY[decay],
                                   float(a_min), _ptr(init_state), _ptr(d_out), _ptr(d_final),
                                   _ptr(dq), _ptr(dk_), _ptr(dv_), _ptr(dg), _ptr(db),
                                   _ptr(dinit), B, H, T, dk, dv, int(chunk), DTYPE[q.dtype],
                                   _ptr(saved), saved.numel(), _ptr(workspace), workspace.numel(),
                                   _stream(q.device)), "gdr_chunk_bwd_saved")
    return dq, dk_, dv_, dg, db, dinit


def decode_step(q, k, v, g, beta, a_min: float, state, *, out=None, decay: str = "affine"):
    """One token for N sequences.  q,k [N,H,dk], v [N,H,dv], g,beta [N,H] fp32,
    state [N,H,dk,dv] fp32 updated in place.  Returns out [N,H,dv]."""
    lib = load()
    N, H, dk = q.shape
    dv = v.shape[-1]
    if q.dtype not in DTYPE or k.dtype != q.dtype or v.dtype != q.dtype:
        raise TypeError("q, k, v must share one dtype, float32 or bfloat16")
    _f32(g, "g"), _f32(beta, "beta"), _f32(state, "state")
    if out is None:
        out = torch.empty((N, H, dv), dtype=q.dtype, device=q.device)
    if decay != "affine":
        if decay not in DECAY:
            raise ValueError(f"unknown decay {decay!r}")
        _check(lib.gdr_decode_step_ex(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), DECAY[decay],
                                      float(a_min), _ptr(state), _ptr(out), N, H, dk, dv,
                                      DTYPE[q.dtype], _stream(q.device)), "gdr_decode_step_ex")
        return out
    _check(lib.gdr_decode_step(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), float(a_min),
                               _ptr(state), _ptr(out), N, H, dk, dv, DTYPE[q.dtype],
                               _stream(q.device)), "gdr_decode_step")
    return out


def chunk_decay(g, a_min: float, chunk: int = 64, *, gamma=None):
    """gamma [BH,T] = chunk-local cumulative product of alpha.  g [..., T] fp32."""
    lib = load()
    T = g.shape[-1]
    BH = g.numel() // max(T, 1) if T else 0
    _f32(g, "g")
    if gamma is None:
        gamma = torch.empty_like(g)
    _check(lib.gdr_chunk_decay(_ptr(g), float(a_min), _ptr(gamma), BH, T, int(chunk),
                               _stream(g.device)), "gdr_chunk_decay")
    return gamma


def chunk_wy(k, v, beta, gamma, chunk: int = 64):
    """U [BH,T,dv], Wk [BH,T,dk] (fp32) of the intra-chunk WY/UT transform."""
    lib = load()
    *lead, T, dk = k.shape
    dv = v.shape[-1]
    BH = k.numel() // max(T * dk, 1)
    U = torch.empty((*lead, T, dv), dtype=torch.float32, device=k.device)
    Wk = torch.empty((*lead, T, dk), dtype=torch.float32, device=k.device)
    _check(lib.gdr_chunk_wy(_ptr(k), _ptr(v), _ptr(beta), _ptr(gamma), _ptr(U), _ptr(Wk), BH, T,
                            dk, dv, int(chunk), DTYPE[k.dtype], _stream(k.device)),
           "gdr_chunk_wy")
    return U, Wk


def chunk_state(k, gamma, U, Wk, init_state=None, chunk: int = 64, want_mn: bool = True):
    """W [BH,T,dv], Mn [BH,NC,dk,dv] (or None), final [BH,dk,dv] of the state pass."""
    lib = load()
    *lead, T, dk = k.shape
    dv = U.shape[-1]
    BH = k.numel() // max(T * dk, 1)
    NC = (T + chunk - 1) // chunk
    W = torch.empty_like(U)
    Mn = (torch.empty((*lead, NC, dk, dv), dtype=torch.float32, device=k.device)
          if want_mn else None)
    fin = torch.empty((*lead, dk, dv), dtype=torch.float32, device=k.device)
    _check(lib.gdr_chunk_state(_ptr(k), _ptr(gamma), _ptr(U), _ptr(Wk), _ptr(init_state),
                               _ptr(W), _ptr(Mn), _ptr(fin), BH, T, dk, dv, int(chunk),
                               DTYPE[k.dtype], _stream(k.device)), "gdr_chunk_state")
    return W, Mn, fin


def chunk_output(q, k, gamma, Mn, W, chunk: int = 64):
    """out [BH,T,dv] in q's dtype from the per-chunk states and W."""
    lib = load()
    *lead, T, dk = q.shape
    dv = W.shape[-1]
    BH = q.numel() // max(T * dk, 1)
    out = torch.empty((*lead, T, dv), dtype=q.dtype, device=q.device)
    _check(lib.gdr_chunk_output(_ptr(q), _ptr(k), _ptr(gamma), _ptr(Mn), _ptr(W), _ptr(out), BH,
                                T, dk, dv, int(chunk), DTYPE[q.dtype], _stream(q.device)),
           "gdr_chunk_output")
    return out


def chunk_fwd_kernels(B, H, T, dk, dv, chunk=64, a_min=0.95, dtype=torch.bfloat16) -> int:
    """How many kernels one chunk_fwd call with these arguments launches."""
    return int(load().gdr_chunk_fwd_kernels(B, H, T, dk, dv, chunk, float(a_min), DTYPE[dtype]))


PATHS = {0: "none", 1: "staged (on the workspace)", 2: "fused one CTA per head",
         3: "fused two-CTA cluster per head", 4: "prep + chain, two CTAs per head",
         5: "prep + chain, one CTA per head", 6: "one-pass CUDA-core kernel",
         7: "prep + segment maps + scan + chain over sequence segments"}


def chunk_fwd_path(B, H, T, dk, dv, chunk=64, a_min=0.95, dtype=torch.bfloat16,
                   workspace: bool = True) -> int:
    """Which path one chunk_fwd call with these arguments takes on the current
    device (see PATHS; -1 = rejected); workspace=False: the single-launch path."""
    fn = load().gdr_chunk_fwd_ws_path if workspace else load().gdr_chunk_fwd_path
    return int(fn(B, H, T, dk, dv, chunk, float(a_min), DTYPE[dtype]))


def mla_decode_workspace_size(N, H, Lmax, dc=512, dh=128) -> int:
    """Bytes of workspace one latent-attention decode step needs (0 if unsupported)."""
    return int(load().gdr_mla_decode_workspace_size(N, H, Lmax, dc, dh))


def mla_decode(q_abs, ckv, seqlens, w_uv, gate, scale: float, *, out=None, workspace=None):
    """One decode step of gated multi-head latent attention.  q_abs [N,H,dc] bf16 (the
    query with the key up-projection absorbed), ckv [N,Lmax,dc] bf16 (latent cache),
    seqlens [N] int32 on the device, w_uv [H,dh,dc] bf16, gate [N,H,dh] fp32 (the gate's
    pre-activation).  Returns out [N,H,dh] bf16.  workspace: None (from torch's caching
    allocator) or a uint8 CUDA tensor of at least mla_decode_workspace_size bytes."""
    lib = load()
    N, H, dc = q_abs.shape
    Lmax = ckv.shape[1]
    dh = w_uv.shape[1]
    for t, name in ((q_abs, "q_abs"), (ckv, "ckv"), (w_uv, "w_uv")):
        if t.dtype != torch.bfloat16:
            raise TypeError(f"{name} must be bfloat16")
    _f32(gate, "gate")
    if seqlens.dtype != torch.int32:
        raise TypeError("seqlens must be int32")
    if out is None:
        out = torch.empty((N, H, dh), dtype=torch.bfloat16, device=q_abs.device)
    need = mla_decode_workspace_size(N, H, Lmax, dc, dh)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=q_abs.device)
    elif workspace.dtype != torch.uint8 or workspace.numel() < need:
        raise ValueError(f"workspace must be a uint8 tensor of at least {need} bytes")
    _check(lib.gdr_mla_decode(_ptr(q_abs), _ptr(ckv), _ptr(seqlens), _ptr(w_uv), _ptr(gate),
                              float(scale), _ptr(out), N, H, Lmax, dc, dh, _ptr(workspace),
                              workspace.numel(), _stream(q_abs.device)), "gdr_mla_decode")
    return out


def last_device_error(device=None) -> int:
    """Synchronise the current stream and return (and clear) the device error word
    as a status code (0 = ok, 5 = a bounded wait timed out)."""
    lib = load()
    return int(lib.gdr_last_device_error(_stream(device)))


# ---- the paged 8-bit cache of the exact-attention layers
#
# These run once a layer for every token served, and their small calls take a few
# microseconds on the device: the checks below read each property of a tensor once, and the
# stream's handle is taken without building a Stream object (by a function that a torch build
# without CUDA does not have, so it is looked up when a call needs it).

def _raw_stream(index):
    return torch._C._cuda_getCurrentRawStream(index)


def _all_here(*tensors):
    """The tensors (None: none) are on the current device, where the kernels are launched."""
    here = torch._C._cuda_getDevice()
    for t in tensors:
        if t is not None and t.get_device() != here:
            raise ValueError(f"a tensor is on {t.device}, the current device is cuda:{here}")
    return here


def _int(t, name, shape=None):
    """Device pointer of a contiguous int32 CUDA tensor."""
    if t.dtype is not torch.int32 or not t.is_cuda or not t.is_contiguous():
        raise TypeError(f"{name} must be a contiguous int32 CUDA tensor")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}")
    return t.data_ptr()


def _rows(t, name):
    """Device pointer and token stride of a [tokens, heads, D] CUDA tensor whose tokens may
    be strided (a slice of a wider projection) and whose heads are contiguous."""
    if t.dtype not in DTYPE:
        raise TypeError(f"{name} must be float32 or bfloat16")
    if not t.is_cuda or t.dim() != 3:
        raise ValueError(f"{name} must be a [tokens, heads, D] CUDA tensor")
    n, h, d = t.shape
    if t.is_contiguous():
        return t.data_ptr(), h * d
    st = t.stride()
    if (st[2] != 1 and d > 1) or (st[1] != d and h > 1):
        raise ValueError(f"{name}: the heads of a token must be contiguous")
    return t.data_ptr(), st[0] if n > 1 else h * d


def _scratch(workspace, need):
    """A workspace that was given: `need` bytes in a row, which an expanded or strided tensor has not."""
    if workspace.dtype is not torch.uint8 or not workspace.is_cuda or workspace.numel() < need or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous uint8 CUDA tensor of at least {need} bytes")


def _kv8_cache(k_cache, v_cache, k_scale, v_scale):
    code = KV8.get(k_cache.dtype)
    if code is None or v_cache.dtype is not k_cache.dtype:
        raise TypeError("k_cache, v_cache must share one dtype, float8_e4m3fn or int8")
    shape = k_cache.shape
    if len(shape) != 4 or v_cache.shape != shape:
        raise ValueError("k_cache, v_cache must be [num_pages, Hkv, page, D]")
    if k_scale.dtype is not torch.float32 or v_scale.dtype is not torch.float32:
        raise TypeError("k_scale, v_scale must be float32")
    if k_scale.shape != shape[:2] or v_scale.shape != shape[:2]:
        raise ValueError("k_scale, v_scale must be [num_pages, Hkv]")
    if not (k_cache.is_cuda and v_cache.is_cuda and k_scale.is_cuda and v_scale.is_cuda
            and k_cache.is_contiguous() and v_cache.is_contiguous()
            and k_scale.is_contiguous() and v_scale.is_contiguous()):
        raise ValueError("libgdr takes contiguous CUDA tensors")
    return code, shape


def page_plan(kv_len, q_len, block_table, free_ring, free_state, page: int, max_tokens: int, held=None):
    """Places for the new tokens of a step, on the device.  kv_len, q_len [S] (q_len < 0:
    finished), block_table [S,W], free_ring [num_pages], free_state [2] = (head, count), all
    int32; block_table and free_ring are updated in place.  Returns int32 (kv_len_out [S],
    cu_q [S+1], slots [max_tokens], positions [max_tokens], granted [S], free_state_out [2]).
    held [S] int32: the pages that each request's row has, where tokens may have been taken back
    (kv_len lowered after refused drafts); held_out [S], the next call's, is then returned too."""
    lib = _lib or load()
    S, W = block_table.shape
    n, dev = int(max_tokens), block_table.device
    i32, empty = torch.int32, torch.empty
    kv, granted = empty(S, dtype=i32, device=dev), empty(S, dtype=i32, device=dev)
    slots, positions = empty(n, dtype=i32, device=dev), empty(n, dtype=i32, device=dev)
    cu, st = empty(S + 1, dtype=i32, device=dev), empty(2, dtype=i32, device=dev)
    held_out = None if held is None else empty(S, dtype=i32, device=dev)
    code = lib.gdr_page_plan_ex(_int(kv_len, "kv_len", (S,)), _int(q_len, "q_len", (S,)),
                                None if held is None else _int(held, "held", (S,)),
                                _int(block_table, "block_table"), _int(free_ring, "free_ring"),
                                _int(free_state, "free_state", (2,)), kv.data_ptr(), cu.data_ptr(),
                                slots.data_ptr(), positions.data_ptr(), granted.data_ptr(),
                                None if held is None else held_out.data_ptr(), st.data_ptr(), S, W, page,
                                free_ring.numel(), n, _raw_stream(dev.index))
    if code:
        raise GdrError(code, "gdr_page_plan")
    out = kv, cu, slots, positions, granted, st
    return out if held is None else (*out, held_out)


def kv8_append(k, v, slots, k_cache, v_cache, k_scale, v_scale) -> None:
    """Quantise the new tokens' k, v [T,Hkv,D] (fp32 or bf16; tokens may be strided) into the
    paged cache at slots [T] int32 (negative: dropped).  k_cache, v_cache [num_pages,Hkv,page,D]
    float8_e4m3fn or int8, k_scale, v_scale [num_pages,Hkv] fp32, all updated in place."""
    lib = _lib or load()
    kv, (N, H, P, D) = _kv8_cache(k_cache, v_cache, k_scale, v_scale)
    (kp, kst), (vp, vst) = _rows(k, "k"), _rows(v, "v")
    T = k.shape[0]
    if k.dtype is not v.dtype:
        raise TypeError("k, v must share one dtype, float32 or bfloat16")
    if k.shape != (T, H, D) or v.shape != (T, H, D):
        raise ValueError(f"k, v must be [T, {H}, {D}]")
    code = lib.gdr_kv8_append(kp, vp, kst, vst, _int(slots, "slots", (T,)), k_cache.data_ptr(),
                              v_cache.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), T, H, D,
                              P, N, DTYPE[k.dtype], kv, _raw_stream(k_cache.device.index))
    if code:
        raise GdrError(code, "gdr_kv8_append")


def kv8_attn_workspace_size(S, max_q, total_q, Hq, Hkv, D, dtype=torch.bfloat16) -> int:
    """Bytes of workspace kv8_attn needs (0: none)."""
    return int(load().gdr_kv8_attn_workspace_size(S, max_q, total_q, Hq, Hkv, D, DTYPE[dtype]))


def kv8_attn(q, k_cache, v_cache, k_scale, v_scale, block_table, kv_len, scale: float, *,
             cu_q=None, max_q: int = None, out=None, want_lse: bool = False, workspace=None):
    """Attention over the paged 8-bit cache.  q [total_q,Hq,D] fp32 or bf16 (tokens may be
    strided), block_table [S,W] and kv_len [S] int32, cu_q [S+1] int32 first query of each
    request (None: one query a request), max_q the most queries of a request (to be given with
    cu_q: it chooses the kernel, and another value costs time).  Query i of n
    sees the first kv_len - n + 1 + i keys.  workspace: None (allocated here) or a uint8 CUDA
    tensor of kv8_attn_workspace_size bytes.  Returns out [total_q,Hq,D], or (out, lse
    [total_q,Hq] fp32) if want_lse."""
    lib = _lib or load()
    kv, (N, Hkv, P, D) = _kv8_cache(k_cache, v_cache, k_scale, v_scale)
    qp, qst = _rows(q, "q")
    T, Hq, dq = q.shape
    S, W = block_table.shape
    dtype, dev = q.dtype, k_cache.device
    if dq != D:
        raise ValueError(f"q must be [total_q, Hq, {D}]")
    if out is None:
        out = torch.empty((T, Hq, D), dtype=dtype, device=dev)
    elif out.dtype is not dtype or out.shape != q.shape or not out.is_cuda or not out.is_contiguous():
        raise ValueError("out must be a contiguous CUDA tensor of q's shape and dtype")
    lse = torch.empty((T, Hq), dtype=torch.float32, device=dev) if want_lse else None
    if max_q is None:
        if cu_q is not None:
            raise ValueError("cu_q wants max_q, the most queries of a request")
        max_q = 1
    elif max_q == 0:            # as a small one: what the lengths say is computed
        max_q = 1
    el = DTYPE[dtype]
    need = lib.gdr_kv8_attn_workspace_size(S, max_q, T, Hq, Hkv, D, el)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=dev)
    else:
        _scratch(workspace, need)
    code = lib.gdr_kv8_attn(qp, qst, k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(),
                            v_scale.data_ptr(), _int(block_table, "block_table"),
                            _int(kv_len, "kv_len", (S,)),
                            None if cu_q is None else _int(cu_q, "cu_q", (S + 1,)), scale,
                            out.data_ptr(), None if lse is None else lse.data_ptr(), S, max_q,
                            T, Hq, Hkv, D, W, P, N, el, kv, workspace.data_ptr(), need,
                            _raw_stream(dev.index))
    if code:
        raise GdrError(code, "gdr_kv8_attn")
    return (out, lse) if want_lse else out


def kv8_shared_plan(block_table, kv_len, cu_group, page: int, *, cu_q=None):
    """What the requests of each group have in common, for kv8_attn_shared (once a step for all
    layers).  block_table [S,W], kv_len [S], cu_group [groups + 1] (group g: the requests cu_group[g]
    up to cu_group[g + 1]; ascending) and cu_q [S+1] (None: one query a request) int32.  A group has in
    common what all of its requests with queries have, so one that leaves the prefix early belongs in
    another.  Returns int32 (shared [S]: tokens of the pages in common, lead [groups]: the request whose row
    they are read by, -1: none)."""
    lib = _lib or load()
    S, W = block_table.shape
    groups, dev = cu_group.numel() - 1, block_table.device
    shared = torch.empty(S, dtype=torch.int32, device=dev)
    lead = torch.empty(max(groups, 0), dtype=torch.int32, device=dev)
    args = (_int(block_table, "block_table"), _int(kv_len, "kv_len", (S,)),
            None if cu_q is None else _int(cu_q, "cu_q", (S + 1,)), _int(cu_group, "cu_group"))
    here = _all_here(block_table, kv_len, cu_q, cu_group)
    code = lib.gdr_kv8_shared_plan(*args, shared.data_ptr(), lead.data_ptr(), S, groups, W, page, _raw_stream(here))
    if code:
        raise GdrError(code, "gdr_kv8_shared_plan")
    return shared, lead


def kv8_attn_shared_workspace_size(S, max_q, groups, max_group_q, total_q, Hq, Hkv, D, dtype=torch.bfloat16) -> int:
    """Bytes of workspace kv8_attn_shared needs."""
    return int(load().gdr_kv8_attn_shared_workspace_size(S, max_q, groups, max_group_q, total_q, Hq, Hkv, D, DTYPE[dtype]))


def kv8_attn_shared(q, k_cache, v_cache, k_scale, v_scale, block_table, kv_len, scale: float, cu_group, shared, lead, *,
                    cu_q=None, max_q: int = None, max_group_q: int, out=None, want_lse: bool = False, workspace=None):
    """kv8_attn for requests that share prefixes: the pages that the requests of a group have in common
    are read once for all of them.  cu_group, shared, lead: kv8_shared_plan's, for these very tables,
    lengths, cu_q and groups (another step's give wrong results); max_group_q: the most queries that the
    requests of a group have together; the rest as kv8_attn.  workspace: None (allocated here) or a uint8
    CUDA tensor of kv8_attn_shared_workspace_size bytes.  Returns out, or (out, lse) if want_lse."""
    lib = _lib or load()
    kv, (N, Hkv, P, D) = _kv8_cache(k_cache, v_cache, k_scale, v_scale)
    qp, qst = _rows(q, "q")
    T, Hq, dq = q.shape
    S, W = block_table.shape
    groups = cu_group.numel() - 1
    dtype, dev = q.dtype, k_cache.device
    if dq != D:
        raise ValueError(f"q must be [total_q, Hq, {D}]")
    if out is None:
        out = torch.empty((T, Hq, D), dtype=dtype, device=dev)
    elif out.dtype is not dtype or out.shape != q.shape or not out.is_cuda or not out.is_contiguous():
        raise ValueError("out must be a contiguous CUDA tensor of q's shape and dtype")
    lse = torch.empty((T, Hq), dtype=torch.float32, device=dev) if want_lse else None
    if max_q is None:
        if cu_q is not None:
            raise ValueError("cu_q wants max_q, the most queries of a request")
        max_q = 1
    # 0 as a small one: what the lengths say is computed
    max_q, max_group_q = max_q or 1, max_group_q or 1
    el = DTYPE[dtype]
    need = lib.gdr_kv8_attn_shared_workspace_size(S, max_q, groups, max_group_q, T, Hq, Hkv, D, el)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=dev)
    else:
        _scratch(workspace, need)
    here = _all_here(q, k_cache, v_cache, k_scale, v_scale, block_table, kv_len, cu_q, cu_group, shared, lead, out,
                     workspace)
    code = lib.gdr_kv8_attn_shared(qp, qst, k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(),
                                   v_scale.data_ptr(), _int(block_table, "block_table"), _int(kv_len, "kv_len", (S,)),
                                   None if cu_q is None else _int(cu_q, "cu_q", (S + 1,)), _int(cu_group, "cu_group"),
                                   _int(shared, "shared", (S,)), _int(lead, "lead", (groups,)), scale, out.data_ptr(),
                                   None if lse is None else lse.data_ptr(), S, max_q, groups, max_group_q, T, Hq, Hkv,
                                   D, W, P, N, el, kv, workspace.data_ptr(), need, _raw_stream(here))
    if code:
        raise GdrError(code, "gdr_kv8_attn_shared")
    return (out, lse) if want_lse else out


# ---- norms of queries and keys with the rotation by position (checks as sparing as above)

def _weights(t, name, D):
    if t is None:
        return None
    if t.dtype is not torch.float32 or not t.is_cuda or not t.is_contiguous():
        raise TypeError(f"{name} must be a contiguous float32 CUDA tensor")
    if t.shape != (D,):
        raise ValueError(f"{name} must have shape ({D},)")
    return t.data_ptr()


def _norm_how(q, k, norm, q_weight, k_weight, positions, freq, pairs):
    """What both directions check: T, heads, D, and the arguments from the weights to the pairs."""
    T, Hq, D = q.shape
    if k is not None and (k.dtype is not q.dtype or k.dim() != 3 or k.shape[0] != T or k.shape[2] != D):
        raise ValueError(f"k must be [{T}, heads, {D}] of q's dtype")
    if norm not in NORM or pairs not in PAIRS:
        raise ValueError(f"unknown norm {norm!r} or pairs {pairs!r}")
    rot, fp = 0, None
    if freq is not None:
        if positions is None:
            raise ValueError("freq wants positions")
        if freq.dtype is not torch.float64 or not freq.is_cuda or not freq.is_contiguous() or freq.dim() != 1:
            raise TypeError("freq must be a contiguous float64 CUDA tensor [rot_dim / 2]")
        rot, fp = 2 * freq.shape[0], freq.data_ptr()
    return (T, Hq, 0 if k is None else k.shape[1], D, _weights(q_weight, "q_weight", D),
            _weights(k_weight, "k_weight", D), NORM[norm],
            None if positions is None else _int(positions, "positions", (T,)), fp, rot, PAIRS[pairs])


def _like(t, out, name):
    """A new tensor of t's shape, or `out`, checked: its pointer and token stride too."""
    if out is None:
        shape = t.shape
        out = torch.empty(shape, dtype=t.dtype, device=t.device)
        return out, out.data_ptr(), shape[1] * shape[2]
    if out.shape != t.shape or out.dtype is not t.dtype:
        raise ValueError(f"{name} must have its input's shape and dtype")
    return (out, *_rows(out, name))


def qk_norm_rope(q, k=None, *, norm="rms", q_weight=None, k_weight=None, eps: float = 1e-6, positions=None,
                 freq=None, pairs="half", q_out=None, k_out=None):
    """Norms of queries and keys for each head and the rotation by position, in one pass.  q [T,Hq,D]
    and k [T,Hk,D] (or None) fp32 or bf16, tokens may be strided; norm "rms" (mean square), "l2" (unit
    length) or "none"; q_weight, k_weight [D] fp32 or None; positions [T] int32 (negative: not a token,
    its rows of q_out and k_out are left as they were, and hold anything where these are allocated here);
    freq [rot_dim / 2] fp64, radians a position (None: no rotation); pairs "half" (i, i + rot_dim / 2) or
    "adjacent" (2 i, 2 i + 1).  q_out, k_out may be q and k.  Returns (q_out, k_out)."""
    lib = _lib or load()
    qp, qst = _rows(q, "q")
    kp, kst = (None, 0) if k is None else _rows(k, "k")
    T, Hq, Hk, D, qw, kw, kind, pos, fp, rot, pr = _norm_how(q, k, norm, q_weight, k_weight, positions, freq, pairs)
    q_out, qo, qos = _like(q, q_out, "q_out")
    ko, kos = None, 0
    if k is not None:
        k_out, ko, kos = _like(k, k_out, "k_out")
    here = _all_here(q, k, q_weight, k_weight, positions, freq, q_out, k_out if k is not None else None)
    code = lib.gdr_qk_norm_rope(qp, qst, kp, kst, qw, kw, eps, kind, pos, fp, rot, pr, qo, qos, ko, kos, T, Hq,
                                Hk, D, DTYPE[q.dtype], _raw_stream(here))
    if code:
        raise GdrError(code, "gdr_qk_norm_rope")
    return q_out, (None if k is None else k_out)


def qk_norm_rope_bwd_workspace_size(D) -> int:
    """Bytes of workspace qk_norm_rope_bwd needs on the current device where weights have gradients."""
    return int(load().gdr_qk_norm_rope_bwd_workspace_size(int(D)))


def qk_norm_rope_bwd(q, k, d_q_out, d_k_out, *, norm="rms", q_weight=None, k_weight=None, eps: float = 1e-6,
                     positions=None, freq=None, pairs="half", d_q=None, d_k=None, workspace=None):
    """Gradients through qk_norm_rope (the same arguments) given those of its outputs.  d_q, d_k may be
    d_q_out and d_k_out (or q and k) themselves.  workspace: None (allocated here) or a uint8 CUDA tensor
    of qk_norm_rope_bwd_workspace_size bytes.  Returns (d_q, d_k, d_q_weight, d_k_weight), the weights'
    [D] fp32, None for weights that are None."""
    lib = _lib or load()
    qp, qst = _rows(q, "q")
    kp, kst = (None, 0) if k is None else _rows(k, "k")
    T, Hq, Hk, D, qw, kw, kind, pos, fp, rot, pr = _norm_how(q, k, norm, q_weight, k_weight, positions, freq, pairs)
    if d_q_out.shape != q.shape or d_q_out.dtype is not q.dtype:
        raise ValueError("d_q_out must have q's shape and dtype")
    gp, gst = _rows(d_q_out, "d_q_out")
    d_q, dp, dst = _like(q, d_q, "d_q")
    hp, hst, ep, est = None, 0, None, 0
    if k is not None:
        if d_k_out.shape != k.shape or d_k_out.dtype is not k.dtype:
            raise ValueError("d_k_out must have k's shape and dtype")
        hp, hst = _rows(d_k_out, "d_k_out")
        d_k, ep, est = _like(k, d_k, "d_k")
    new = lambda w: None if w is None else torch.empty((D,), dtype=torch.float32, device=q.device)  # noqa: E731
    dqw, dkw = new(q_weight), new(k_weight if k is not None else None)
    wp, wn = None, 0
    if dqw is not None or dkw is not None:
        wn = lib.gdr_qk_norm_rope_bwd_workspace_size(D)
        if workspace is None:
            workspace = torch.empty(max(wn, 16), dtype=torch.uint8, device=q.device)
        else:
            _scratch(workspace, wn)
        wp = workspace.data_ptr()
    here = _all_here(q, k, q_weight, k_weight, positions, freq, d_q_out, d_k_out if k is not None else None, d_q,
                     d_k if k is not None else None, workspace if wp is not None else None)
    code = lib.gdr_qk_norm_rope_bwd(qp, qst, kp, kst, qw, kw, eps, kind, pos, fp, rot, pr, gp, gst, hp, hst, dp,
                                    dst, ep, est, None if dqw is None else dqw.data_ptr(),
                                    None if dkw is None else dkw.data_ptr(), T, Hq, Hk, D, DTYPE[q.dtype], wp, wn,
                                    _raw_stream(here))
    if code:
        raise GdrError(code, "gdr_qk_norm_rope_bwd")
    return d_q, (None if k is None else d_k), dqw, dkw
