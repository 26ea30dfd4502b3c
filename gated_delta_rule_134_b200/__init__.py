"""KDA (fine-grained gated delta rule) for B200: Python binding of libkda.so,
with the other layers of a hybrid stack beside it: the gated linear recurrence,
the query/key norm with the position rotation, and the attention of one new
token over a paged key-value cache.

Argument marshalling only: every step of the computation runs in the CUDA
kernels behind the C ABI declared in include/kda.h. PyTorch provides device
memory and the current CUDA stream. There is no CPU fallback: if the library
cannot be loaded, every call raises.
"""
from __future__ import annotations

import ctypes
import functools
import os

__all__ = ["load", "chunk_fwd", "chunk_fwd_varlen", "chunk_bwd", "chunk_fwd_noalloc", "noalloc_status", "decode_step",
           "workspace_size", "workspace_status", "chunk_fwd_timeout_test", "KDAError", "library_path", "STATUS",
           "recurrence_fwd", "recurrence_bwd", "recurrence_step", "recurrence_status", "recurrence_timeout_test", "qk_norm_rope", "qk_norm_rope_bwd", "attn_decode",
           "attn_decode_workspace_size"]

_PKG = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_PKG, "libkda.so")

STATUS = {0: "KDA_OK", 1: "KDA_ERR_INVALID_ARG", 2: "KDA_ERR_UNSUPPORTED", 3: "KDA_ERR_CUDA",
          4: "KDA_ERR_TIMEOUT"}
_DTYPE = {"f32": 0, "bf16": 1}
_ALGO = {"auto": 0, "simt": 1, "tc": 2, "tc_scan": 3}
# Variant switches (include/kda.h): gate "channel" = log_alpha [.., dk], "scalar" =
# one per token and head, "none" = no decay (log_alpha may be None).
GATES = {"channel": 0, "scalar": 1, "none": 2}
NORMS = {"l2": 0, "rms": 1}


class KDAError(RuntimeError):
    def __init__(self, fn: str, code: int, msg: str):
        super().__init__(f"{fn} -> {STATUS.get(code, code)}: {msg}")
        self.code = code


_lib = None


def library_path() -> str:
    return _LIB_PATH


def load(build_if_stale: bool = True):
    """Load libkda.so (building it in-tree with nvcc if it is missing or older
    than its sources). Raises if it cannot be built or loaded."""
    global _lib
    if _lib is not None:
        return _lib
    if build_if_stale:
        from . import build as _build
        if not _build.up_to_date():
            _build.build()
    if not os.path.exists(_LIB_PATH):
        raise RuntimeError(f"libkda.so not found at {_LIB_PATH}; run python -m gated_delta_rule_134_b200.build")
    lib = ctypes.CDLL(_LIB_PATH)
    P, I, Z = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
    lib.kda_status_string.argtypes = [I]
    lib.kda_status_string.restype = ctypes.c_char_p
    lib.kda_chunk_fwd_workspace_size.argtypes = [I] * 8
    lib.kda_chunk_fwd_workspace_size.restype = Z
    lib.kda_chunk_fwd.argtypes = [P] * 8 + [I] * 7 + [P, Z, P]
    lib.kda_chunk_fwd.restype = I
    lib.kda_chunk_fwd_ex.argtypes = [P] * 8 + [I] * 7 + [P, Z, I, P]
    lib.kda_chunk_fwd_ex.restype = I
    lib.kda_workspace_status.argtypes = [P, Z, P]
    lib.kda_chunk_fwd_timeout_test.argtypes = [P] * 8 + [I] * 7 + [P, Z, ctypes.c_longlong, P]
    lib.kda_chunk_fwd_timeout_test.restype = I
    lib.kda_workspace_status.restype = I
    lib.kda_decode_step.argtypes = [P] * 8 + [I] * 5 + [P]
    lib.kda_decode_step.restype = I
    lib.kda_chunk_fwd_noalloc.argtypes = [P] * 8 + [I] * 7 + [P]
    lib.kda_chunk_fwd_noalloc.restype = I
    lib.kda_noalloc_status.argtypes = [P]
    lib.kda_noalloc_status.restype = I
    lib.kda_chunk_fwd_v.argtypes = [P] * 8 + [I] * 9 + [P, Z, I, P]
    lib.kda_chunk_fwd_v.restype = I
    lib.kda_decode_step_v.argtypes = [P] * 8 + [I] * 7 + [P]
    lib.kda_decode_step_v.restype = I
    lib.kda_chunk_fwd_varlen.argtypes = [P] * 9 + [I] * 9 + [P, Z, I, P]
    lib.kda_chunk_fwd_varlen.restype = I
    lib.kda_chunk_bwd_workspace_size.argtypes = [I] * 5
    lib.kda_chunk_bwd_workspace_size.restype = Z
    lib.kda_chunk_bwd.argtypes = [P] * 14 + [I] * 8 + [P, Z, P]
    lib.kda_chunk_bwd.restype = I
    lib.kda_chunk_bwd_ex.argtypes = [P] * 14 + [I] * 9 + [P, Z, P]
    lib.kda_chunk_bwd_ex.restype = I
    lib.kda_chunk_bwd_workspace_size_ex.argtypes = [I] * 6
    lib.kda_chunk_bwd_workspace_size_ex.restype = Z
    F, L = ctypes.c_float, ctypes.c_longlong
    lib.kda_recurrence_fwd.argtypes = [P] * 6 + [I] * 4 + [P]
    lib.kda_recurrence_fwd.restype = I
    lib.kda_recurrence_bwd.argtypes = [P] * 9 + [I] * 4 + [P]
    lib.kda_recurrence_bwd.restype = I
    lib.kda_recurrence_status.argtypes = [P]
    lib.kda_recurrence_status.restype = I
    lib.kda_recurrence_timeout_test.argtypes = [P] * 3 + [I] * 4 + [L, P]
    lib.kda_recurrence_timeout_test.restype = I
    lib.kda_recurrence_step.argtypes = [P] * 5 + [I] * 3 + [P]
    lib.kda_recurrence_step.restype = I
    lib.kda_qk_norm_rope.argtypes = [P] * 7 + [I] + [P] * 2 + [I] * 6 + [L] * 4 + [I, F, F, I, I, P]
    lib.kda_qk_norm_rope.restype = I
    lib.kda_qk_norm_rope_bwd_workspace_size.argtypes = [I] * 4
    lib.kda_qk_norm_rope_bwd_workspace_size.restype = Z
    lib.kda_qk_norm_rope_bwd.argtypes = [P] * 9 + [I] + [P] * 4 + [I] * 6 + [L] * 4 + [I, F, F, I, I, P, Z, P]
    lib.kda_qk_norm_rope_bwd.restype = I
    lib.kda_attn_decode_workspace_size.argtypes = [I] * 4
    lib.kda_attn_decode_workspace_size.restype = Z
    lib.kda_attn_decode.argtypes = [P] * 9 + [I] * 8 + [F, I, P, Z, P]
    lib.kda_attn_decode.restype = I
    _lib = lib
    return lib


def _check(fn: str, code: int):
    if code != 0:
        raise KDAError(fn, code, load().kda_status_string(code).decode())


def _ptr(t):
    return None if t is None else t.data_ptr()


def _dtype_of(t) -> str:
    import torch
    dt = t.dtype
    if dt == torch.bfloat16:
        return "bf16"
    if dt == torch.float32:
        return "f32"
    raise TypeError(f"unsupported dtype {t.dtype}; use float32 or bfloat16")


def _stream(stream, device=None):
    """The stream handle to pass: the given torch stream, else the current
    stream of `device` (the tensors' device), else of the current device."""
    import torch
    if stream is None:
        # the handle alone where torch offers it: building a Stream object costs 2 us a call
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        if raw is not None and device is not None and device.index is not None:
            return raw(device.index)
        stream = torch.cuda.current_stream(device)
    return stream.cuda_stream


class _Here:
    """Stands for torch.cuda.device where the device is the current one already."""

    def __enter__(self):
        return None

    def __exit__(self, *exc):
        return False


_HERE = _Here()


def _on(device):
    """Make the tensors' device current for the call: the library launches on
    the current device (and the allocation-free entry point looks up its
    scratch array there), so it must be the device the pointers live on."""
    import torch
    if device is not None and device.index is not None and device.index == torch.cuda.current_device():
        return _HERE
    return torch.cuda.device(device)


def _need(t, name, shape, dtype, device):
    # get_device() is the index of a CUDA tensor's device, -1 for others; device.index is None for the CPU
    if t.dtype == dtype and t.shape == shape and t.is_contiguous() and t.get_device() == device.index:
        return
    if not t.is_cuda:
        raise ValueError(f"{name}: must be a CUDA tensor (this library has no CPU path)")
    if t.device != device or t.dtype != dtype or tuple(t.shape) != tuple(shape) or not t.is_contiguous():
        raise ValueError(f"{name}: expected contiguous {dtype} {tuple(shape)} on {device}, "
                         f"got {t.dtype} {tuple(t.shape)} on {t.device}")


def workspace_size(B, T, H, dk, dv, chunk=64, dtype="bf16", algo="auto") -> int:
    return int(load().kda_chunk_fwd_workspace_size(B, T, H, dk, dv, chunk, _DTYPE[dtype], _ALGO[algo]))


def _gate_shape(gate, lead, dk):
    if gate not in GATES:
        raise ValueError(f"gate must be one of {sorted(GATES)}")
    return None if gate == "none" else (tuple(lead) + (dk,) if gate == "channel" else tuple(lead))


def chunk_fwd(q, k, v, log_alpha, beta, S0=None, *, chunk: int = 64, algo: str = "auto",
              output_final_state: bool = True, o=None, S_T=None, workspace=None, stream=None,
              erase: bool = True, gate: str = "channel"):
    """kda_chunk_fwd(q, k, v, log_alpha, beta, S0 -> o, S_T) on CUDA tensors.

    q, k: [B,T,H,dk]; v: [B,T,H,dv]; beta: [B,T,H]; log_alpha: [B,T,H,dk]
    (gate "channel"), [B,T,H] (gate "scalar") or None (gate "none"), all
    float32 or all bfloat16; S0: [B,H,dk,dv] float32 or None. erase=False
    selects the additive-write variants (kda_chunk_fwd_v). Returns (o, S_T)
    with S_T None when output_final_state is False."""
    import torch
    lib = load()
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    dt, dev = q.dtype, q.device
    _need(q, "q", (B, T, H, dk), dt, dev)
    _need(k, "k", (B, T, H, dk), dt, dev)
    gshape = _gate_shape(gate, (B, T, H), dk)
    if gshape is not None:
        _need(log_alpha, "log_alpha", gshape, dt, dev)
    _need(v, "v", (B, T, H, dv), dt, dev)
    _need(beta, "beta", (B, T, H), dt, dev)
    if S0 is not None:
        _need(S0, "S0", (B, H, dk, dv), torch.float32, dev)
    if o is None:
        o = torch.empty(B, T, H, dv, dtype=dt, device=dev)
    _need(o, "o", (B, T, H, dv), dt, dev)
    if output_final_state and S_T is None:
        S_T = torch.empty(B, H, dk, dv, dtype=torch.float32, device=dev)
    if S_T is not None:
        _need(S_T, "S_T", (B, H, dk, dv), torch.float32, dev)
    dts = _dtype_of(q)
    ws_bytes = workspace_size(B, T, H, dk, dv, chunk, dts, algo)
    if ws_bytes and workspace is None:
        workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=dev)
    ws_len = 0 if workspace is None else workspace.numel() * workspace.element_size()
    la = log_alpha if gshape is not None else None
    with _on(dev):
        code = lib.kda_chunk_fwd_v(_ptr(q), _ptr(k), _ptr(v), _ptr(la), _ptr(beta), _ptr(S0), _ptr(o),
                                   _ptr(S_T), B, T, H, dk, dv, chunk, _DTYPE[dts], int(bool(erase)), GATES[gate],
                                   _ptr(workspace), ws_len, _ALGO[algo], _stream(stream, dev))
    _check("kda_chunk_fwd_v", code)
    return o, S_T


def chunk_fwd_varlen(q, k, v, log_alpha, beta, cu_seqlens, S0=None, *, chunk: int = 64, algo: str = "auto",
                     output_final_state: bool = True, o=None, S_T=None, workspace=None, stream=None,
                     erase: bool = True, gate: str = "channel"):
    """kda_chunk_fwd_varlen: N packed sequences. q, k [total_T,H,dk]; v
    [total_T,H,dv]; beta [total_T,H]; log_alpha [total_T,H,dk] / [total_T,H] /
    None by gate; cu_seqlens int32 CUDA tensor [N+1]; S0 [N,H,dk,dv] float32
    or None. Returns (o [total_T,H,dv], S_T [N,H,dk,dv] or None)."""
    import torch
    lib = load()
    TT, H, dk = q.shape
    dv = v.shape[-1]
    N = cu_seqlens.numel() - 1
    dt, dev = q.dtype, q.device
    _need(q, "q", (TT, H, dk), dt, dev)
    _need(k, "k", (TT, H, dk), dt, dev)
    gshape = _gate_shape(gate, (TT, H), dk)
    if gshape is not None:
        _need(log_alpha, "log_alpha", gshape, dt, dev)
    _need(v, "v", (TT, H, dv), dt, dev)
    _need(beta, "beta", (TT, H), dt, dev)
    _need(cu_seqlens, "cu_seqlens", (N + 1,), torch.int32, dev)
    if S0 is not None:
        _need(S0, "S0", (N, H, dk, dv), torch.float32, dev)
    if o is None:
        o = torch.empty(TT, H, dv, dtype=dt, device=dev)
    _need(o, "o", (TT, H, dv), dt, dev)
    if output_final_state and S_T is None:
        S_T = torch.empty(N, H, dk, dv, dtype=torch.float32, device=dev)
    if S_T is not None:
        _need(S_T, "S_T", (N, H, dk, dv), torch.float32, dev)
    dts = _dtype_of(q)
    # packed batches never take the segment scan: size the workspace for one pass
    ws_bytes = workspace_size(N, TT, H, dk, dv, chunk, dts, "tc" if algo == "auto" and dts == "bf16" and
                              dk == dv == 128 and chunk == 64 else algo)
    if ws_bytes and workspace is None:
        workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=dev)
    ws_len = 0 if workspace is None else workspace.numel() * workspace.element_size()
    la = log_alpha if gshape is not None else None
    with _on(dev):
        code = lib.kda_chunk_fwd_varlen(_ptr(q), _ptr(k), _ptr(v), _ptr(la), _ptr(beta), _ptr(S0), _ptr(o),
                                        _ptr(S_T), _ptr(cu_seqlens), N, TT, H, dk, dv, chunk, _DTYPE[dts],
                                        int(bool(erase)), GATES[gate], _ptr(workspace), ws_len, _ALGO[algo],
                                        _stream(stream, dev))
    _check("kda_chunk_fwd_varlen", code)
    return o, S_T


BWD_MODES = {"auto": 0, "all": 1, "low": 2}


def chunk_bwd(q, k, v, log_alpha, beta, S0, dO, dS_T=None, *, erase: bool = True, gate: str = "channel",
              want_dS0: bool = True, workspace=None, stream=None, memory: str = "auto") -> dict:
    """kda_chunk_bwd_ex: gradients of a loss with dL/do = dO [B,T,H,dv] and
    dL/dS_T = dS_T [B,H,dk,dv] (None: 0). Inputs as for chunk_fwd. memory:
    "auto", "all" (keep every chunk's state) or "low" (one per 64 tokens and a
    recompute sweep). Returns dict dq, dk, dv, dlog_alpha (None without a
    gate), dbeta, dS0 (None unless want_dS0)."""
    import torch
    lib = load()
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    dt, dev = q.dtype, q.device
    _need(q, "q", (B, T, H, dk), dt, dev)
    _need(k, "k", (B, T, H, dk), dt, dev)
    gshape = _gate_shape(gate, (B, T, H), dk)
    if gshape is not None:
        _need(log_alpha, "log_alpha", gshape, dt, dev)
    _need(v, "v", (B, T, H, dv), dt, dev)
    _need(beta, "beta", (B, T, H), dt, dev)
    _need(dO, "dO", (B, T, H, dv), dt, dev)
    if S0 is not None:
        _need(S0, "S0", (B, H, dk, dv), torch.float32, dev)
    if dS_T is not None:
        _need(dS_T, "dS_T", (B, H, dk, dv), torch.float32, dev)
    g = {"dq": torch.empty_like(q), "dk": torch.empty_like(k), "dv": torch.empty_like(v),
         "dlog_alpha": None if gshape is None else torch.empty(gshape, dtype=dt, device=dev),
         "dbeta": torch.empty_like(beta),
         "dS0": torch.empty(B, H, dk, dv, dtype=torch.float32, device=dev) if want_dS0 else None}
    mode = BWD_MODES[memory]
    ws_bytes = int(lib.kda_chunk_bwd_workspace_size_ex(B, T, H, dk, dv, mode))
    if ws_bytes and workspace is None:
        workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=dev)
    ws_len = 0 if workspace is None else workspace.numel() * workspace.element_size()
    la = log_alpha if gshape is not None else None
    with _on(dev):
        code = lib.kda_chunk_bwd_ex(_ptr(q), _ptr(k), _ptr(v), _ptr(la), _ptr(beta), _ptr(S0), _ptr(dO),
                                    _ptr(dS_T), _ptr(g["dq"]), _ptr(g["dk"]), _ptr(g["dv"]), _ptr(g["dlog_alpha"]),
                                    _ptr(g["dbeta"]), _ptr(g["dS0"]), B, T, H, dk, dv, _DTYPE[_dtype_of(q)],
                                    int(bool(erase)), GATES[gate], mode, _ptr(workspace), ws_len,
                                    _stream(stream, dev))
    _check("kda_chunk_bwd_ex", code)
    return g


def workspace_status(workspace, stream=None) -> int:
    """Synchronise and return the device-side status word of a workspace."""
    ws_len = 0 if workspace is None else workspace.numel() * workspace.element_size()
    dev = None if workspace is None else workspace.device
    with _on(dev):
        return int(load().kda_workspace_status(_ptr(workspace), ws_len, _stream(stream, dev)))


def decode_step(q, k, v, log_alpha, beta, S, *, S_out=None, o=None, stream=None, erase: bool = True,
                gate: str = "channel"):
    """kda_decode_step(q, k, v, log_alpha, beta, S -> o, S'): one token per
    sequence. q, k [N,H,dk]; log_alpha [N,H,dk] / [N,H] / None by gate; v
    [N,H,dv]; beta [N,H]; S [N,H,dk,dv] float32. S_out defaults to S
    (in-place update). Returns (o, S_out)."""
    import torch
    lib = load()
    N, H, dk = q.shape
    dv = v.shape[-1]
    dt, dev = q.dtype, q.device
    _need(q, "q", (N, H, dk), dt, dev)
    _need(k, "k", (N, H, dk), dt, dev)
    gshape = _gate_shape(gate, (N, H), dk)
    if gshape is not None:
        _need(log_alpha, "log_alpha", gshape, dt, dev)
    _need(v, "v", (N, H, dv), dt, dev)
    _need(beta, "beta", (N, H), dt, dev)
    _need(S, "S", (N, H, dk, dv), torch.float32, dev)
    if S_out is None:
        S_out = S
    _need(S_out, "S_out", (N, H, dk, dv), torch.float32, dev)
    if o is None:
        o = torch.empty(N, H, dv, dtype=dt, device=dev)
    _need(o, "o", (N, H, dv), dt, dev)
    la = log_alpha if gshape is not None else None
    with _on(dev):
        code = lib.kda_decode_step_v(_ptr(q), _ptr(k), _ptr(v), _ptr(la), _ptr(beta), _ptr(S), _ptr(S_out),
                                     _ptr(o), N, H, dk, dv, _DTYPE[_dtype_of(q)], int(bool(erase)), GATES[gate],
                                     _stream(stream, dev))
    _check("kda_decode_step_v", code)
    return o, S_out


def chunk_fwd_noalloc(q, k, v, log_alpha, beta, S0=None, *, o, S_T=None, chunk: int = 64, stream=None):
    """kda_chunk_fwd_noalloc: the tensor-core prefill without a workspace.

    For callers that must not allocate device memory where they run the
    prefill: the library keeps the kernel's small scratch in a fixed array of
    its own, so only inputs and caller-owned outputs (o, and S_T if wanted)
    are passed. bf16 inputs, dk = dv = 128, chunk = 64. Calls that overlap on
    the GPU share that array and race; noalloc_status reads its status word.
    Returns (o, S_T)."""
    import torch
    lib = load()
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    dt, dev = q.dtype, q.device
    _need(q, "q", (B, T, H, dk), dt, dev)
    _need(k, "k", (B, T, H, dk), dt, dev)
    _need(log_alpha, "log_alpha", (B, T, H, dk), dt, dev)
    _need(v, "v", (B, T, H, dv), dt, dev)
    _need(beta, "beta", (B, T, H), dt, dev)
    _need(o, "o", (B, T, H, dv), dt, dev)
    if S0 is not None:
        _need(S0, "S0", (B, H, dk, dv), torch.float32, dev)
    if S_T is not None:
        _need(S_T, "S_T", (B, H, dk, dv), torch.float32, dev)
    with _on(dev):
        code = lib.kda_chunk_fwd_noalloc(_ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(beta), _ptr(S0),
                                         _ptr(o), _ptr(S_T), B, T, H, dk, dv, chunk, _DTYPE[_dtype_of(q)],
                                         _stream(stream, dev))
    _check("kda_chunk_fwd_noalloc", code)
    return o, S_T


def chunk_fwd_timeout_test(q, k, v, log_alpha, beta, S0=None, *, o, S_T, workspace, wait_budget_cycles: int,
                           stream=None):
    """kda_chunk_fwd_timeout_test: the tensor-core prefill with its first k/q
    load withheld and every wait bounded by wait_budget_cycles SM cycles, so
    the kernel gives up and records KDA_ERR_TIMEOUT in `workspace` (read it
    with workspace_status). A test hook for the timeout path; o and S_T are
    left undefined."""
    import torch
    lib = load()
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    dt, dev = q.dtype, q.device
    _need(q, "q", (B, T, H, dk), dt, dev)
    _need(k, "k", (B, T, H, dk), dt, dev)
    _need(log_alpha, "log_alpha", (B, T, H, dk), dt, dev)
    _need(v, "v", (B, T, H, dv), dt, dev)
    _need(beta, "beta", (B, T, H), dt, dev)
    _need(o, "o", (B, T, H, dv), dt, dev)
    _need(S_T, "S_T", (B, H, dk, dv), torch.float32, dev)
    if S0 is not None:
        _need(S0, "S0", (B, H, dk, dv), torch.float32, dev)
    ws_len = workspace.numel() * workspace.element_size()
    with _on(dev):
        code = lib.kda_chunk_fwd_timeout_test(_ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(beta), _ptr(S0),
                                              _ptr(o), _ptr(S_T), B, T, H, dk, dv, 64, _DTYPE[_dtype_of(q)],
                                              _ptr(workspace), ws_len, int(wait_budget_cycles),
                                              _stream(stream, dev))
    _check("kda_chunk_fwd_timeout_test", code)
    return o, S_T


def noalloc_status(device=None, stream=None) -> int:
    """kda_noalloc_status: synchronise and return the status word the last
    chunk_fwd_noalloc on `device` left in the library's own scratch array
    (0 = KDA_OK, 4 = KDA_ERR_TIMEOUT). Allocates nothing."""
    import torch
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    with _on(dev):
        return int(load().kda_noalloc_status(_stream(stream, dev)))


# ---------------------------------------------------------------- what the stack's other layers share


def _memory_of(stream):
    """Outputs and workspaces that a call allocates belong to the stream its
    kernels run on: from another stream's pool they could be memory that this
    one's pending work still uses, and a workspace would go back there while
    the kernels run."""
    if stream is None:
        return _HERE
    import torch
    return torch.cuda.stream(stream)


def _scratch_bytes(workspace, device) -> int:
    """Size of a workspace that the caller gave (or None): the kernels write all of it, so its elements have to be memory
    of its own, on the tensors' device."""
    if workspace is None:
        return 0
    if workspace.device != device or not workspace.is_contiguous():
        raise ValueError(f"workspace: expected a contiguous tensor on {device}, got strides {tuple(workspace.stride())} of "
                         f"{tuple(workspace.shape)} on {workspace.device}")
    return workspace.numel() * workspace.element_size()


def _int32(**sizes):
    """The C calls take sizes as int: refused here, since ctypes would cut them."""
    for name, value in sizes.items():
        if not -0x80000000 <= value <= 0x7fffffff:
            raise ValueError(f"{name}: {value} is not in [-2^31, 2^31)")


# ---------------------------------------------------------------- gated linear recurrence


def _recurrence_sizes(log_alpha, cu_seqlens):
    """(N, T, D) of a dense [B,T,D] or a packed [T,D] batch."""
    import torch
    if cu_seqlens is None:
        if log_alpha.dim() != 3:
            raise ValueError(f"log_alpha: expected [B,T,D], got {tuple(log_alpha.shape)}")
        N, T, D = log_alpha.shape
        _int32(B=N, T=T, D=D)
        return N, T, D
    if log_alpha.dim() != 2:
        raise ValueError(f"log_alpha: expected packed [total_T,D], got {tuple(log_alpha.shape)}")
    N = cu_seqlens.numel() - 1
    if N < 0:
        raise ValueError("cu_seqlens: expected N + 1 offsets")
    T, D = log_alpha.shape
    _int32(N=N, total_T=T, D=D)
    _need(cu_seqlens, "cu_seqlens", (N + 1,), torch.int32, log_alpha.device)
    return N, T, D


def recurrence_fwd(log_alpha, x, h0=None, *, cu_seqlens=None, output_final_state: bool = True, h=None, h_T=None,
                   stream=None):
    """kda_recurrence_fwd: h_t = exp(log_alpha_t) h_{t-1} + x_t per channel.

    log_alpha, x: [B,T,D], or packed [total_T,D] with cu_seqlens int32 [N+1];
    both float32 or both bfloat16. h0: [B or N,D] float32 or None (zero).
    Returns (h, h_T): h like x, h_T [B or N,D] float32 (None when
    output_final_state is False). h may be x, h_T may be h0. Tokens outside
    every packed sequence are not written: an h made here holds anything
    there."""
    import torch
    lib = load()
    N, T, D = _recurrence_sizes(log_alpha, cu_seqlens)
    dt, dev, shape = log_alpha.dtype, log_alpha.device, log_alpha.shape
    dts = _dtype_of(log_alpha)
    _need(log_alpha, "log_alpha", shape, dt, dev)
    _need(x, "x", shape, dt, dev)
    if h0 is not None:
        _need(h0, "h0", (N, D), torch.float32, dev)
    if h is not None:
        _need(h, "h", shape, dt, dev)
    if h_T is not None:
        _need(h_T, "h_T", (N, D), torch.float32, dev)
    with _memory_of(stream):
        if h is None:
            h = torch.empty_like(x)
        if h_T is None and output_final_state:
            h_T = torch.empty(N, D, dtype=torch.float32, device=dev)
    with _on(dev):
        code = lib.kda_recurrence_fwd(_ptr(log_alpha), _ptr(x), _ptr(h0), _ptr(h), _ptr(h_T), _ptr(cu_seqlens),
                                      N, T, D, _DTYPE[dts], _stream(stream, dev))
    _check("kda_recurrence_fwd", code)
    return h, h_T


def recurrence_bwd(log_alpha, h, h0, dh, dh_T=None, *, cu_seqlens=None, want_dh0: bool = True, dx=None, dlog_alpha=None,
                   stream=None) -> dict:
    """kda_recurrence_bwd: gradients of a loss with dL/dh = dh and dL/dh_T =
    dh_T ([B or N,D] float32 or None). log_alpha, h0, cu_seqlens as for
    recurrence_fwd, h its output. Returns dict dx, dlog_alpha, dh0 (None
    unless want_dh0). dx may be dh. Tokens outside every packed sequence are
    not written: for a batch with such tokens give a dx and dlog_alpha that
    hold zeros there."""
    import torch
    lib = load()
    N, T, D = _recurrence_sizes(log_alpha, cu_seqlens)
    dt, dev, shape = log_alpha.dtype, log_alpha.device, log_alpha.shape
    dts = _dtype_of(log_alpha)
    _need(log_alpha, "log_alpha", shape, dt, dev)
    _need(h, "h", shape, dt, dev)
    _need(dh, "dh", shape, dt, dev)
    if h0 is not None:
        _need(h0, "h0", (N, D), torch.float32, dev)
    if dh_T is not None:
        _need(dh_T, "dh_T", (N, D), torch.float32, dev)
    if dx is not None:
        _need(dx, "dx", shape, dt, dev)
    if dlog_alpha is not None:
        _need(dlog_alpha, "dlog_alpha", shape, dt, dev)
    with _memory_of(stream):
        g = {"dx": torch.empty_like(dh) if dx is None else dx,
             "dlog_alpha": torch.empty_like(log_alpha) if dlog_alpha is None else dlog_alpha,
             "dh0": torch.empty(N, D, dtype=torch.float32, device=dev) if want_dh0 else None}
    with _on(dev):
        code = lib.kda_recurrence_bwd(_ptr(log_alpha), _ptr(h), _ptr(h0), _ptr(dh), _ptr(dh_T), _ptr(g["dx"]),
                                      _ptr(g["dlog_alpha"]), _ptr(g["dh0"]), _ptr(cu_seqlens), N, T, D, _DTYPE[dts],
                                      _stream(stream, dev))
    _check("kda_recurrence_bwd", code)
    return g


def recurrence_step(log_alpha, x, h, *, h_out=None, y=None, stream=None):
    """kda_recurrence_step: one token per sequence. log_alpha, x: [N,D]; h
    [N,D] float32. h_out defaults to h (in-place update). Returns (y, h_out)
    with y = h_out in the inputs' dtype."""
    import torch
    lib = load()
    if log_alpha.dim() != 2:
        raise ValueError(f"log_alpha: expected [N,D], got {tuple(log_alpha.shape)}")
    N, D = log_alpha.shape
    _int32(N=N, D=D)
    dt, dev = log_alpha.dtype, log_alpha.device
    dts = _dtype_of(log_alpha)
    _need(log_alpha, "log_alpha", (N, D), dt, dev)
    _need(x, "x", (N, D), dt, dev)
    _need(h, "h", (N, D), torch.float32, dev)
    if h_out is None:
        h_out = h
    else:
        _need(h_out, "h_out", (N, D), torch.float32, dev)
    if y is None:
        with _memory_of(stream):
            y = torch.empty_like(x)
    else:
        _need(y, "y", (N, D), dt, dev)
    with _on(dev):
        code = lib.kda_recurrence_step(_ptr(log_alpha), _ptr(x), _ptr(h), _ptr(h_out), _ptr(y), N, D, _DTYPE[dts],
                                       _stream(stream, dev))
    _check("kda_recurrence_step", code)
    return y, h_out


def recurrence_status(device=None, stream=None) -> int:
    """kda_recurrence_status: synchronise and return whether a wait inside a
    recurrence_fwd or recurrence_bwd on `device` gave up since this was last
    asked (0 = KDA_OK, 4 = KDA_ERR_TIMEOUT: those outputs are invalid)."""
    import torch
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    with _on(dev):
        return int(load().kda_recurrence_status(_stream(stream, dev)))


def recurrence_timeout_test(log_alpha, x, *, h, wait_budget_cycles: int, stream=None):
    """kda_recurrence_timeout_test: recurrence_fwd with the first CTA of every
    cluster sending nothing and every wait bounded by wait_budget_cycles SM
    cycles, so that the waits give up (read recurrence_status). A test hook; h
    is left undefined."""
    lib = load()
    N, T, D = _recurrence_sizes(log_alpha, None)
    dt, dev = log_alpha.dtype, log_alpha.device
    for t, name in ((log_alpha, "log_alpha"), (x, "x"), (h, "h")):
        _need(t, name, (N, T, D), dt, dev)
    with _on(dev):
        code = lib.kda_recurrence_timeout_test(_ptr(log_alpha), _ptr(x), _ptr(h), N, T, D, _DTYPE[_dtype_of(x)],
                                               int(wait_budget_cycles), _stream(stream, dev))
    _check("kda_recurrence_timeout_test", code)


# ---------------------------------------------------------------- query/key norm and rotation


def _heads_view(t, name, lead, d, dt, dev):
    """t [*lead, H, d] as [n, H, d] without a copy: any head and token strides, channels contiguous."""
    if not t.is_cuda:
        raise ValueError(f"{name}: must be a CUDA tensor (this library has no CPU path)")
    if t.device != dev or t.dtype != dt or tuple(t.shape[:-2]) != tuple(lead) or t.shape[-1] != d:
        raise ValueError(f"{name}: expected {dt} {tuple(lead) + ('heads', d)} on {dev}, got {t.dtype} "
                         f"{tuple(t.shape)} on {t.device}")
    if t.numel() and t.stride(-1) != 1:
        raise ValueError(f"{name}: the channels of a head must be contiguous")
    if t.dim() == 3:
        return t
    n = 1
    for s in lead:
        n *= s
    try:
        return t.view(n, t.shape[-2], d)
    except RuntimeError:
        raise ValueError(f"{name}: the leading dimensions {tuple(lead)} must have one common stride") from None


def _qk_args(q, k, q_weight, k_weight, cos, sin, positions, norm):
    """Checks what the two directions share. Returns the pointers of q, k, weights, tables and positions, pos_bytes, and
    the sizes and strides that follow the outputs in the C calls."""
    import torch
    if norm not in NORMS:
        raise ValueError(f"norm must be one of {sorted(NORMS)}")
    qs, ks = q.shape, k.shape
    if len(qs) < 3 or len(ks) != len(qs):
        raise ValueError(f"q, k: expected [..., tokens, heads, d], got {tuple(qs)} and {tuple(ks)}")
    dt, dev, d = q.dtype, q.device, qs[-1]
    sq, sk = q.stride(), k.stride()
    if not (len(qs) == 3 and q.is_cuda and sq[2] == sk[2] == 1 and ks[0] == qs[0] and ks[2] == d and k.dtype == dt
            and k.device == dev):
        q, k = _heads_view(q, "q", qs[:-2], d, dt, dev), _heads_view(k, "k", qs[:-2], d, dt, dev)
        sq, sk = q.stride(), k.stride()
    n = q.shape[0]
    _int32(tokens=n)
    if q_weight is not None:
        _need(q_weight, "q_weight", (d,), dt, dev)
    if k_weight is not None:
        _need(k_weight, "k_weight", (d,), dt, dev)
    rot = max_pos = pos_bytes = 0
    if positions is not None:
        if cos is None or sin is None:
            raise ValueError("positions need the cos and sin tables")
        if cos.dim() != 2:
            raise ValueError(f"cos: expected [max_pos, rot/2], got {tuple(cos.shape)}")
        table = cos.shape
        max_pos, rot = table[0], 2 * table[1]
        _need(cos, "cos", table, torch.float32, dev)
        _need(sin, "sin", table, torch.float32, dev)
        pos_dt = positions.dtype
        if pos_dt != torch.int64 and pos_dt != torch.int32:
            raise TypeError(f"positions: expected int32 or int64, got {pos_dt}")
        pos_bytes = 8 if pos_dt == torch.int64 else 4
        if positions.numel() != n:
            raise ValueError(f"positions: expected one per token ({n}), got {tuple(positions.shape)}")
        _need(positions, "positions", positions.shape, pos_dt, dev)
    return ((q.data_ptr(), k.data_ptr(), _ptr(q_weight), _ptr(k_weight), _ptr(cos), _ptr(sin), _ptr(positions),
             pos_bytes),
            (n, q.shape[1], k.shape[1], d, rot, max_pos, sq[0], sq[1], sk[0], sk[1], NORMS[norm]))


def qk_norm_rope(q, k, q_weight=None, k_weight=None, cos=None, sin=None, positions=None, *, norm: str = "rms",
                 eps: float = 1e-6, q_scale: float = 1.0, interleaved: bool = False, q_out=None, k_out=None,
                 stream=None):
    """kda_qk_norm_rope: queries and keys normalised per head and rotated by
    position in one pass.

    q: [..., Hq, d], k: [..., Hk, d] with the same leading dimensions, both
    float32 or both bfloat16; slices of a fused projection are read in place
    (channels contiguous, other strides multiples of 16 bytes). q_weight,
    k_weight: [d] or None. positions: int32 or int64, one per token, or None
    (no rotation); cos, sin: [max_pos, rot/2] float32. norm: "l2" or "rms".
    Returns contiguous (q_out, k_out); q_out may be q where q is contiguous."""
    import torch
    lib = load()
    dts = _dtype_of(q)
    inputs, sizes = _qk_args(q, k, q_weight, k_weight, cos, sin, positions, norm)
    dt, dev = q.dtype, q.device
    if q_out is not None:
        _need(q_out, "q_out", q.shape, dt, dev)
    if k_out is not None:
        _need(k_out, "k_out", k.shape, dt, dev)
    with _memory_of(stream):
        if q_out is None:
            q_out = torch.empty(q.shape, dtype=dt, device=dev)
        if k_out is None:
            k_out = torch.empty(k.shape, dtype=dt, device=dev)
    with _on(dev):
        code = lib.kda_qk_norm_rope(*inputs, q_out.data_ptr(), k_out.data_ptr(), *sizes, eps, q_scale,
                                    1 if interleaved else 0, _DTYPE[dts], _stream(stream, dev))
    _check("kda_qk_norm_rope", code)
    return q_out, k_out


@functools.lru_cache(maxsize=256)
def _qk_workspace_size(n, Hq, Hk, d) -> int:
    return int(load().kda_qk_norm_rope_bwd_workspace_size(n, Hq, Hk, d))


def qk_norm_rope_bwd(dq_out, dk_out, q, k, q_weight=None, k_weight=None, cos=None, sin=None, positions=None, *,
                     norm: str = "rms", eps: float = 1e-6, q_scale: float = 1.0, interleaved: bool = False,
                     workspace=None, stream=None) -> dict:
    """kda_qk_norm_rope_bwd: gradients of a loss with dL/dq_out = dq_out and
    dL/dk_out = dk_out (contiguous, shaped like q and k); the other arguments
    as for qk_norm_rope. Returns dict dq, dk (contiguous), dq_weight,
    dk_weight (float32 [d]; None without a weight)."""
    import torch
    lib = load()
    dts = _dtype_of(q)
    inputs, sizes = _qk_args(q, k, q_weight, k_weight, cos, sin, positions, norm)
    dt, dev, d = q.dtype, q.device, q.shape[-1]
    _need(dq_out, "dq_out", q.shape, dt, dev)
    _need(dk_out, "dk_out", k.shape, dt, dev)
    ws_len = _scratch_bytes(workspace, dev)
    with _memory_of(stream):
        dq, dk = torch.empty(q.shape, dtype=dt, device=dev), torch.empty(k.shape, dtype=dt, device=dev)
        dqw = None if q_weight is None else torch.empty(d, dtype=torch.float32, device=dev)
        dkw = None if k_weight is None else torch.empty(d, dtype=torch.float32, device=dev)
        if workspace is None and (dqw is not None or dkw is not None):
            ws_len = _qk_workspace_size(*sizes[:4])
            workspace = torch.empty(ws_len, dtype=torch.uint8, device=dev)
    with _on(dev):
        code = lib.kda_qk_norm_rope_bwd(dq_out.data_ptr(), dk_out.data_ptr(), *inputs, dq.data_ptr(), dk.data_ptr(),
                                        _ptr(dqw), _ptr(dkw), *sizes, eps, q_scale, 1 if interleaved else 0,
                                        _DTYPE[dts], _ptr(workspace), ws_len, _stream(stream, dev))
    _check("kda_qk_norm_rope_bwd", code)
    return {"dq": dq, "dk": dk, "dq_weight": dqw, "dk_weight": dkw}


# ---------------------------------------------------------------- paged decode attention


@functools.lru_cache(maxsize=256)
def attn_decode_workspace_size(N, Hq, Hk, d) -> int:
    return int(load().kda_attn_decode_workspace_size(N, Hq, Hk, d))


def attn_decode(q, k_cache, v_cache, page_table, seq_lens, *, k=None, v=None, scale=None, window: int = 0, o=None,
                lse=None, return_lse: bool = False, workspace=None, stream=None):
    """kda_attn_decode: one new token per sequence over a paged key-value cache.

    q: [N,Hq,d]; k, v: [N,Hk,d], the new token's key and value, put into the
    cache at position seq_lens[n] (or both None); k_cache, v_cache:
    [n_pages,Hk,page_size,d], updated in place; page_table: int32
    [N,max_pages]; seq_lens: int32 [N], positions held before the call,
    negative for rows of a padded batch. scale defaults to d**-0.5; window > 0
    attends to the last `window` positions only. Returns o [N,Hq,d], or (o,
    lse) with lse [N,Hq] float32 when return_lse is set or lse is given."""
    import torch
    lib = load()
    if q.dim() != 3 or k_cache.dim() != 4 or page_table.dim() != 2:
        raise ValueError(f"expected q [N,Hq,d], k_cache [n_pages,Hk,page_size,d], page_table [N,max_pages], got "
                         f"{tuple(q.shape)}, {tuple(k_cache.shape)}, {tuple(page_table.shape)}")
    N, Hq, d = q.shape
    n_pages, Hk, page_size, _ = k_cache.shape
    max_pages = page_table.shape[1]
    window = int(window)
    _int32(N=N, Hq=Hq, n_pages=n_pages, Hk=Hk, page_size=page_size, max_pages=max_pages, window=window)
    dt, dev = q.dtype, q.device
    dts = _dtype_of(q)
    _need(q, "q", (N, Hq, d), dt, dev)
    _need(k_cache, "k_cache", (n_pages, Hk, page_size, d), dt, dev)
    _need(v_cache, "v_cache", (n_pages, Hk, page_size, d), dt, dev)
    _need(page_table, "page_table", (N, max_pages), torch.int32, dev)
    _need(seq_lens, "seq_lens", (N,), torch.int32, dev)
    if (k is None) != (v is None):
        raise ValueError("k and v: give both or neither")
    if k is not None:
        _need(k, "k", (N, Hk, d), dt, dev)
        _need(v, "v", (N, Hk, d), dt, dev)
    if o is not None:
        _need(o, "o", (N, Hq, d), dt, dev)
    if lse is not None:
        _need(lse, "lse", (N, Hq), torch.float32, dev)
        return_lse = True
    ws_len = _scratch_bytes(workspace, dev)
    with _memory_of(stream):
        if o is None:
            o = torch.empty_like(q)
        if lse is None and return_lse:
            lse = torch.empty(N, Hq, dtype=torch.float32, device=dev)
        if workspace is None:
            ws_len = attn_decode_workspace_size(N, Hq, Hk, d)
            workspace = torch.empty(ws_len, dtype=torch.uint8, device=dev) if ws_len else None
    with _on(dev):
        code = lib.kda_attn_decode(_ptr(q), _ptr(k), _ptr(v), _ptr(k_cache), _ptr(v_cache), _ptr(page_table),
                                   _ptr(seq_lens), _ptr(o), _ptr(lse), N, Hq, Hk, d, n_pages, page_size, max_pages,
                                   window, d ** -0.5 if scale is None else scale, _DTYPE[dts], _ptr(workspace),
                                   ws_len, _stream(stream, dev))
    _check("kda_attn_decode", code)
    return (o, lse) if return_lse else o
