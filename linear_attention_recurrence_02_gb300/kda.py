"""Thin ctypes binding of libkda.so (declared in include/kda.h).

Argument marshalling only: shapes and dtypes are read from the torch tensors
passed in, their device pointers and the current CUDA stream are handed to
the C ABI, and a non-OK status raises ``KdaError``. Every step of the
computation runs in the library's CUDA kernels; there is no fallback. If the
library has not been built, the first call raises.
"""
from __future__ import annotations

import ctypes
import os
import threading

from . import build as _build

KDA_OK, KDA_ERR_INVALID_ARG, KDA_ERR_UNSUPPORTED, KDA_ERR_CUDA, KDA_ERR_TIMEOUT, KDA_ERR_DEVICE_CHECK = range(6)
# gate forms: one log-gate per key channel (KDA), per head (Gated DeltaNet), none (DeltaNet)
KDA_GATE_CHANNEL, KDA_GATE_HEAD, KDA_GATE_NONE = range(3)
KDA_DECODE_OVERLAP_PREV = 1  # launch flag of kda_shortconv_decode_step_ex
KDA_ACT_SIGMOID, KDA_ACT_SILU = 0, 1  # output-gate activations of kda_gated_rmsnorm
_ACTS = {"sigmoid": KDA_ACT_SIGMOID, "silu": KDA_ACT_SILU}
_GATES = {"channel": KDA_GATE_CHANNEL, "head": KDA_GATE_HEAD, "none": KDA_GATE_NONE}


def _gate_code(gate):
    if isinstance(gate, str):
        return _GATES[gate]
    return int(gate)


def _check_gate(g, gate, lead, H, D):
    """Shape of g for a gate form: [..., H, D], [..., H], or absent."""
    code = _gate_code(gate)
    if code == KDA_GATE_CHANNEL:
        ok = g is not None and tuple(g.shape) == (*lead, H, D)
    elif code == KDA_GATE_HEAD:
        ok = g is not None and tuple(g.shape) == (*lead, H)
    else:
        ok = True
    if not ok:
        raise ValueError("g shape does not match the gate form")
    return code
KDA_F32, KDA_BF16 = 0, 1

_lib = None
_lock = threading.Lock()

_vp = ctypes.c_void_p
_ci = ctypes.c_int
_cf = ctypes.c_float
_i64 = ctypes.c_int64
_sz = ctypes.c_size_t

_SIGNATURES = {
    "kda_status_string": ([_ci], ctypes.c_char_p),
    "kda_last_error_detail": ([], ctypes.c_char_p),
    "kda_abi_version": ([], _ci),
    "kda_state_bytes": ([_ci, _ci, _ci, _ci], _sz),
    "kda_shortconv_ring_bytes": ([_ci, _ci, _ci, _ci, _ci], _sz),
    "kda_shortconv_step": ([_vp, _vp, _vp, _vp, _ci, _ci, _ci, _ci, _vp], _ci),
    "kda_shortconv_prefill": ([_vp, _vp, _vp, _vp, _vp, _vp, _ci, _i64, _ci, _ci, _ci, _vp], _ci),
    "kda_decode_step": ([_vp, _vp, _vp, _vp, _vp, _vp, _vp, _ci, _ci, _ci, _ci, _cf, _vp], _ci),
    "kda_decode_step_gated": ([_vp, _vp, _vp, _vp, _vp, _vp, _vp, _ci, _ci, _ci, _ci, _ci, _cf, _vp], _ci),
    "kda_shortconv_decode_step_gated": ([_vp, _vp, _vp, _vp, _vp, _vp, _vp, _ci, _ci, _ci, _ci, _ci, _cf, _vp],
                                        _ci),
    "kda_chunk_prefill_gated": ([_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _ci, _i64, _ci, _ci, _ci, _ci, _ci,
                                 _cf, _vp, _sz, _vp], _ci),
    "kda_shortconv_decode_step": ([_vp, _vp, _vp, _vp, _vp, _vp, _vp, _ci, _ci, _ci, _ci, _cf, _vp], _ci),
    "kda_shortconv_decode_step_ex": ([_vp, _vp, _vp, _vp, _vp, _vp, _vp, _ci, _ci, _ci, _ci, _ci, _cf,
                                      ctypes.c_uint, _vp], _ci),
    "kda_shortconv_decode_step_epi": ([_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _ci, _ci, _ci, _ci, _ci, _ci,
                                       _cf, _cf, ctypes.c_uint, _vp], _ci),
    "kda_chunk_prefill_workspace_bytes": ([_i64, _ci, _ci, _ci, _ci], _sz),
    "kda_chunk_prefill_route": ([_ci, _ci, _ci], ctypes.c_char_p),
    "kda_chunk_prefill": ([_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _ci, _i64, _ci, _ci, _ci, _ci,
                           _cf, _vp, _sz, _vp], _ci),
    "kda_chunk_prefill_noalloc": ([_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _ci, _i64, _ci, _ci, _ci,
                                   _ci, _cf, _vp], _ci),
    "kda_gated_rmsnorm": ([_vp, _vp, _vp, _vp, _i64, _ci, _ci, _ci, _ci, _cf, _vp], _ci),
    "kda_add_rmsnorm_fp8": ([_vp, _vp, _vp, _vp, _vp, _vp, _i64, _ci, _ci, _ci, _cf, _vp], _ci),
    "kda_gated_rmsnorm_fp8": ([_vp, _vp, _vp, _vp, _vp, _i64, _ci, _ci, _ci, _ci, _cf, _vp], _ci),
    "kda_fp8_linear": ([_vp, _vp, _vp, _vp, _vp, _i64, _ci, _ci, _i64, _i64, _i64, _ci, _vp], _ci),
    "kda_shortconv_decode_step_proj": ([_vp] * 11 + [_ci] * 7 + [_cf, _cf, ctypes.c_uint, _vp, _sz, _vp], _ci),
    "kda_shortconv_decode_step_proj_workspace_bytes": ([_ci, _ci, _ci], _sz),
    "kda_chunk_prefill_proj": ([_vp] * 8 + [_ci, _i64, _ci, _ci, _ci, _ci, _ci, _cf, _vp, _vp, _ci, _cf, _vp, _vp, _vp,
                                _ci, _vp, _sz, _vp], _ci),
    "kda_chunk_prefill_proj_workspace_bytes": ([_i64, _ci, _ci, _ci, _ci], _sz),
    "kda_chunk_prefill_scan_workspace_bytes": ([_i64, _ci, _ci, _ci, _ci], _sz),
    "kda_chunk_prefill_split": ([_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _ci, _i64, _ci, _ci, _ci, _ci,
                                 _ci, _cf, _vp, _sz, _vp], _ci),
    "kda_chunk_prefill_split_workspace_bytes": ([_vp, _ci, _ci, _ci, _ci], _sz),
    "kda_chunk_prefill_split_plan": ([_vp, _ci, _ci, _ci, _ci, _vp], _ci),
    "kda_chunk_prefill_epi": ([_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _ci, _i64, _ci, _ci, _ci, _ci, _ci,
                               _cf, _vp, _vp, _ci, _cf, _vp, _sz, _vp], _ci),
    "kda_chunk_prefill_scan": ([_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _ci, _ci, _ci, _ci, _ci, _cf, _ci,
                                _vp, _sz, _vp], _ci),
    "kda_qk_norm_rope": ([_vp] * 8 + [_i64, _ci, _ci, _ci, _ci, _i64, _i64, _i64, _i64, _ci, _cf, _ci, _vp], _ci),
    "kda_kv4_cache_bytes": ([_i64, _ci, _ci, _ci], _sz),
    "kda_kv4_append": ([_vp] * 6 + [_ci, _i64, _ci, _ci, _ci, _i64, _ci, _i64, _i64, _i64, _ci, _vp], _ci),
    "kda_kv4_read": ([_vp] * 6 + [_ci, _i64, _ci, _ci, _ci, _i64, _ci, _i64, _i64, _i64, _ci, _vp], _ci),
    "kda_kv4_attention": ([_vp] * 7 + [_ci, _i64, _ci, _ci, _ci, _ci, _i64, _ci, _i64, _i64, _i64, _cf, _ci, _i64, _ci,
                                       _vp, _sz, _vp], _ci),
    "kda_kv4_attention_workspace_bytes": ([_ci, _i64, _ci, _ci, _ci, _ci, _ci, _ci, _i64, _ci], _sz),
    "kda_sync_status": ([_vp], _ci),
    "kda_selftest_bounded_wait": ([ctypes.c_longlong, _vp], _ci),
}


class KdaError(RuntimeError):
    def __init__(self, status: int, detail: str):
        self.status = status
        super().__init__(f"{_status_string(status)} ({detail})")


def library_path() -> str:
    return _build.LIB


def lib():
    """The loaded CDLL with argument types set (raises if not built)."""
    global _lib
    with _lock:
        if _lib is None:
            path = _build.LIB
            if not os.path.exists(path):
                raise RuntimeError(f"{path} is missing: build it first "
                                   "(python -c 'import __graft_entry__ as g; g.build()')")
            handle = ctypes.CDLL(path)
            for name, (args, res) in _SIGNATURES.items():
                fn = getattr(handle, name)
                fn.argtypes = args
                fn.restype = res
            _lib = handle
    return _lib


def exported_symbols():
    return list(_SIGNATURES)


def _status_string(status: int) -> str:
    try:
        return lib().kda_status_string(status).decode()
    except Exception:  # library unavailable while formatting an error
        return f"status {status}"


def _check(status: int):
    if status != KDA_OK:
        raise KdaError(status, lib().kda_last_error_detail().decode())


def _dtype_code(t) -> int:
    import torch
    if t.dtype == torch.bfloat16:
        return KDA_BF16
    if t.dtype == torch.float32:
        return KDA_F32
    raise TypeError(f"unsupported dtype {t.dtype}; use float32 or bfloat16")


def _ptr(t):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("tensors must be on a CUDA device")
    if not t.is_contiguous():
        raise ValueError("tensors must be contiguous")
    return t.data_ptr()


def _stream(stream, device):
    import torch
    if stream is None:
        stream = torch.cuda.current_stream(device)
    return stream.cuda_stream


def _on_stream(stream):
    """Context in which `stream` is current (nothing changes for None). Device memory that a call needs for
    itself is allocated in it: the caching allocator gives a block back to the stream that it was allocated
    on, in that stream's order. Allocated on another stream, the block could be handed out there again while
    the call's kernels still use it, or still be in use by work queued there before."""
    import contextlib
    import torch
    return contextlib.nullcontext() if stream is None else torch.cuda.stream(stream)


def _scratch(workspace, need, device, stream):
    """The caller's workspace and its size, or `need` bytes allocated for a call on `stream` when None."""
    if workspace is None and need > 0:
        import torch
        with _on_stream(stream):
            workspace = torch.empty(need, dtype=torch.uint8, device=device)
    return workspace, 0 if workspace is None else workspace.numel() * workspace.element_size()


def state_bytes(layers, heads, dk, dv) -> int:
    return int(lib().kda_state_bytes(layers, heads, dk, dv))


def shortconv_ring_bytes(layers, batch, heads, d, elem_bytes) -> int:
    return int(lib().kda_shortconv_ring_bytes(layers, batch, heads, d, elem_bytes))


def kda_shortconv_step(x, ring, w, y, stream=None):
    """x [B,3,H,D], ring [B,3,H,3,D] (in/out), w [3,H,D,4] fp32, y [3,B,H,D]."""
    B, P, H, D = x.shape
    if P != 3 or tuple(ring.shape) != (B, 3, H, 3, D) or tuple(w.shape) != (3, H, D, 4) \
            or tuple(y.shape) != (3, B, H, D):
        raise ValueError("shape mismatch")
    _check(lib().kda_shortconv_step(_ptr(x), _ptr(ring), _ptr(w), _ptr(y), B, H, D, _dtype_code(x),
                                    _stream(stream, x.device)))


def kda_shortconv_prefill(x, w, y, ring_in=None, ring_out=None, cu_seqlens=None, stream=None):
    """x [T,3,H,D]; w [3,H,D,4] fp32; y [3,T,H,D]; rings [N,3,H,3,D] or None;
    cu_seqlens int64 [N+1] on the device (or None for one sequence)."""
    T, P, H, D = x.shape
    N = 1 if cu_seqlens is None else cu_seqlens.shape[0] - 1
    if P != 3 or tuple(w.shape) != (3, H, D, 4) or tuple(y.shape) != (3, T, H, D):
        raise ValueError("shape mismatch")
    for r in (ring_in, ring_out):
        if r is not None and tuple(r.shape) != (N, 3, H, 3, D):
            raise ValueError("ring shape mismatch")
    _check(lib().kda_shortconv_prefill(_ptr(x), _ptr(ring_in), _ptr(w), _ptr(y), _ptr(ring_out),
                                       _ptr(cu_seqlens), N, T, H, D, _dtype_code(x), _stream(stream, x.device)))


def kda_decode_step(q, k, v, g, beta, state, out, l2_eps=1e-6, stream=None):
    """q,k,v,out [B,H,D]; g [B,H,D] fp32; beta [B,H] fp32; state [B,H,D,D] fp32 (in/out)."""
    B, H, D = q.shape
    if tuple(g.shape) != (B, H, D) or tuple(beta.shape) != (B, H) or tuple(state.shape) != (B, H, D, D) \
            or tuple(out.shape) != (B, H, D):
        raise ValueError("shape mismatch")
    _check(lib().kda_decode_step(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(state), _ptr(out),
                                 B, H, D, _dtype_code(q), float(l2_eps), _stream(stream, q.device)))


def kda_decode_step_gated(q, k, v, g, beta, state, out, gate="channel", l2_eps=1e-6, stream=None):
    """kda_decode_step with gate "channel" (g [B,H,D]), "head" (g [B,H]) or "none" (g unused)."""
    B, H, D = q.shape
    code = _check_gate(g, gate, (B,), H, D)
    if tuple(beta.shape) != (B, H) or tuple(state.shape) != (B, H, D, D) or tuple(out.shape) != (B, H, D):
        raise ValueError("shape mismatch")
    _check(lib().kda_decode_step_gated(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(state), _ptr(out),
                                       B, H, D, _dtype_code(q), code, float(l2_eps), _stream(stream, q.device)))


def kda_shortconv_decode_step_gated(x, ring, w, g, beta, state, out, gate="channel", l2_eps=1e-6, stream=None):
    """kda_shortconv_decode_step with a gate form as in kda_decode_step_gated."""
    B, P, H, D = x.shape
    code = _check_gate(g, gate, (B,), H, D)
    if P != 3 or tuple(ring.shape) != (B, 3, H, 3, D) or tuple(w.shape) != (3, H, D, 4) \
            or tuple(beta.shape) != (B, H) or tuple(state.shape) != (B, H, D, D) or tuple(out.shape) != (B, H, D):
        raise ValueError("shape mismatch")
    _check(lib().kda_shortconv_decode_step_gated(_ptr(x), _ptr(ring), _ptr(w), _ptr(g), _ptr(beta), _ptr(state),
                                                 _ptr(out), B, H, D, _dtype_code(x), code, float(l2_eps),
                                                 _stream(stream, x.device)))


def kda_shortconv_decode_step_ex(x, ring, w, g, beta, state, out, gate="channel", l2_eps=1e-6,
                                 overlap_prev=False, stream=None):
    """kda_shortconv_decode_step_gated with launch flags. overlap_prev=True is
    the caller's promise that the kernel enqueued just before on the stream
    does not write `state` (e.g. the step of another layer); the launch may
    then overlap that kernel's tail (KDA_DECODE_OVERLAP_PREV)."""
    B, P, H, D = x.shape
    code = _check_gate(g, gate, (B,), H, D)
    if P != 3 or tuple(ring.shape) != (B, 3, H, 3, D) or tuple(w.shape) != (3, H, D, 4) \
            or tuple(beta.shape) != (B, H) or tuple(state.shape) != (B, H, D, D) or tuple(out.shape) != (B, H, D):
        raise ValueError("shape mismatch")
    flags = KDA_DECODE_OVERLAP_PREV if overlap_prev else 0
    _check(lib().kda_shortconv_decode_step_ex(_ptr(x), _ptr(ring), _ptr(w), _ptr(g), _ptr(beta), _ptr(state),
                                              _ptr(out), B, H, D, _dtype_code(x), code, float(l2_eps), flags,
                                              _stream(stream, x.device)))


def kda_shortconv_decode_step_epi(x, ring, w, g, beta, state, out_gate, norm_weight, y, gate="channel",
                                  act="sigmoid", l2_eps=1e-6, norm_eps=1e-6, overlap_prev=False, stream=None):
    """Fused short conv + decode step whose output goes through the gated
    RMSNorm epilogue before it is stored: y = RMSNorm(o) * norm_weight *
    act(out_gate), o the step's output (fp32 inside the kernel). out_gate and
    y [B,H,D] like x; norm_weight [D] fp32; other arguments as
    kda_shortconv_decode_step_ex."""
    B, P, H, D = x.shape
    code = _check_gate(g, gate, (B,), H, D)
    if P != 3 or tuple(ring.shape) != (B, 3, H, 3, D) or tuple(w.shape) != (3, H, D, 4) \
            or tuple(beta.shape) != (B, H) or tuple(state.shape) != (B, H, D, D) or tuple(y.shape) != (B, H, D) \
            or tuple(out_gate.shape) != (B, H, D) or tuple(norm_weight.shape) != (D,):
        raise ValueError("shape mismatch")
    if act not in _ACTS:
        raise ValueError(f"act must be one of {sorted(_ACTS)}")
    flags = KDA_DECODE_OVERLAP_PREV if overlap_prev else 0
    _check(lib().kda_shortconv_decode_step_epi(_ptr(x), _ptr(ring), _ptr(w), _ptr(g), _ptr(beta), _ptr(state),
                                               _ptr(out_gate), _ptr(norm_weight), _ptr(y), B, H, D, _dtype_code(x),
                                               code, _ACTS[act], float(l2_eps), float(norm_eps), flags,
                                               _stream(stream, x.device)))


def kda_shortconv_decode_step(x, ring, w, g, beta, state, out, l2_eps=1e-6, stream=None):
    """Fused short conv + decode step. x [B,3,H,D], ring [B,3,H,3,D] (in/out),
    w [3,H,D,4] fp32, g [B,H,D] fp32, beta [B,H] fp32, state [B,H,D,D] fp32
    (in/out), out [B,H,D]."""
    B, P, H, D = x.shape
    if P != 3 or tuple(ring.shape) != (B, 3, H, 3, D) or tuple(w.shape) != (3, H, D, 4) \
            or tuple(g.shape) != (B, H, D) or tuple(beta.shape) != (B, H) \
            or tuple(state.shape) != (B, H, D, D) or tuple(out.shape) != (B, H, D):
        raise ValueError("shape mismatch")
    _check(lib().kda_shortconv_decode_step(_ptr(x), _ptr(ring), _ptr(w), _ptr(g), _ptr(beta), _ptr(state),
                                           _ptr(out), B, H, D, _dtype_code(x), float(l2_eps),
                                           _stream(stream, x.device)))


def kda_gated_rmsnorm(o, gate, weight, y, act="sigmoid", eps=1e-6, stream=None):
    """Output epilogue: y = RMSNorm(o) * weight * act(gate) per (token, head)
    row. o, gate, y [T,H,D] (y may be o); weight [D] fp32; act "sigmoid" or
    "silu"."""
    T, H, D = o.shape
    if tuple(gate.shape) != (T, H, D) or tuple(y.shape) != (T, H, D) or tuple(weight.shape) != (D,):
        raise ValueError("shape mismatch")
    if act not in _ACTS:
        raise ValueError(f"act must be one of {sorted(_ACTS)}")
    _check(lib().kda_gated_rmsnorm(_ptr(o), _ptr(gate), _ptr(weight), _ptr(y), T, H, D, _dtype_code(o),
                                   _ACTS[act], float(eps), _stream(stream, o.device)))


_calls = None


def _fastcall():
    """The extension that checks the tensors of the 8-bit operators and of the softmax-attention layers' and calls the
    library (raises if not built)."""
    global _calls
    if _calls is None:
        import importlib.machinery
        import importlib.util
        import torch
        path = _build.FASTCALL
        if not os.path.exists(path):
            raise RuntimeError(f"{path} is missing: build it first, with a C compiler and Python.h "
                               "(python -c 'import __graft_entry__ as g; g.build()')")
        spec = importlib.util.spec_from_loader(
            "kda_fastcall", importlib.machinery.ExtensionFileLoader("kda_fastcall", path))
        mod = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(mod)
        handle = lib()
        mod.setup(*(ctypes.cast(f, ctypes.c_void_p).value for f in (
                      handle.kda_add_rmsnorm_fp8, handle.kda_gated_rmsnorm_fp8, handle.kda_fp8_linear,
                      handle.kda_qk_norm_rope, handle.kda_kv4_append, handle.kda_kv4_read, handle.kda_kv4_attention,
                      handle.kda_kv4_attention_workspace_bytes)),
                  torch.float32, torch.bfloat16, torch.float8_e4m3fn, torch.float64, torch.int64, torch.int32, torch.uint8,
                  torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream)
        _calls = mod
    return _calls


def _settle(status, fn, device, *args):
    """A call's status other than KDA_OK: an error, or (-1) tensors on another device than the current one
    and no stream named: the call again with that device current (the handle of a default stream does not
    name its device)."""
    if status == -1:
        import torch
        with torch.cuda.device(device):
            status = fn(*args)
    if status != KDA_OK:
        _check(status)


def kda_add_rmsnorm_fp8(x, weight, y, scales, residual=None, sum_out=None, eps=1e-6, stream=None):
    """h = x + residual, then RMSNorm(h) * weight in 8 bits. x [T,N] fp32 or bf16; residual [T,N] fp32
    or bf16, or None (h = x); weight [N] fp32; sum_out receives h (residual's shape and type; may be
    residual, or x where the types agree), or None; y [T,N] float8_e4m3fn; scales [ceil(N/128),T] fp32
    with y about code * scales[channel // 128, token]."""
    fn = (_calls or _fastcall()).add_rmsnorm
    status = fn(x, weight, y, scales, residual, sum_out, eps, stream)
    if status:
        _settle(status, fn, x.device, x, weight, y, scales, residual, sum_out, eps, stream)


def kda_gated_rmsnorm_fp8(o, gate, weight, y, scales, act="sigmoid", eps=1e-6, stream=None):
    """kda_gated_rmsnorm with its output in 8 bits. o, gate [T,H,D]; weight [D] fp32; y [T,H,D]
    float8_e4m3fn; scales [ceil(H*D/128),T] fp32, one per token and 128 of its H * D channels."""
    code = _ACTS.get(act)
    if code is None:
        raise ValueError(f"act must be one of {sorted(_ACTS)}")
    fn = (_calls or _fastcall()).gated_rmsnorm
    status = fn(o, gate, weight, y, scales, code, eps, stream)
    if status:
        _settle(status, fn, o.device, o, gate, weight, y, scales, code, eps, stream)


def kda_fp8_linear(a, a_scales, w, w_scales, y, stream=None):
    """y[m,n] = sum_k a[m,k] a_scales[k//128,m] * w[n,k] w_scales[n//128,k//128]. a [M,K], w [N,K]
    float8_e4m3fn (rows contiguous, row strides multiples of 16); a_scales [ceil(K/128),M] and w_scales
    [ceil(N/128),ceil(K/128)] fp32; y [M,N] bf16 or fp32 (rows contiguous)."""
    fn = (_calls or _fastcall()).linear
    status = fn(a, a_scales, w, w_scales, y, stream)
    if status:
        _settle(status, fn, a.device, a, a_scales, w, w_scales, y, stream)


def _check_kinds(like, floats, ints, x, workspace, stream):
    """Types and devices of a one-call way out's tensors (None: absent): the library sees pointers alone, and would
    read and write past the end of a tensor of a narrower type. `like` have x's type, `floats` float32, `ints` int64.
    A given stream has to be on their device too."""
    import torch
    for group, dtype, what in ((like, x.dtype, "must have the inputs' dtype"),
                               (floats, torch.float32, "must be float32"), (ints, torch.int64, "must be int64")):
        for name, t in group.items():
            if t is not None and t.dtype != dtype:
                raise TypeError(f"{name} {what}")
    for t in (*like.values(), *floats.values(), *ints.values(), workspace):
        if t is not None and t.device != x.device:
            raise ValueError("tensors must be on one CUDA device")
    if stream is not None and getattr(stream, "device", x.device) != x.device:
        raise ValueError("stream must be on the tensors' device")


def _check_proj(out_gate, norm_weight, proj, proj_scales, y, lead, H, D, x):
    """Shapes, types and devices of the output projection's arguments; returns Nout."""
    import torch
    Nout = proj.shape[0]
    if tuple(out_gate.shape) != (lead, H, D) or tuple(norm_weight.shape) != (D,) \
            or tuple(proj.shape) != (Nout, H * D) or tuple(y.shape) != (lead, Nout) \
            or tuple(proj_scales.shape) != ((Nout + 127) // 128, (H * D + 127) // 128):
        raise ValueError("shape mismatch")
    if proj.dtype != torch.float8_e4m3fn:
        raise TypeError("8-bit codes must be torch.float8_e4m3fn")
    if proj_scales.dtype != torch.float32 or norm_weight.dtype != torch.float32:
        raise TypeError("scales and norm weights must be float32")
    if out_gate.dtype != x.dtype or y.dtype != x.dtype:
        raise TypeError("out_gate and y must have the inputs' dtype")
    for t in (out_gate, norm_weight, proj, proj_scales, y):
        if t.device != x.device:
            raise ValueError("tensors must be on one CUDA device")
    return Nout


def _current(device):
    """Context in which `device` is current (a default stream's handle does not name its device)."""
    import torch
    if device.type != "cuda":
        raise ValueError("tensors must be on a CUDA device")
    return torch.cuda.device(device)


def kda_shortconv_decode_step_proj(x, ring, w, g, beta, state, out_gate, norm_weight, proj, proj_scales, y,
                                   gate="channel", act="sigmoid", l2_eps=1e-6, norm_eps=1e-6, overlap_prev=False,
                                   workspace=None, stream=None):
    """Fused short conv + decode step, gated RMSNorm in 8 bits and output projection in one call. proj
    [Nout,H*D] float8_e4m3fn with proj_scales [ceil(Nout/128),ceil(H*D/128)] fp32; y [B,Nout] like x;
    workspace: a device uint8 tensor of kda_shortconv_decode_step_proj_workspace_bytes (allocated here when
    None); other arguments as kda_shortconv_decode_step_epi."""
    B, P, H, D = x.shape
    code = _check_gate(g, gate, (B,), H, D)
    if P != 3 or tuple(ring.shape) != (B, 3, H, 3, D) or tuple(w.shape) != (3, H, D, 4) \
            or tuple(beta.shape) != (B, H) or tuple(state.shape) != (B, H, D, D):
        raise ValueError("shape mismatch")
    if act not in _ACTS:
        raise ValueError(f"act must be one of {sorted(_ACTS)}")
    Nout = _check_proj(out_gate, norm_weight, proj, proj_scales, y, B, H, D, x)
    _check_kinds({"ring": ring}, {"w": w, "g": None if code == KDA_GATE_NONE else g, "beta": beta, "state": state},
                 {}, x, workspace, stream)
    workspace, size = _scratch(workspace, kda_shortconv_decode_step_proj_workspace_bytes(B, H, D), x.device, stream)
    flags = KDA_DECODE_OVERLAP_PREV if overlap_prev else 0
    with _current(x.device):
        _check(lib().kda_shortconv_decode_step_proj(
            _ptr(x), _ptr(ring), _ptr(w), _ptr(g), _ptr(beta), _ptr(state), _ptr(out_gate), _ptr(norm_weight),
            _ptr(proj), _ptr(proj_scales), _ptr(y), B, H, D, Nout, _dtype_code(x), code, _ACTS[act], float(l2_eps),
            float(norm_eps), flags, _ptr(workspace), size, _stream(stream, x.device)))


def kda_shortconv_decode_step_proj_workspace_bytes(B, H, D) -> int:
    return int(lib().kda_shortconv_decode_step_proj_workspace_bytes(B, H, D))


def kda_chunk_prefill_proj(q, k, v, g, beta, out_gate, norm_weight, proj, proj_scales, y, gate="channel",
                           act="sigmoid", norm_eps=1e-6, initial_state=None, final_state=None, cu_seqlens=None,
                           chunk_size=64, l2_eps=1e-6, workspace=None, stream=None):
    """Chunked prefill, gated RMSNorm in 8 bits and output projection in one call. proj, proj_scales as
    kda_shortconv_decode_step_proj; y [T,Nout] like q; workspace: a device uint8 tensor of
    kda_chunk_prefill_proj_workspace_bytes (allocated here when None); other arguments as
    kda_chunk_prefill_epi."""
    T, H, D = q.shape
    code = _check_gate(g, gate, (T,), H, D)
    if act not in _ACTS:
        raise ValueError(f"act must be one of {sorted(_ACTS)}")
    N = 1 if cu_seqlens is None else cu_seqlens.shape[0] - 1
    if tuple(k.shape) != (T, H, D) or tuple(v.shape) != (T, H, D) or tuple(beta.shape) != (T, H):
        raise ValueError("shape mismatch")
    for st in (initial_state, final_state):
        if st is not None and st.numel() != N * H * D * D:
            raise ValueError("state shape mismatch")
    Nout = _check_proj(out_gate, norm_weight, proj, proj_scales, y, T, H, D, q)
    _check_kinds({"k": k, "v": v}, {"g": None if code == KDA_GATE_NONE else g, "beta": beta,
                                    "initial_state": initial_state, "final_state": final_state},
                 {"cu_seqlens": cu_seqlens}, q, workspace, stream)
    workspace, size = _scratch(workspace, kda_chunk_prefill_proj_workspace_bytes(T, N, H, D, chunk_size), q.device,
                               stream)
    with _current(q.device):
        _check(lib().kda_chunk_prefill_proj(
            _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(initial_state), _ptr(final_state), _ptr(cu_seqlens),
            N, T, H, D, chunk_size, _dtype_code(q), code, float(l2_eps), _ptr(out_gate), _ptr(norm_weight), _ACTS[act],
            float(norm_eps), _ptr(proj), _ptr(proj_scales), _ptr(y), Nout, _ptr(workspace), size,
            _stream(stream, q.device)))


def kda_chunk_prefill_proj_workspace_bytes(total_tokens, num_seqs, H, D, C) -> int:
    return int(lib().kda_chunk_prefill_proj_workspace_bytes(total_tokens, num_seqs, H, D, C))


def kda_chunk_prefill_epi(q, k, v, g, beta, out, out_gate, norm_weight, gate="channel", act="sigmoid",
                          norm_eps=1e-6, initial_state=None, final_state=None, cu_seqlens=None, chunk_size=64,
                          l2_eps=1e-6, workspace=None, stream=None):
    """kda_chunk_prefill_gated whose output goes through the gated RMSNorm
    epilogue in the same call: out = RMSNorm(o) * norm_weight * act(out_gate).
    out_gate [T,H,D] like q; norm_weight [D] fp32."""
    T, H, D = q.shape
    code = _check_gate(g, gate, (T,), H, D)
    if tuple(out_gate.shape) != (T, H, D) or tuple(norm_weight.shape) != (D,):
        raise ValueError("shape mismatch")
    if act not in _ACTS:
        raise ValueError(f"act must be one of {sorted(_ACTS)}")
    N = 1 if cu_seqlens is None else cu_seqlens.shape[0] - 1
    workspace, wsz = _scratch(workspace, kda_chunk_prefill_workspace_bytes(T, N, H, D, chunk_size), q.device, stream)
    _check(lib().kda_chunk_prefill_epi(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(initial_state),
                                       _ptr(final_state), _ptr(out), _ptr(cu_seqlens), N, T, H, D, chunk_size,
                                       _dtype_code(q), code, float(l2_eps), _ptr(out_gate), _ptr(norm_weight),
                                       _ACTS[act], float(norm_eps), _ptr(workspace), wsz, _stream(stream, q.device)))


def kda_chunk_prefill_scan_workspace_bytes(T, H, D, C, segments) -> int:
    return int(lib().kda_chunk_prefill_scan_workspace_bytes(T, H, D, C, segments))


def kda_chunk_prefill_scan(q, k, v, g, beta, out, segments, initial_state=None, final_state=None, gate="channel",
                           chunk_size=64, l2_eps=1e-6, workspace=None, stream=None):
    """Prefill of one long sequence split into `segments` runs processed side
    by side. q,k,v,out [T,H,D]; g per `gate`; beta [T,H]; states [H,D,D] fp32.
    workspace: a device uint8 tensor of kda_chunk_prefill_scan_workspace_bytes
    (allocated here when None)."""
    T, H, D = q.shape
    code = _check_gate(g, gate, (T,), H, D)
    workspace, wsz = _scratch(workspace, kda_chunk_prefill_scan_workspace_bytes(T, H, D, chunk_size, segments), q.device,
                              stream)
    _check(lib().kda_chunk_prefill_scan(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(initial_state),
                                        _ptr(final_state), _ptr(out), T, H, D, chunk_size, _dtype_code(q), code,
                                        float(l2_eps), int(segments), _ptr(workspace), wsz,
                                        _stream(stream, q.device)))


def kda_chunk_prefill_route(D, C, dtype) -> str | None:
    """Name of the kernel the chunked prefill runs for this head dimension, chunk size and dtype
    (torch.bfloat16 / torch.float32 or the KDA_* dtype code); None for an unsupported shape."""
    if isinstance(dtype, int):
        code = dtype
    else:
        import torch
        code = {torch.bfloat16: KDA_BF16, torch.float32: KDA_F32}[dtype]
    r = lib().kda_chunk_prefill_route(int(D), int(C), int(code))
    return None if r is None else r.decode()


def kda_chunk_prefill_workspace_bytes(total_tokens, num_seqs, H, D, C) -> int:
    return int(lib().kda_chunk_prefill_workspace_bytes(total_tokens, num_seqs, H, D, C))


def kda_chunk_prefill(q, k, v, g, beta, out, initial_state=None, final_state=None, cu_seqlens=None,
                      chunk_size=64, l2_eps=1e-6, workspace=None, stream=None):
    """q,k,v,out [T,H,D]; g [T,H,D] fp32; beta [T,H] fp32; states [N,H,D,D] fp32;
    cu_seqlens int64 [N+1] on the device (or None for one sequence)."""
    T, H, D = q.shape
    N = 1 if cu_seqlens is None else cu_seqlens.shape[0] - 1
    workspace, wsz = _scratch(workspace, kda_chunk_prefill_workspace_bytes(T, N, H, D, chunk_size), q.device, stream)
    _check(lib().kda_chunk_prefill(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(initial_state),
                                   _ptr(final_state), _ptr(out), _ptr(cu_seqlens), N, T, H, D, chunk_size,
                                   _dtype_code(q), float(l2_eps), _ptr(workspace), wsz,
                                   _stream(stream, q.device)))


def kda_chunk_prefill_gated(q, k, v, g, beta, out, gate="channel", initial_state=None, final_state=None,
                            cu_seqlens=None, chunk_size=64, l2_eps=1e-6, workspace=None, stream=None):
    """kda_chunk_prefill with gate "channel" (g [T,H,D]), "head" (g [T,H]) or "none" (g unused)."""
    T, H, D = q.shape
    code = _check_gate(g, gate, (T,), H, D)
    N = 1 if cu_seqlens is None else cu_seqlens.shape[0] - 1
    workspace, wsz = _scratch(workspace, kda_chunk_prefill_workspace_bytes(T, N, H, D, chunk_size), q.device, stream)
    _check(lib().kda_chunk_prefill_gated(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(initial_state),
                                         _ptr(final_state), _ptr(out), _ptr(cu_seqlens), N, T, H, D, chunk_size,
                                         _dtype_code(q), code, float(l2_eps), _ptr(workspace), wsz,
                                         _stream(stream, q.device)))


def _host_cu(cu_seqlens):
    import numpy as np
    a = cu_seqlens.detach().cpu().numpy() if hasattr(cu_seqlens, "detach") else cu_seqlens
    return np.ascontiguousarray(a, dtype=np.int64)


def kda_chunk_prefill_split_plan(cu_seqlens, H, chunk_size=64, sms=0):
    """Segment count per sequence that kda_chunk_prefill_split uses (1: kept whole) and the number of
    split sequences; `sms` <= 0 plans for the current device."""
    import numpy as np
    cu = _host_cu(cu_seqlens)
    N = cu.shape[0] - 1
    seg = np.zeros(max(N, 1), dtype=np.int32)
    n = lib().kda_chunk_prefill_split_plan(cu.ctypes.data, N, H, chunk_size, sms, seg.ctypes.data)
    if n < 0:
        raise KdaError(KDA_ERR_INVALID_ARG, "invalid cu_seqlens")
    return seg[:N], n


def kda_chunk_prefill_split(q, k, v, g, beta, out, cu_seqlens, gate="channel", initial_state=None,
                            final_state=None, chunk_size=64, l2_eps=1e-6, workspace=None, stream=None):
    """Chunked prefill of a packed batch that splits its long sequences through the chunk-state scan.
    cu_seqlens: the [N+1] offsets, on the host or the device (a host copy is taken here, a device
    copy made when it lives on the host); other arguments as kda_chunk_prefill_gated."""
    import torch
    T, H, D = q.shape
    code = _check_gate(g, gate, (T,), H, D)
    host = _host_cu(cu_seqlens)
    dev_cu = cu_seqlens
    if not (hasattr(cu_seqlens, "is_cuda") and cu_seqlens.is_cuda):
        with _on_stream(stream):
            dev_cu = torch.from_numpy(host).to(q.device)
    N = host.shape[0] - 1
    need = int(lib().kda_chunk_prefill_split_workspace_bytes(host.ctypes.data, N, H, D, chunk_size))
    workspace, wsz = _scratch(workspace, need, q.device, stream)
    _check(lib().kda_chunk_prefill_split(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(initial_state),
                                         _ptr(final_state), _ptr(out), _ptr(dev_cu), host.ctypes.data, N, T, H, D,
                                         chunk_size, _dtype_code(q), code, float(l2_eps), _ptr(workspace), wsz,
                                         _stream(stream, q.device)))


def kda_chunk_prefill_noalloc(q, k, v, g, beta, out, initial_state=None, final_state=None, cu_seqlens=None,
                              chunk_size=64, l2_eps=1e-6, stream=None):
    """kda_chunk_prefill without a workspace, for callers that cannot allocate
    device memory: the launch-order scratch lives in a fixed array owned by
    the library (at most 4096 sequences). Overlapping calls race on it."""
    T, H, D = q.shape
    N = 1 if cu_seqlens is None else cu_seqlens.shape[0] - 1
    _check(lib().kda_chunk_prefill_noalloc(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(initial_state),
                                           _ptr(final_state), _ptr(out), _ptr(cu_seqlens), N, T, H, D, chunk_size,
                                           _dtype_code(q), float(l2_eps), _stream(stream, q.device)))


def kda_qk_norm_rope(q, k, q_out, k_out, positions, inv_freq, q_weight=None, k_weight=None, eps=1e-6,
                     interleaved=False, stream=None):
    """RMSNorm of every query and key head (skipped where its weight is None) and the rotation of the first
    2 * len(inv_freq) channels by positions * inv_freq. q [T,Hq,D], k [T,Hk,D] and the outputs: heads contiguous,
    any token stride; k and k_out may be None; q_out may be q, k_out k. positions int64 [T] and inv_freq fp64 [R/2]
    (both None: no rotation); weights [D] fp32. interleaved: pairs are neighbouring channels, else i and i + R/2."""
    fn = (_calls or _fastcall()).norm_rope
    args = (q, k, q_out, k_out, positions, inv_freq, q_weight, k_weight, eps, interleaved, stream)
    status = fn(*args)
    if status:
        _settle(status, fn, q.device, *args)


def kda_kv4_cache_bytes(pages, Hk, page_size, D) -> int:
    return int(lib().kda_kv4_cache_bytes(pages, Hk, page_size, D))


def kda_kv4_cache_shape(pages, Hk, page_size, D):
    """Shape of the uint8 tensor that holds `pages` pages of page_size tokens of Hk key/value heads."""
    if pages != 0 and kda_kv4_cache_bytes(pages, Hk, page_size, D) == 0:
        raise ValueError("page_size must be 16, 32, 64, 128 or 256, D 64 or 128, Hk 1 to 32768, pages at most 2^31 - 1")
    return pages, Hk, page_size // 16, 18 * D


def kda_kv4_append(k, v, cache, block_table, lens, cu_seqlens=None, stream=None):
    """Quantise new keys and values k, v [T,Hk,D] (heads contiguous, any token stride) into the 4-bit cache (uint8
    [pages,Hk,page_size/16,18*D]). block_table int32 [B,cols]; lens int64 [B] counts the new tokens; cu_seqlens int64
    [B+1] (None: one new token for each sequence): the new tokens are the last ones of each sequence."""
    fn = (_calls or _fastcall()).kv4_rows
    status = fn(k, v, cache, block_table, lens, cu_seqlens, stream, False)
    if status:
        _settle(status, fn, k.device, k, v, cache, block_table, lens, cu_seqlens, stream, False)


def kda_kv4_read(cache, block_table, lens, k, v, cu_seqlens=None, stream=None):
    """What the cache holds for the last cu_seqlens[b+1] - cu_seqlens[b] tokens of each sequence, into k, v
    [T,Hk,D]. Arguments as kda_kv4_append."""
    fn = (_calls or _fastcall()).kv4_rows
    status = fn(k, v, cache, block_table, lens, cu_seqlens, stream, True)
    if status:
        _settle(status, fn, k.device, k, v, cache, block_table, lens, cu_seqlens, stream, True)


def kda_kv4_attention(q, cache, block_table, lens, out, cu_seqlens=None, scale=None, causal=True, window=0, lse=None,
                      workspace=None, stream=None):
    """out = softmax(scale q K^T + mask) V over the 4-bit cache for new queries q [T,Hq,D] (heads contiguous, any token
    stride; out alike), Hq a multiple of the cache's heads. scale: 1/sqrt(D) when None. causal: a query sees the tokens
    up to its own position, else all of lens[b]; window > 0: only the last `window` of them. lse [T,Hq] fp32 or None
    receives the log of the sum of exponentials. workspace: a device uint8 tensor of
    kda_kv4_attention_workspace_bytes (allocated here when None); other arguments as kda_kv4_append."""
    fn = (_calls or _fastcall()).kv4_attention
    args = (q, cache, block_table, lens, out, cu_seqlens, scale, causal, window, lse)
    status = fn(*args, workspace, stream)
    if status == -1:
        with _current(q.device):
            return kda_kv4_attention(*args[:6], scale=scale, causal=causal, window=window, lse=lse, workspace=workspace,
                                     stream=stream)
    if status < -1:  # the workspace that these sizes need
        workspace, _ = _scratch(None, -status, q.device, stream)
        status = fn(*args, workspace, stream)
    if status:
        _check(status)


def kda_kv4_attention_workspace_bytes(B, T, Hq, Hk, D, page_size, table_cols, with_cu_seqlens, dtype, window=0) -> int:
    """Workspace of a kda_kv4_attention of these sizes on the current device (0: none); dtype torch.bfloat16 or
    torch.float32."""
    import torch
    code = {torch.bfloat16: KDA_BF16, torch.float32: KDA_F32}[dtype]
    return int(lib().kda_kv4_attention_workspace_bytes(B, T, Hq, Hk, D, page_size, table_cols, int(with_cu_seqlens), window,
                                                       code))


def kda_selftest_bounded_wait(limit_cycles=2_000_000, stream=None, device=None):
    """Launch the bounded-wait diagnostic (a wait nothing completes); the next
    kda_sync_status on the stream then raises with KDA_ERR_TIMEOUT."""
    import torch
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else device
    _check(lib().kda_selftest_bounded_wait(int(limit_cycles), _stream(stream, dev)))


def kda_sync_status(stream=None, device=None):
    import torch
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else device
    _check(lib().kda_sync_status(_stream(stream, dev)))
