"""Python binding of the gfx950 gated delta rule library (``libgdn.so``).

Argument marshalling only: each function checks tensor dtypes, shapes and
devices, allocates outputs and workspace with torch (device memory is torch's
business), and calls the C entry point of the same name on torch's current
stream.  All computation happens in the HIP kernels; there is no fallback.
If the library is not built, every call raises.
"""
from __future__ import annotations

import ctypes
import os

__all__ = [
    "lib_path", "load", "status_string",
    "gdn_chunk_fwd", "gdn_chunk_intra", "gdn_chunk_walk", "gdn2_chunk_fwd", "gdn_recurrent_step",
    "gdn2_recurrent_step", "gdn_chunk_bwd", "gdn_chunk_bwd_workspace", "gdn_chunk_fwd_varlen",
    "gdn2_chunk_fwd_varlen", "gdn2_chunk_fwd_varlen_workspace",
    "gdn_chunk_fwd_workspace", "gdn2_chunk_fwd_workspace", "gdn_prologue", "gdn_gated_rmsnorm",
    "gdn2_chunk_bwd", "gdn2_chunk_bwd_workspace", "gdn2_chunk_fwd_noalloc", "gdn2_chunk_fwd_noalloc_max_bytes",
    "gdn_add_rmsnorm", "gdn_add_rmsnorm_bwd", "gdn_add_rmsnorm_bwd_workspace", "gdn_quantize_rows",
    "gdn_linear", "gdn_linear_workspace", "gdn_linear_bwd", "gdn_linear_bwd_workspace",
    "gdn_linear_plan", "gdn_linear_bwd_plan",
    "gdn_add_layernorm", "gdn_add_layernorm_bwd", "gdn_add_layernorm_bwd_workspace",
    "gdn_gated_linear", "gdn_gated_linear_workspace", "gdn_gated_linear_bwd", "gdn_gated_linear_bwd_workspace",
    "gdn_causal_conv", "gdn_causal_conv_varlen",
    "gdn_selective_scan", "gdn_selective_scan_workspace", "gdn_selective_scan_varlen",
    "gdn_selective_scan_varlen_workspace", "gdn_selective_step",
    "clock_probe",
    "GDN_F32", "GDN_BF16", "GDN_F8E4M3", "BT",
]

_HERE = os.path.dirname(os.path.abspath(__file__))
lib_path = os.path.join(_HERE, "libgdn.so")

GDN_F32, GDN_BF16, GDN_F8E4M3 = 0, 1, 2
BT = 64
_lib = None

_vp = ctypes.c_void_p
_i = ctypes.c_int
_f = ctypes.c_float
_sz = ctypes.c_size_t


def load():
    """Load libgdn.so and declare its C signatures (raises if not built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(lib_path):
        raise RuntimeError(f"{lib_path} is not built; run `python gated_delta_rule_34_amd/build.py`")
    lib = ctypes.CDLL(lib_path)
    lib.gdn_status_string.restype = ctypes.c_char_p
    lib.gdn_status_string.argtypes = [_i]
    lib.gdn_chunk_fwd_workspace.restype = _sz
    lib.gdn_chunk_fwd_workspace.argtypes = [_i] * 6
    lib.gdn2_chunk_fwd_workspace.restype = _sz
    lib.gdn2_chunk_fwd_workspace.argtypes = [_i] * 6
    lib.gdn_chunk_fwd.restype = _i
    lib.gdn_chunk_fwd.argtypes = [_vp] * 8 + [_i] * 6 + [_f, _vp, _sz, _vp]
    lib.gdn_chunk_intra.restype = _i
    lib.gdn_chunk_intra.argtypes = [_vp] * 5 + [_i] * 5 + [_vp]
    lib.gdn_chunk_walk.restype = _i
    lib.gdn_chunk_walk.argtypes = [_vp] * 9 + [_i] * 6 + [_f, _vp]
    lib.gdn2_chunk_fwd.restype = _i
    lib.gdn2_chunk_fwd.argtypes = [_vp] * 9 + [_i] * 6 + [_f, _vp, _sz, _vp]
    lib.gdn_recurrent_step.restype = _i
    lib.gdn_recurrent_step.argtypes = [_vp] * 7 + [_i] * 5 + [_f, _vp]
    lib.gdn_chunk_fwd_varlen.restype = _i
    lib.gdn_chunk_fwd_varlen.argtypes = [_vp] * 9 + [_i] * 6 + [_f, _vp]
    lib.gdn2_chunk_fwd_varlen_workspace.restype = _sz
    lib.gdn2_chunk_fwd_varlen_workspace.argtypes = [_i] * 6
    lib.gdn2_chunk_fwd_varlen.restype = _i
    lib.gdn2_chunk_fwd_varlen.argtypes = [_vp] * 10 + [_i] * 6 + [_f, _vp, _sz, _vp]
    lib.gdn_chunk_bwd_workspace.restype = _sz
    lib.gdn_chunk_bwd_workspace.argtypes = [_i] * 6
    lib.gdn_chunk_bwd.restype = _i
    lib.gdn_chunk_bwd.argtypes = [_vp] * 14 + [_i] * 6 + [_f, _vp, _sz, _vp]
    lib.gdn2_recurrent_step.restype = _i
    lib.gdn2_recurrent_step.argtypes = [_vp] * 8 + [_i] * 5 + [_f, _vp]
    lib.gdn2_chunk_bwd_workspace.restype = _sz
    lib.gdn2_chunk_bwd_workspace.argtypes = [_i] * 6
    lib.gdn2_chunk_bwd.restype = _i
    lib.gdn2_chunk_bwd.argtypes = [_vp] * 16 + [_i] * 6 + [_f, _vp, _sz, _vp]
    lib.gdn_prologue.restype = _i
    lib.gdn_prologue.argtypes = [_vp] * 17 + [_i] * 5 + [_vp]
    lib.gdn2_chunk_fwd_noalloc.restype = _i
    lib.gdn2_chunk_fwd_noalloc.argtypes = [_vp] * 9 + [_i] * 6 + [_f, _vp]
    lib.gdn2_chunk_fwd_noalloc_max_bytes.restype = _sz
    lib.gdn2_chunk_fwd_noalloc_max_bytes.argtypes = []
    lib.gdn_clock_probe.restype = _i
    lib.gdn_clock_probe.argtypes = [_vp, _i, _i, _vp]
    lib.gdn_gated_rmsnorm.restype = _i
    lib.gdn_gated_rmsnorm.argtypes = [_vp] * 4 + [ctypes.c_longlong, _i, _f, _vp]
    _ll = ctypes.c_longlong
    lib.gdn_add_rmsnorm.restype = _i
    lib.gdn_add_rmsnorm.argtypes = [_vp] * 7 + [_ll, _i, _i, _i, _i, _f, _vp]
    lib.gdn_add_rmsnorm_bwd_workspace.restype = _sz
    lib.gdn_add_rmsnorm_bwd_workspace.argtypes = [_ll, _i]
    lib.gdn_add_rmsnorm_bwd.restype = _i
    lib.gdn_add_rmsnorm_bwd.argtypes = [_vp] * 7 + [_ll, _i, _i, _i, _vp, _sz, _vp]
    lib.gdn_quantize_rows.restype = _i
    lib.gdn_quantize_rows.argtypes = [_vp] * 3 + [_ll, _i, _i, _vp]
    lib.gdn_linear_workspace.restype = _sz
    lib.gdn_linear_workspace.argtypes = [_i] * 4
    lib.gdn_linear.restype = _i
    lib.gdn_linear.argtypes = [_vp] * 8 + [_i] * 6 + [_vp, _sz, _vp]
    lib.gdn_linear_bwd_workspace.restype = _sz
    lib.gdn_linear_bwd_workspace.argtypes = [_i] * 9
    lib.gdn_linear_plan.restype = _i
    lib.gdn_linear_plan.argtypes = [_i] * 4 + [_vp]
    lib.gdn_linear_bwd_plan.restype = _i
    lib.gdn_linear_bwd_plan.argtypes = [_i] * 9 + [_vp]
    lib.gdn_linear_bwd.restype = _i
    lib.gdn_linear_bwd.argtypes = [_vp] * 7 + [_i] * 6 + [_vp, _sz, _vp]
    lib.gdn_add_layernorm.restype = _i
    lib.gdn_add_layernorm.argtypes = [_vp] * 9 + [_ll, _i, _i, _i, _i, _f, _vp]
    lib.gdn_add_layernorm_bwd_workspace.restype = _sz
    lib.gdn_add_layernorm_bwd_workspace.argtypes = [_ll, _i]
    lib.gdn_add_layernorm_bwd.restype = _i
    lib.gdn_add_layernorm_bwd.argtypes = [_vp] * 9 + [_ll, _i, _i, _i, _vp, _sz, _vp]
    lib.gdn_gated_linear_workspace.restype = _sz
    lib.gdn_gated_linear_workspace.argtypes = [_i] * 4
    lib.gdn_gated_linear.restype = _i
    lib.gdn_gated_linear.argtypes = [_vp] * 7 + [_i] * 6 + [_vp, _sz, _vp]
    lib.gdn_gated_linear_bwd_workspace.restype = _sz
    lib.gdn_gated_linear_bwd_workspace.argtypes = [_i] * 9
    lib.gdn_gated_linear_bwd.restype = _i
    lib.gdn_gated_linear_bwd.argtypes = [_vp] * 7 + [_i] * 6 + [_vp, _sz, _vp]
    lib.gdn_causal_conv.restype = _i
    lib.gdn_causal_conv.argtypes = [_vp] * 6 + [_i] * 6 + [_vp]
    lib.gdn_causal_conv_varlen.restype = _i
    lib.gdn_causal_conv_varlen.argtypes = [_vp] * 7 + [_i] * 6 + [_vp]
    lib.gdn_selective_scan_workspace.restype = _sz
    lib.gdn_selective_scan_workspace.argtypes = [_i] * 4
    lib.gdn_selective_scan.restype = _i
    lib.gdn_selective_scan.argtypes = [_vp] * 11 + [_i] * 5 + [_vp, _sz, _vp]
    lib.gdn_selective_scan_varlen_workspace.restype = _sz
    lib.gdn_selective_scan_varlen_workspace.argtypes = [_i] * 4
    lib.gdn_selective_scan_varlen.restype = _i
    lib.gdn_selective_scan_varlen.argtypes = [_vp] * 12 + [_i] * 5 + [_vp, _sz, _vp]
    lib.gdn_selective_step.restype = _i
    lib.gdn_selective_step.argtypes = [_vp] * 11 + [_i] * 4 + [_vp]
    _lib = lib
    return lib


def status_string(code: int) -> str:
    return load().gdn_status_string(code).decode()


def _check(code: int, what: str):
    if code != 0:
        raise RuntimeError(f"{what} failed: {status_string(code)} (status {code})")


_torch_module = None


def _torch():
    global _torch_module
    if _torch_module is None:
        import torch
        _torch_module = torch
    return _torch_module


def _dtype_code(t):
    torch = _torch()
    if t.dtype == torch.bfloat16:
        return GDN_BF16
    if t.dtype == torch.float32:
        return GDN_F32
    raise TypeError(f"q/k/v must be bfloat16 or float32, got {t.dtype}")


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _need(t, name, shape, dtype, device):
    if t is not None and t.dtype is dtype and t.shape == shape and t.device == device and t.is_contiguous():
        return
    if t is None:
        raise ValueError(f"{name} is required")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name}: expected device {device}, got {t.device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _stream(device):
    torch = _torch()
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _workspace(nbytes, device):
    torch = _torch()
    ws = torch.empty(max(int(nbytes), 256) + 256, dtype=torch.uint8, device=device)
    off = (-ws.data_ptr()) % 256
    return ws, ws[off:off + max(int(nbytes), 256)]


def gdn_chunk_fwd_workspace(B, T, H, Dk, Dv, dtype_code):
    return int(load().gdn_chunk_fwd_workspace(B, T, H, Dk, Dv, dtype_code))


def gdn2_chunk_fwd_workspace(B, T, H, Dk, Dv, dtype_code):
    return int(load().gdn2_chunk_fwd_workspace(B, T, H, Dk, Dv, dtype_code))


def gdn_chunk_fwd(q, k, v, g, beta, h0=None, scale=None, output_final_state=True, workspace=None,
                  out=None, final_state=None):
    """Chunked Gated DeltaNet forward.  q, k [B,T,H,Dk], v [B,T,H,Dv] (bf16 or fp32),
    g, beta [B,T,H] fp32, h0 [B,H,Dk,Dv] fp32 or None.  Returns (o fp32, ht or None)."""
    torch = _torch()
    B, T, H, Dk = q.shape
    Dv = v.shape[-1]
    dev = q.device
    dt = _dtype_code(q)
    _need(q, "q", (B, T, H, Dk), q.dtype, dev)
    _need(k, "k", (B, T, H, Dk), q.dtype, dev)
    _need(v, "v", (B, T, H, Dv), q.dtype, dev)
    _need(g, "g", (B, T, H), torch.float32, dev)
    _need(beta, "beta", (B, T, H), torch.float32, dev)
    if h0 is not None:
        _need(h0, "h0", (B, H, Dk, Dv), torch.float32, dev)
    if scale is None:
        scale = Dk ** -0.5
    o = out if out is not None else torch.empty((B, T, H, Dv), dtype=torch.float32, device=dev)
    _need(o, "out", (B, T, H, Dv), torch.float32, dev)
    ht = None
    if output_final_state:
        ht = final_state if final_state is not None else torch.empty((B, H, Dk, Dv), dtype=torch.float32,
                                                                     device=dev)
        _need(ht, "final_state", (B, H, Dk, Dv), torch.float32, dev)
    lib = load()
    need = lib.gdn_chunk_fwd_workspace(B, T, H, Dk, Dv, dt)
    if need == 0:
        _check(2, "gdn_chunk_fwd_workspace")
    if workspace is None:
        _, ws = _workspace(need, dev)
    else:
        ws = workspace
    _check(lib.gdn_chunk_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(h0), _ptr(o), _ptr(ht),
                             B, T, H, Dk, Dv, dt, float(scale), _ptr(ws), ws.numel() * ws.element_size(),
                             _stream(dev)), "gdn_chunk_fwd")
    return o, ht


def gdn_chunk_fwd_varlen(q, k, v, g, beta, cu_seqlens, h0=None, scale=None, output_final_state=True):
    """Chunked forward over packed variable-length sequences.  q, k [total_T,H,Dk] and
    v [total_T,H,Dv] bf16 (a leading batch dim of 1 is accepted), g, beta [total_T,H]
    fp32, cu_seqlens int32 [N+1] on the device, h0 [N,H,Dk,Dv] fp32 or None.
    Returns (o [total_T,H,Dv] fp32, ht [N,H,Dk,Dv] or None)."""
    torch = _torch()
    if q.dim() == 4:
        q, k, v, g, beta = q[0], k[0], v[0], g[0], beta[0]
    total_T, H, Dk = q.shape
    Dv = v.shape[-1]
    dev = q.device
    N = cu_seqlens.numel() - 1
    dt = _dtype_code(q)
    _need(q, "q", (total_T, H, Dk), q.dtype, dev)
    _need(k, "k", (total_T, H, Dk), q.dtype, dev)
    _need(v, "v", (total_T, H, Dv), q.dtype, dev)
    _need(g, "g", (total_T, H), torch.float32, dev)
    _need(beta, "beta", (total_T, H), torch.float32, dev)
    _need(cu_seqlens, "cu_seqlens", (N + 1,), torch.int32, dev)
    if h0 is not None:
        _need(h0, "h0", (N, H, Dk, Dv), torch.float32, dev)
    if scale is None:
        scale = Dk ** -0.5
    o = torch.empty((total_T, H, Dv), dtype=torch.float32, device=dev)
    ht = torch.empty((N, H, Dk, Dv), dtype=torch.float32, device=dev) if output_final_state else None
    _check(load().gdn_chunk_fwd_varlen(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(cu_seqlens), _ptr(h0),
                                       _ptr(o), _ptr(ht), N, total_T, H, Dk, Dv, dt, float(scale), _stream(dev)),
           "gdn_chunk_fwd_varlen")
    return o, ht


def gdn2_chunk_fwd_varlen_workspace(N, total_T, H, Dk, Dv, dtype_code):
    return load().gdn2_chunk_fwd_varlen_workspace(N, total_T, H, Dk, Dv, dtype_code)


def gdn2_chunk_fwd_varlen(q, k, v, log_alpha, b, w, cu_seqlens, h0=None, scale=None, output_final_state=True,
                          workspace=None):
    """Gated DeltaNet-2 forward over packed variable-length sequences.  q, k, b
    [total_T,H,Dk] and v, w [total_T,H,Dv] bf16 (a leading batch dim of 1 is accepted),
    log_alpha [total_T,H,Dk] fp32, cu_seqlens int32 [N+1] on the device, h0 [N,H,Dk,Dv]
    fp32 or None.  Returns (o [total_T,H,Dv] fp32, ht [N,H,Dk,Dv] or None)."""
    torch = _torch()
    if q.dim() == 4:
        q, k, v, log_alpha, b, w = q[0], k[0], v[0], log_alpha[0], b[0], w[0]
    total_T, H, Dk = q.shape
    Dv = v.shape[-1]
    dev = q.device
    N = cu_seqlens.numel() - 1
    dt = _dtype_code(q)
    for t, name, d in ((q, "q", Dk), (k, "k", Dk), (v, "v", Dv), (b, "b", Dk), (w, "w", Dv)):
        _need(t, name, (total_T, H, d), q.dtype, dev)
    _need(log_alpha, "log_alpha", (total_T, H, Dk), torch.float32, dev)
    _need(cu_seqlens, "cu_seqlens", (N + 1,), torch.int32, dev)
    if h0 is not None:
        _need(h0, "h0", (N, H, Dk, Dv), torch.float32, dev)
    if scale is None:
        scale = Dk ** -0.5
    o = torch.empty((total_T, H, Dv), dtype=torch.float32, device=dev)
    ht = torch.empty((N, H, Dk, Dv), dtype=torch.float32, device=dev) if output_final_state else None
    lib = load()
    need = lib.gdn2_chunk_fwd_varlen_workspace(N, total_T, H, Dk, Dv, dt)
    if need == 0:
        _check(2, "gdn2_chunk_fwd_varlen_workspace")
    ws = workspace if workspace is not None else _workspace(need, dev)[1]
    _check(lib.gdn2_chunk_fwd_varlen(_ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(b), _ptr(w),
                                     _ptr(cu_seqlens), _ptr(h0), _ptr(o), _ptr(ht), N, total_T, H, Dk, Dv, dt,
                                     float(scale), _ptr(ws), ws.numel() * ws.element_size(), _stream(dev)),
           "gdn2_chunk_fwd_varlen")
    return o, ht


def gdn_chunk_bwd_workspace(B, T, H, Dk, Dv, dtype_code):
    return int(load().gdn_chunk_bwd_workspace(B, T, H, Dk, Dv, dtype_code))


def gdn_chunk_bwd(q, k, v, g, beta, h0, do, dht=None, scale=None, workspace=None):
    """Backward of gdn_chunk_fwd: gradients of sum(do * o) + sum(dht * ht).
    Inputs as gdn_chunk_fwd (h0 may be None), do [B,T,H,Dv] fp32, dht [B,H,Dk,Dv]
    fp32 or None.  Returns (dq, dk, dv, dg, dbeta, dh0) fp32; dh0 is None when h0 is."""
    torch = _torch()
    B, T, H, Dk = q.shape
    Dv = v.shape[-1]
    dev = q.device
    dt = _dtype_code(q)
    _need(q, "q", (B, T, H, Dk), q.dtype, dev)
    _need(k, "k", (B, T, H, Dk), q.dtype, dev)
    _need(v, "v", (B, T, H, Dv), q.dtype, dev)
    _need(g, "g", (B, T, H), torch.float32, dev)
    _need(beta, "beta", (B, T, H), torch.float32, dev)
    _need(do, "do", (B, T, H, Dv), torch.float32, dev)
    if h0 is not None:
        _need(h0, "h0", (B, H, Dk, Dv), torch.float32, dev)
    if dht is not None:
        _need(dht, "dht", (B, H, Dk, Dv), torch.float32, dev)
    if scale is None:
        scale = Dk ** -0.5
    f32 = dict(dtype=torch.float32, device=dev)
    dq = torch.empty((B, T, H, Dk), **f32)
    dk = torch.empty((B, T, H, Dk), **f32)
    dv = torch.empty((B, T, H, Dv), **f32)
    dg = torch.empty((B, T, H), **f32)
    dbeta = torch.empty((B, T, H), **f32)
    dh0 = torch.empty((B, H, Dk, Dv), **f32) if h0 is not None else None
    lib = load()
    need = lib.gdn_chunk_bwd_workspace(B, T, H, Dk, Dv, dt)
    if need == 0:
        _check(2, "gdn_chunk_bwd_workspace")
    ws = workspace if workspace is not None else _workspace(need, dev)[1]
    _check(lib.gdn_chunk_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(h0), _ptr(do), _ptr(dht),
                             _ptr(dq), _ptr(dk), _ptr(dv), _ptr(dg), _ptr(dbeta), _ptr(dh0), B, T, H, Dk, Dv, dt,
                             float(scale), _ptr(ws), ws.numel() * ws.element_size(), _stream(dev)), "gdn_chunk_bwd")
    return dq, dk, dv, dg, dbeta, dh0


def gdn2_chunk_bwd_workspace(B, T, H, Dk, Dv, dtype_code):
    return int(load().gdn2_chunk_bwd_workspace(B, T, H, Dk, Dv, dtype_code))


def gdn2_chunk_bwd(q, k, v, log_alpha, b, w, h0, do, dht=None, scale=None, workspace=None):
    """Backward of gdn2_chunk_fwd.  Inputs as gdn2_chunk_fwd (h0 may be None), do
    [B,T,H,Dv] fp32, dht [B,H,Dk,Dv] fp32 or None.  Returns (dq, dk, dv, dlog_alpha,
    db, dw, dh0) in fp32 (dh0 None when h0 is None)."""
    torch = _torch()
    B, T, H, Dk = q.shape
    Dv = v.shape[-1]
    dev = q.device
    dt = _dtype_code(q)
    _need(q, "q", (B, T, H, Dk), q.dtype, dev)
    _need(k, "k", (B, T, H, Dk), q.dtype, dev)
    _need(v, "v", (B, T, H, Dv), q.dtype, dev)
    _need(log_alpha, "log_alpha", (B, T, H, Dk), torch.float32, dev)
    _need(b, "b", (B, T, H, Dk), q.dtype, dev)
    _need(w, "w", (B, T, H, Dv), q.dtype, dev)
    _need(do, "do", (B, T, H, Dv), torch.float32, dev)
    if h0 is not None:
        _need(h0, "h0", (B, H, Dk, Dv), torch.float32, dev)
    if dht is not None:
        _need(dht, "dht", (B, H, Dk, Dv), torch.float32, dev)
    if scale is None:
        scale = Dk ** -0.5
    f32 = torch.float32
    dq = torch.empty((B, T, H, Dk), dtype=f32, device=dev)
    dk = torch.empty((B, T, H, Dk), dtype=f32, device=dev)
    dla = torch.empty((B, T, H, Dk), dtype=f32, device=dev)
    db = torch.empty((B, T, H, Dk), dtype=f32, device=dev)
    dv = torch.empty((B, T, H, Dv), dtype=f32, device=dev)
    dw = torch.empty((B, T, H, Dv), dtype=f32, device=dev)
    dh0 = torch.empty((B, H, Dk, Dv), dtype=f32, device=dev) if h0 is not None else None
    nbytes = gdn2_chunk_bwd_workspace(B, T, H, Dk, Dv, dt)
    if workspace is None:
        _hold, ws = _workspace(nbytes, dev)
    else:
        ws = workspace
    _check(load().gdn2_chunk_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(b), _ptr(w), _ptr(h0), _ptr(do),
                                 _ptr(dht), _ptr(dq), _ptr(dk), _ptr(dv), _ptr(dla), _ptr(db), _ptr(dw), _ptr(dh0),
                                 B, T, H, Dk, Dv, dt, float(scale), _ptr(ws), ws.numel(), _stream(dev)),
           "gdn2_chunk_bwd")
    return dq, dk, dv, dla, db, dw, dh0


def gdn_chunk_intra(k, g, beta, G2_out=None, Tinv_out=None):
    """State-independent chunk stage: returns (G2 [B,H,NT,64], Tinv [B,H,NT,64,64]) fp32,
    Tinv = (I + A)^-1 - I per chunk.  Preallocated outputs may be passed in."""
    torch = _torch()
    B, T, H, Dk = k.shape
    dev = k.device
    dt = _dtype_code(k)
    _need(k, "k", (B, T, H, Dk), k.dtype, dev)
    _need(g, "g", (B, T, H), torch.float32, dev)
    _need(beta, "beta", (B, T, H), torch.float32, dev)
    NT = (T + BT - 1) // BT
    G2 = G2_out if G2_out is not None else torch.empty((B, H, NT, BT), dtype=torch.float32, device=dev)
    Tinv = Tinv_out if Tinv_out is not None else torch.empty((B, H, NT, BT, BT), dtype=torch.float32, device=dev)
    _need(G2, "G2_out", (B, H, NT, BT), torch.float32, dev)
    _need(Tinv, "Tinv_out", (B, H, NT, BT, BT), torch.float32, dev)
    _check(load().gdn_chunk_intra(_ptr(k), _ptr(g), _ptr(beta), _ptr(G2), _ptr(Tinv), B, T, H, Dk, dt,
                                  _stream(dev)), "gdn_chunk_intra")
    return G2, Tinv


def gdn_chunk_walk(q, k, v, beta, G2, Tinv, h0=None, scale=None, output_final_state=True, out=None,
                   final_state=None):
    """Sequential stage of the chunked forward on the outputs of gdn_chunk_intra.
    Returns (o fp32, ht or None)."""
    torch = _torch()
    B, T, H, Dk = q.shape
    Dv = v.shape[-1]
    dev = q.device
    dt = _dtype_code(q)
    NT = (T + BT - 1) // BT
    _need(q, "q", (B, T, H, Dk), q.dtype, dev)
    _need(k, "k", (B, T, H, Dk), q.dtype, dev)
    _need(v, "v", (B, T, H, Dv), q.dtype, dev)
    _need(beta, "beta", (B, T, H), torch.float32, dev)
    _need(G2, "G2", (B, H, NT, BT), torch.float32, dev)
    _need(Tinv, "Tinv", (B, H, NT, BT, BT), torch.float32, dev)
    if h0 is not None:
        _need(h0, "h0", (B, H, Dk, Dv), torch.float32, dev)
    if scale is None:
        scale = Dk ** -0.5
    o = out if out is not None else torch.empty((B, T, H, Dv), dtype=torch.float32, device=dev)
    _need(o, "out", (B, T, H, Dv), torch.float32, dev)
    ht = None
    if output_final_state:
        ht = final_state if final_state is not None else torch.empty((B, H, Dk, Dv), dtype=torch.float32,
                                                                     device=dev)
        _need(ht, "final_state", (B, H, Dk, Dv), torch.float32, dev)
    _check(load().gdn_chunk_walk(_ptr(q), _ptr(k), _ptr(v), _ptr(beta), _ptr(G2), _ptr(Tinv), _ptr(h0), _ptr(o),
                                 _ptr(ht), B, T, H, Dk, Dv, dt, float(scale), _stream(dev)), "gdn_chunk_walk")
    return o, ht


def gdn2_chunk_fwd(q, k, v, log_alpha, b, w, h0=None, scale=None, output_final_state=True, workspace=None,
                   out=None, final_state=None):
    """Chunked Gated DeltaNet-2 forward.  log_alpha [B,T,H,Dk] fp32; b [B,T,H,Dk] and
    w [B,T,H,Dv] in the dtype of q.  Returns (o fp32, ht or None)."""
    torch = _torch()
    B, T, H, Dk = q.shape
    Dv = v.shape[-1]
    dev = q.device
    dt = _dtype_code(q)
    _need(q, "q", (B, T, H, Dk), q.dtype, dev)
    _need(k, "k", (B, T, H, Dk), q.dtype, dev)
    _need(v, "v", (B, T, H, Dv), q.dtype, dev)
    _need(log_alpha, "log_alpha", (B, T, H, Dk), torch.float32, dev)
    _need(b, "b", (B, T, H, Dk), q.dtype, dev)
    _need(w, "w", (B, T, H, Dv), q.dtype, dev)
    if h0 is not None:
        _need(h0, "h0", (B, H, Dk, Dv), torch.float32, dev)
    if scale is None:
        scale = Dk ** -0.5
    o = out if out is not None else torch.empty((B, T, H, Dv), dtype=torch.float32, device=dev)
    _need(o, "out", (B, T, H, Dv), torch.float32, dev)
    ht = None
    if output_final_state:
        ht = final_state if final_state is not None else torch.empty((B, H, Dk, Dv), dtype=torch.float32,
                                                                     device=dev)
        _need(ht, "final_state", (B, H, Dk, Dv), torch.float32, dev)
    lib = load()
    need = lib.gdn2_chunk_fwd_workspace(B, T, H, Dk, Dv, dt)
    if need == 0:
        _check(2, "gdn2_chunk_fwd_workspace")
    if workspace is None:
        _, ws = _workspace(need, dev)
    else:
        ws = workspace
    _check(lib.gdn2_chunk_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(b), _ptr(w), _ptr(h0), _ptr(o),
                              _ptr(ht), B, T, H, Dk, Dv, dt, float(scale), _ptr(ws),
                              ws.numel() * ws.element_size(), _stream(dev)), "gdn2_chunk_fwd")
    return o, ht


def gdn2_chunk_fwd_noalloc_max_bytes() -> int:
    """Size of the library's fixed device workspace used by gdn2_chunk_fwd_noalloc."""
    return int(load().gdn2_chunk_fwd_noalloc_max_bytes())


def gdn2_chunk_fwd_noalloc(q, k, v, log_alpha, b, w, h0=None, scale=None, out=None, final_state=None):
    """gdn2_chunk_fwd through the entry point that takes its workspace from the
    library's fixed device array instead of an argument.  `out` (and
    `final_state`, when the final state is wanted) should be preallocated by
    callers that cannot allocate; otherwise they are allocated here with torch
    (the C entry point itself allocates nothing).  Returns (o, ht or None)."""
    torch = _torch()
    B, T, H, Dk = q.shape
    Dv = v.shape[-1]
    dev = q.device
    dt = _dtype_code(q)
    _need(q, "q", (B, T, H, Dk), q.dtype, dev)
    _need(k, "k", (B, T, H, Dk), q.dtype, dev)
    _need(v, "v", (B, T, H, Dv), q.dtype, dev)
    _need(log_alpha, "log_alpha", (B, T, H, Dk), torch.float32, dev)
    _need(b, "b", (B, T, H, Dk), q.dtype, dev)
    _need(w, "w", (B, T, H, Dv), q.dtype, dev)
    if h0 is not None:
        _need(h0, "h0", (B, H, Dk, Dv), torch.float32, dev)
    if scale is None:
        scale = Dk ** -0.5
    o = out if out is not None else torch.empty((B, T, H, Dv), dtype=torch.float32, device=dev)
    _need(o, "out", (B, T, H, Dv), torch.float32, dev)
    ht = final_state
    if ht is not None:
        _need(ht, "final_state", (B, H, Dk, Dv), torch.float32, dev)
    _check(load().gdn2_chunk_fwd_noalloc(_ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(b), _ptr(w), _ptr(h0),
                                         _ptr(o), _ptr(ht), B, T, H, Dk, Dv, dt, float(scale), _stream(dev)),
           "gdn2_chunk_fwd_noalloc")
    return o, ht


def gdn_recurrent_step(q, k, v, g, beta, S, scale=None, out=None):
    """One decode token: q, k [B,H,Dk], v [B,H,Dv], g, beta [B,H] fp32, S [B,H,Dk,Dv] fp32
    updated in place.  Returns o [B,H,Dv] fp32."""
    torch = _torch()
    B, H, Dk = q.shape
    Dv = v.shape[-1]
    dev = q.device
    dt = _dtype_code(q)
    _need(q, "q", (B, H, Dk), q.dtype, dev)
    _need(k, "k", (B, H, Dk), q.dtype, dev)
    _need(v, "v", (B, H, Dv), q.dtype, dev)
    _need(g, "g", (B, H), torch.float32, dev)
    _need(beta, "beta", (B, H), torch.float32, dev)
    _need(S, "S", (B, H, Dk, Dv), torch.float32, dev)
    if scale is None:
        scale = Dk ** -0.5
    o = out if out is not None else torch.empty((B, H, Dv), dtype=torch.float32, device=dev)
    _need(o, "out", (B, H, Dv), torch.float32, dev)
    _check(load().gdn_recurrent_step(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(S), _ptr(o),
                                     B, H, Dk, Dv, dt, float(scale), _stream(dev)), "gdn_recurrent_step")
    return o


def gdn2_recurrent_step(q, k, v, log_alpha, b, w, S, scale=None, out=None):
    """One GDN-2 decode token: q, k, b [B,H,Dk] and v, w [B,H,Dv] in the path dtype,
    log_alpha [B,H,Dk] fp32, S [B,H,Dk,Dv] fp32 updated in place.  Returns o [B,H,Dv] fp32."""
    torch = _torch()
    B, H, Dk = q.shape
    Dv = v.shape[-1]
    dev = q.device
    dt = _dtype_code(q)
    _need(q, "q", (B, H, Dk), q.dtype, dev)
    _need(k, "k", (B, H, Dk), q.dtype, dev)
    _need(v, "v", (B, H, Dv), q.dtype, dev)
    _need(log_alpha, "log_alpha", (B, H, Dk), torch.float32, dev)
    _need(b, "b", (B, H, Dk), q.dtype, dev)
    _need(w, "w", (B, H, Dv), q.dtype, dev)
    _need(S, "S", (B, H, Dk, Dv), torch.float32, dev)
    if scale is None:
        scale = Dk ** -0.5
    o = out if out is not None else torch.empty((B, H, Dv), dtype=torch.float32, device=dev)
    _need(o, "out", (B, H, Dv), torch.float32, dev)
    _check(load().gdn2_recurrent_step(_ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(b), _ptr(w), _ptr(S),
                                      _ptr(o), B, H, Dk, Dv, dt, float(scale), _stream(dev)), "gdn2_recurrent_step")
    return o


def gdn_prologue(xq, xk, xv, a, b, wq, wk, wv, A_log, dt_bias, conv_state=None, update_conv_state=False):
    """Short convolution, SiLU, q/k L2 norm and gates in one pass.  xq, xk [B,T,H,Dk] and
    xv [B,T,H,Dv] bf16; a, b [B,T,H] fp32; wq, wk [H*Dk,4], wv [H*Dv,4], A_log, dt_bias [H]
    fp32; conv_state [B,3,H*(2Dk+Dv)] fp32 or None.  Returns (q, k, v bf16, g, beta fp32,
    new conv state or None); with update_conv_state the new state overwrites conv_state."""
    torch = _torch()
    B, T, H, Dk = xq.shape
    Dv = xv.shape[-1]
    dev = xq.device
    bf, f32 = torch.bfloat16, torch.float32
    _need(xq, "xq", (B, T, H, Dk), bf, dev)
    _need(xk, "xk", (B, T, H, Dk), bf, dev)
    _need(xv, "xv", (B, T, H, Dv), bf, dev)
    _need(a, "a", (B, T, H), f32, dev)
    _need(b, "b", (B, T, H), f32, dev)
    _need(wq, "wq", (H * Dk, 4), f32, dev)
    _need(wk, "wk", (H * Dk, 4), f32, dev)
    _need(wv, "wv", (H * Dv, 4), f32, dev)
    _need(A_log, "A_log", (H,), f32, dev)
    _need(dt_bias, "dt_bias", (H,), f32, dev)
    C = H * (2 * Dk + Dv)
    if conv_state is not None:
        _need(conv_state, "conv_state", (B, 3, C), f32, dev)
    if update_conv_state:
        if conv_state is None:
            raise ValueError("update_conv_state needs conv_state")
        new_state = conv_state
    else:
        new_state = torch.empty((B, 3, C), dtype=f32, device=dev)
    q = torch.empty((B, T, H, Dk), dtype=bf, device=dev)
    k = torch.empty((B, T, H, Dk), dtype=bf, device=dev)
    v = torch.empty((B, T, H, Dv), dtype=bf, device=dev)
    g = torch.empty((B, T, H), dtype=f32, device=dev)
    beta = torch.empty((B, T, H), dtype=f32, device=dev)
    _check(load().gdn_prologue(_ptr(xq), _ptr(xk), _ptr(xv), _ptr(a), _ptr(b), _ptr(wq), _ptr(wk), _ptr(wv),
                               _ptr(A_log), _ptr(dt_bias), _ptr(conv_state), _ptr(q), _ptr(k), _ptr(v), _ptr(g),
                               _ptr(beta), _ptr(new_state), B, T, H, Dk, Dv, _stream(dev)), "gdn_prologue")
    return q, k, v, g, beta, new_state


def gdn_gated_rmsnorm(o, z, weight, eps=1e-5, out=None):
    """y = o / sqrt(mean(o^2) + eps) * weight * SiLU(z) over the last axis.  o [..., Dv]
    fp32, z [..., Dv] bf16, weight [Dv] fp32.  Returns y [..., Dv] bf16."""
    torch = _torch()
    Dv = o.shape[-1]
    dev = o.device
    _need(o, "o", tuple(o.shape), torch.float32, dev)
    _need(z, "z", tuple(o.shape), torch.bfloat16, dev)
    _need(weight, "weight", (Dv,), torch.float32, dev)
    y = out if out is not None else torch.empty(o.shape, dtype=torch.bfloat16, device=dev)
    _need(y, "out", tuple(o.shape), torch.bfloat16, dev)
    rows = o.numel() // Dv
    _check(load().gdn_gated_rmsnorm(_ptr(o), _ptr(z), _ptr(weight), _ptr(y), rows, Dv, float(eps), _stream(dev)),
           "gdn_gated_rmsnorm")
    return y


_CODES = {}


def _code(t, name):
    if not _CODES:
        torch = _torch()
        _CODES.update({torch.float32: GDN_F32, torch.bfloat16: GDN_BF16, torch.float8_e4m3fn: GDN_F8E4M3})
    code = _CODES.get(t)
    if code is None:
        raise TypeError(f"{name} must be float32, bfloat16 or float8_e4m3fn, got {t}")
    return code


def _addr(t):
    return None if t is None else t.data_ptr()


def _scratch(nbytes, device):
    """nbytes of 256-byte aligned workspace (torch's allocations are; a slice otherwise)."""
    ws = _torch().empty(nbytes, dtype=_torch().uint8, device=device)
    return ws if ws.data_ptr() % 256 == 0 else _workspace(nbytes, device)[1]


def _given(ws, dev):
    """Size in bytes of a workspace that the caller hands in."""
    if ws.device != dev or not ws.is_contiguous():
        raise ValueError(f"workspace must be contiguous on {dev}, got {ws.device}")
    return ws.numel() * ws.element_size()


_current = None


def _current_device_and_stream():
    """(current device index, handle of the current stream of a device index), the short way where this torch has it
    (0.1 us a call against 2.1)."""
    global _current
    if _current is None:
        torch = _torch()
        torch.cuda.init()
        dev = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
        stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        _current = dev, stream or (lambda i: torch.cuda.current_stream(i).cuda_stream)
    return _current


def _on_device(fn, what, dev, *args):
    """Calls fn(*args, stream) with dev as the current device, on its current stream."""
    if dev.type != "cuda":
        raise ValueError(f"{what}: tensors must be on the GPU, got {dev}")
    current, stream = _current or _current_device_and_stream()
    index = dev.index
    if current() == index:
        code = fn(*args, stream(index))
    else:
        with _torch().cuda.device(dev):
            code = fn(*args, stream(index))
    if code:
        _check(code, what)


def gdn_add_rmsnorm(x, weight, residual=None, eps=1e-5, out_dtype=None, return_rstd=False, out=None,
                    residual_out=None):
    """Residual addition and RMS norm over the last axis: u = x + residual, y = u / sqrt(mean(u^2) + eps) * weight.
    x [..., D] bf16 or fp32, weight [D] fp32, residual [..., D] in the type of x or fp32, or None.  out_dtype: the
    type of x (default) or torch.float8_e4m3fn, with one fp32 scale per row.  residual_out may be residual itself (in
    place).  Returns (y, r, rstd, y_scale): r = u in the type of residual (None without one), rstd [rows] when
    return_rstd, y_scale [rows] for 8-bit y, None otherwise."""
    torch = _torch()
    shape, dev, f32 = tuple(x.shape), x.device, torch.float32
    if not shape:
        raise ValueError("x must have at least one axis")
    D = shape[-1]
    rows = x.numel() // D if D else 0
    _need(x, "x", shape, x.dtype, dev)
    _need(weight, "weight", (D,), f32, dev)
    rdt = x.dtype
    r = None
    if residual is not None:
        rdt = residual.dtype
        _need(residual, "residual", shape, rdt, dev)
        r = residual_out if residual_out is not None else torch.empty_like(residual)
        if r is residual_out:
            _need(r, "residual_out", shape, rdt, dev)
    elif residual_out is not None:
        raise ValueError("residual_out needs residual")
    odt = x.dtype if out_dtype is None else out_dtype
    y = torch.empty_like(x, dtype=odt) if out is None else out
    if out is not None:
        _need(y, "out", shape, odt, dev)
    rstd = torch.empty(shape[:-1], dtype=f32, device=dev) if return_rstd else None
    y_scale = torch.empty(shape[:-1], dtype=f32, device=dev) if odt == torch.float8_e4m3fn else None
    _on_device(load().gdn_add_rmsnorm, "gdn_add_rmsnorm", dev,
               _addr(x), _addr(residual), _addr(weight), _addr(y), _addr(r), _addr(rstd), _addr(y_scale), rows, D,
               _code(x.dtype, "x"), _code(rdt, "residual"), _code(odt, "out_dtype"), float(eps))
    return y, r, rstd, y_scale


def gdn_add_rmsnorm_bwd_workspace(rows, D):
    return int(load().gdn_add_rmsnorm_bwd_workspace(rows, D))


def gdn_add_rmsnorm_bwd(dy, r, weight, rstd, dr=None, need_dweight=True, workspace=None):
    """Gradients of gdn_add_rmsnorm.  dy [..., D] bf16 or fp32; r [..., D]: what the forward returned (x when it had
    no residual); rstd [...] fp32; dr [..., D]: gradient that reaches r from elsewhere, or None.  Returns (dx in the
    type of r: the gradient of x and of residual alike, dweight [D] fp32 or None)."""
    torch = _torch()
    shape, dev, f32 = tuple(dy.shape), dy.device, torch.float32
    if not shape:
        raise ValueError("dy must have at least one axis")
    D = shape[-1]
    rows = dy.numel() // D if D else 0
    _need(dy, "dy", shape, dy.dtype, dev)
    _need(r, "r", shape, r.dtype, dev)
    _need(weight, "weight", (D,), f32, dev)
    _need(rstd, "rstd", shape[:-1], f32, dev)
    if dr is not None:
        _need(dr, "dr", shape, r.dtype, dev)
    dx = torch.empty_like(r)
    dw = ws = None
    nbytes = 0
    lib = load()
    if need_dweight:
        dw = torch.empty((D,), dtype=f32, device=dev)
        if workspace is None:
            nbytes = lib.gdn_add_rmsnorm_bwd_workspace(rows, D)
            ws = _scratch(nbytes, dev)
        else:
            ws, nbytes = workspace, _given(workspace, dev)
    _on_device(lib.gdn_add_rmsnorm_bwd, "gdn_add_rmsnorm_bwd", dev,
               _addr(dy), _addr(r), _addr(weight), _addr(rstd), _addr(dr), _addr(dx), _addr(dw), rows, D,
               _code(dy.dtype, "dy"), _code(r.dtype, "r"), _addr(ws), nbytes)
    return dx, dw


def gdn_add_layernorm(x, weight, bias=None, residual=None, eps=1e-5, out_dtype=None, return_stats=False, out=None,
                      residual_out=None):
    """Residual addition and layer norm over the last axis: u = x + residual,
    y = (u - mean(u)) / sqrt(var(u) + eps) * weight + bias.  bias [D] fp32 or None; the other arguments as
    gdn_add_rmsnorm.  Returns (y, r, mean, rstd, y_scale): r = u in the type of residual (None without one), mean and
    rstd [rows] when return_stats, y_scale [rows] for 8-bit y, None otherwise."""
    torch = _torch()
    shape, dev, f32 = tuple(x.shape), x.device, torch.float32
    if not shape:
        raise ValueError("x must have at least one axis")
    D = shape[-1]
    rows = x.numel() // D if D else 0
    _need(x, "x", shape, x.dtype, dev)
    _need(weight, "weight", (D,), f32, dev)
    if bias is not None:
        _need(bias, "bias", (D,), f32, dev)
    rdt = x.dtype
    r = None
    if residual is not None:
        rdt = residual.dtype
        _need(residual, "residual", shape, rdt, dev)
        r = residual_out if residual_out is not None else torch.empty_like(residual)
        if r is residual_out:
            _need(r, "residual_out", shape, rdt, dev)
    elif residual_out is not None:
        raise ValueError("residual_out needs residual")
    odt = x.dtype if out_dtype is None else out_dtype
    y = torch.empty_like(x, dtype=odt) if out is None else out
    if out is not None:
        _need(y, "out", shape, odt, dev)
    mean = torch.empty(shape[:-1], dtype=f32, device=dev) if return_stats else None
    rstd = torch.empty_like(mean) if return_stats else None
    y_scale = torch.empty(shape[:-1], dtype=f32, device=dev) if odt == torch.float8_e4m3fn else None
    _on_device(load().gdn_add_layernorm, "gdn_add_layernorm", dev,
               _addr(x), _addr(residual), _addr(weight), _addr(bias), _addr(y), _addr(r), _addr(mean), _addr(rstd),
               _addr(y_scale), rows, D, _code(x.dtype, "x"), _code(rdt, "residual"), _code(odt, "out_dtype"),
               float(eps))
    return y, r, mean, rstd, y_scale


def gdn_add_layernorm_bwd_workspace(rows, D):
    return int(load().gdn_add_layernorm_bwd_workspace(rows, D))


def gdn_add_layernorm_bwd(dy, r, weight, mean, rstd, dr=None, need_dweight=True, need_dbias=True, workspace=None):
    """Gradients of gdn_add_layernorm.  dy [..., D] bf16 or fp32; r [..., D]: what the forward returned (x when it had
    no residual); mean, rstd [...] fp32; dr [..., D]: gradient that reaches r from elsewhere, or None.  Returns (dx in
    the type of r: the gradient of x and of residual alike, dweight, dbias [D] fp32 or None)."""
    torch = _torch()
    shape, dev, f32 = tuple(dy.shape), dy.device, torch.float32
    if not shape:
        raise ValueError("dy must have at least one axis")
    D = shape[-1]
    rows = dy.numel() // D if D else 0
    _need(dy, "dy", shape, dy.dtype, dev)
    _need(r, "r", shape, r.dtype, dev)
    _need(weight, "weight", (D,), f32, dev)
    _need(mean, "mean", shape[:-1], f32, dev)
    _need(rstd, "rstd", shape[:-1], f32, dev)
    if dr is not None:
        _need(dr, "dr", shape, r.dtype, dev)
    dx = torch.empty_like(r)
    dw = torch.empty_like(weight) if need_dweight else None
    db = torch.empty_like(weight) if need_dbias else None
    ws, nbytes = None, 0
    lib = load()
    if need_dweight or need_dbias:
        if workspace is None:
            nbytes = lib.gdn_add_layernorm_bwd_workspace(rows, D)
            ws = _scratch(nbytes, dev)
        else:
            ws, nbytes = workspace, _given(workspace, dev)
    _on_device(lib.gdn_add_layernorm_bwd, "gdn_add_layernorm_bwd", dev,
               _addr(dy), _addr(r), _addr(weight), _addr(mean), _addr(rstd), _addr(dr), _addr(dx), _addr(dw), _addr(db),
               rows, D, _code(dy.dtype, "dy"), _code(r.dtype, "r"), _addr(ws), nbytes)
    return dx, dw, db


def gdn_quantize_rows(x):
    """Rows of x [..., D] (bf16 or fp32) in 8 bits: (q float8_e4m3fn [..., D], scale [...] fp32) with
    scale = max|x| / 448 (1 for a row of zeros) and q = x / scale."""
    torch = _torch()
    shape, dev = tuple(x.shape), x.device
    if not shape:
        raise ValueError("x must have at least one axis")
    D = shape[-1]
    _need(x, "x", shape, x.dtype, dev)
    q = torch.empty_like(x, dtype=torch.float8_e4m3fn)
    scale = torch.empty(shape[:-1], dtype=torch.float32, device=dev)
    _on_device(load().gdn_quantize_rows, "gdn_quantize_rows", dev,
               _addr(x), _addr(q), _addr(scale), x.numel() // D if D else 0, D, _code(x.dtype, "x"))
    return q, scale


_ACTS = {"none": 0, "relu": 1, "silu": 2, "gelu": 3}


def _act_code(act):
    code = _ACTS.get(act)
    if code is None:
        raise ValueError(f"act must be one of {sorted(_ACTS)}, got {act!r}")
    return code


def _multiple(K, of):
    if K % of:
        raise ValueError(f"K must be a multiple of {of}, got {K}")


def gdn_linear_workspace(M, N, K, dtype_code):
    return int(load().gdn_linear_workspace(M, N, K, dtype_code))


def gdn_linear(x, weight, bias=None, residual=None, act="none", x_scale=None, w_scale=None, out_dtype=None,
               return_preact=False, workspace=None, out=None):
    """Matrix product with its epilogue: z = (x weight^T) x_scale w_scale + bias, y = act(z) + residual.
    x [..., K], weight [N, K], both bf16, or both float8_e4m3fn with x_scale [...] and w_scale [N] fp32; bias [N] fp32;
    residual [..., N] in out_dtype (bf16, the default, or fp32; out may be residual itself); act: none, relu, silu or
    gelu.  K is a multiple of 8 (16 in 8 bits).  Returns (y [..., N], z bf16 or None): z, the activation's argument,
    with return_preact."""
    torch = _torch()
    dev, dt = x.device, x.dtype
    if x.dim() < 1 or weight.dim() != 2:
        raise ValueError("x must be [..., K] and weight [N, K]")
    K, N = x.shape[-1], weight.shape[0]
    lead = tuple(x.shape[:-1])
    _need(x, "x", lead + (K,), dt, dev)
    _need(weight, "weight", (N, K), dt, dev)
    M = x.numel() // K if K else 0
    f32 = torch.float32
    if dt == torch.float8_e4m3fn:
        _need(x_scale, "x_scale", lead, f32, dev)
        _need(w_scale, "w_scale", (N,), f32, dev)
    elif x_scale is not None or w_scale is not None:
        raise ValueError("x_scale and w_scale belong to float8_e4m3fn operands")
    if bias is not None:
        _need(bias, "bias", (N,), f32, dev)
    _multiple(K, 16 if dt == torch.float8_e4m3fn else 8)
    odt = torch.bfloat16 if out_dtype is None else out_dtype
    shape = lead + (N,)
    if residual is not None:
        _need(residual, "residual", shape, odt, dev)
    y = torch.empty(shape, dtype=odt, device=dev) if out is None else out
    if out is not None:
        _need(y, "out", shape, odt, dev)
    z = torch.empty(shape, dtype=torch.bfloat16, device=dev) if return_preact else None
    lib = load()
    code, ocode = _code(dt, "x"), _code(odt, "out_dtype")
    ws = workspace
    if ws is None:
        nbytes = lib.gdn_linear_workspace(M, N, K, code)
        if nbytes:
            ws = _scratch(nbytes, dev)
    else:
        nbytes = _given(ws, dev)
    _on_device(lib.gdn_linear, "gdn_linear", dev,
               _addr(x), _addr(weight), _addr(x_scale), _addr(w_scale), _addr(bias), _addr(residual), _addr(y),
               _addr(z), M, N, K, code, ocode, _act_code(act), _addr(ws), nbytes)
    return y, z


def gdn_linear_bwd_workspace(M, N, K, dy_code, grad_code, act, need_dx=True, need_dw=True, need_dbias=False):
    return int(load().gdn_linear_bwd_workspace(M, N, K, dy_code, grad_code, _act_code(act), int(need_dx),
                                               int(need_dw), int(need_dbias)))


def gdn_linear_bwd(dy, x, weight, z=None, act="none", bias=False, grad_dtype=None, need_dx=True, need_dw=True,
                   workspace=None):
    """Gradients of gdn_linear with bf16 x [..., K] and weight [N, K]: dz = dy act'(z), dx = dz weight, dw = dz^T x,
    dbias = dz summed over rows.  dy [..., N] bf16 or fp32; z [..., N] bf16, what the forward returned with
    return_preact (required with an activation).  grad_dtype of dx and dw: bf16 (default; dz is rounded to bf16 for the
    products) or fp32 (dz is not rounded).  Returns (dx, dw, dbias fp32), None for what is not asked for; the gradient
    of residual is dy."""
    torch = _torch()
    dev, bf = dy.device, torch.bfloat16
    if x.dim() < 1 or weight.dim() != 2:
        raise ValueError("x must be [..., K] and weight [N, K]")
    K, N = x.shape[-1], weight.shape[0]
    lead = tuple(x.shape[:-1])
    _need(x, "x", lead + (K,), bf, dev)
    _need(weight, "weight", (N, K), bf, dev)
    _need(dy, "dy", lead + (N,), dy.dtype, dev)
    if z is not None and act != "none":
        _need(z, "z", lead + (N,), bf, dev)
    elif act != "none":
        raise ValueError(f"act {act!r} needs z")
    _multiple(K, 8)
    M = x.numel() // K if K else 0
    gdt = bf if grad_dtype is None else grad_dtype
    dx = torch.empty_like(x, dtype=gdt) if need_dx else None
    dw = torch.empty_like(weight, dtype=gdt) if need_dw else None
    db = torch.empty((N,), dtype=torch.float32, device=dev) if bias else None
    lib = load()
    a, dyc, gc = _act_code(act), _code(dy.dtype, "dy"), _code(gdt, "grad_dtype")
    ws = workspace
    if ws is None:
        nbytes = lib.gdn_linear_bwd_workspace(M, N, K, dyc, gc, a, int(need_dx), int(need_dw), int(bool(bias)))
        if nbytes:
            ws = _scratch(nbytes, dev)
    else:
        nbytes = _given(ws, dev)
    _on_device(lib.gdn_linear_bwd, "gdn_linear_bwd", dev,
               _addr(dy), _addr(x), _addr(weight), _addr(z) if a else None, _addr(dx), _addr(dw), _addr(db), M, N, K,
               dyc, gc, a, _addr(ws), nbytes)
    return dx, dw, db


_CUT = ("tile", "splits", "slabs", "buffers")


def gdn_linear_plan(M, N, K, dtype_code):
    """How gdn_linear cuts a product (measurement and test aid): {"tile": edge of the output tiles, 0 for the kernel
    of few rows or columns, "splits": parts of k, "slabs": slabs of 128 bytes of k in each, "buffers": of a slab}."""
    plan = (ctypes.c_int * 4)()
    _check(load().gdn_linear_plan(M, N, K, dtype_code, plan), "gdn_linear_plan")
    return dict(zip(_CUT, plan))


def gdn_linear_bwd_plan(M, N, K, dy_code, grad_code, act, need_dx=True, need_dw=True, need_dbias=False):
    """The same of gdn_linear_bwd: {"parts": bf16 parts of dz, "pair": slab buffers of the launch that dx and dw share
    or 0, "dx": and "dw": their cuts}."""
    plan = (ctypes.c_int * 10)()
    _check(load().gdn_linear_bwd_plan(M, N, K, dy_code, grad_code, _act_code(act), int(need_dx), int(need_dw),
                                      int(need_dbias), plan), "gdn_linear_bwd_plan")
    return {"parts": plan[0], "pair": plan[1], "dx": dict(zip(_CUT, plan[2:6])), "dw": dict(zip(_CUT, plan[6:10]))}


def gdn_gated_linear_workspace(M, N, K, dtype_code):
    return int(load().gdn_gated_linear_workspace(M, N, K, dtype_code))


def _halves(weight):
    if weight.dim() != 2 or weight.shape[0] % 2:
        raise ValueError(f"weight must be [2 N, K], got {tuple(weight.shape)}")
    return weight.shape[0] // 2


def gdn_gated_linear(x, weight, bias=None, act="silu", x_scale=None, w_scale=None, out_dtype=None,
                     return_preact=False, workspace=None, out=None):
    """Gated projection in one kernel: (g, u) = (x weight^T) x_scale w_scale + bias, y = act(g) u.  x [..., K], weight
    [2 N, K] (N gate rows, then N up rows), both bf16, or both float8_e4m3fn with x_scale [...] and w_scale [2 N] fp32;
    bias [2 N] fp32; act: none, relu, silu or gelu.  K is a multiple of 8 (16 in 8 bits).  Returns (y [..., N] in
    out_dtype: bf16, the default, or fp32; z [..., 2 N] bf16 or None): z, that is g and u, with return_preact."""
    torch = _torch()
    dev, dt, f32 = x.device, x.dtype, torch.float32
    if x.dim() < 1:
        raise ValueError("x must be [..., K]")
    N, K = _halves(weight), x.shape[-1]
    lead = tuple(x.shape[:-1])
    _need(x, "x", lead + (K,), dt, dev)
    _need(weight, "weight", (2 * N, K), dt, dev)
    M = x.numel() // K if K else 0
    if dt == torch.float8_e4m3fn:
        _need(x_scale, "x_scale", lead, f32, dev)
        _need(w_scale, "w_scale", (2 * N,), f32, dev)
    elif x_scale is not None or w_scale is not None:
        raise ValueError("x_scale and w_scale belong to float8_e4m3fn operands")
    if bias is not None:
        _need(bias, "bias", (2 * N,), f32, dev)
    _multiple(K, 16 if dt == torch.float8_e4m3fn else 8)
    odt = torch.bfloat16 if out_dtype is None else out_dtype
    y = torch.empty(lead + (N,), dtype=odt, device=dev) if out is None else out
    if out is not None:
        _need(y, "out", lead + (N,), odt, dev)
    z = torch.empty(lead + (2 * N,), dtype=torch.bfloat16, device=dev) if return_preact else None
    lib = load()
    code, ocode = _code(dt, "x"), _code(odt, "out_dtype")
    ws = workspace
    if ws is None:
        nbytes = lib.gdn_gated_linear_workspace(M, N, K, code)
        if nbytes:
            ws = _scratch(nbytes, dev)
    else:
        nbytes = _given(ws, dev)
    _on_device(lib.gdn_gated_linear, "gdn_gated_linear", dev,
               _addr(x), _addr(weight), _addr(x_scale), _addr(w_scale), _addr(bias), _addr(y), _addr(z), M, N, K, code,
               ocode, _act_code(act), _addr(ws), nbytes)
    return y, z


def gdn_gated_linear_bwd_workspace(M, N, K, dy_code, grad_code, act, need_dx=True, need_dw=True, need_dbias=False):
    return int(load().gdn_gated_linear_bwd_workspace(M, N, K, dy_code, grad_code, _act_code(act), int(need_dx),
                                                     int(need_dw), int(need_dbias)))


def gdn_gated_linear_bwd(dy, x, weight, z, act="silu", bias=False, grad_dtype=None, need_dx=True, need_dw=True,
                         workspace=None):
    """Gradients of gdn_gated_linear with bf16 x [..., K] and weight [2 N, K]: dg = dy u act'(g), du = dy act(g),
    dx = (dg, du) weight, dw = (dg, du)^T x, dbias = (dg, du) summed over rows.  dy [..., N] bf16 or fp32; z [..., 2 N]
    bf16: what the forward returned with return_preact.  grad_dtype of dx and dw: bf16 (default; dg and du are rounded
    to bf16 for the products) or fp32 (they are not rounded).  Returns (dx, dw [2 N, K], dbias [2 N] fp32), None for
    what is not asked for."""
    torch = _torch()
    dev, bf = dy.device, torch.bfloat16
    if x.dim() < 1:
        raise ValueError("x must be [..., K]")
    N, K = _halves(weight), x.shape[-1]
    lead = tuple(x.shape[:-1])
    _need(x, "x", lead + (K,), bf, dev)
    _need(weight, "weight", (2 * N, K), bf, dev)
    _need(dy, "dy", lead + (N,), dy.dtype, dev)
    _need(z, "z", lead + (2 * N,), bf, dev)
    _multiple(K, 8)
    M = x.numel() // K if K else 0
    gdt = bf if grad_dtype is None else grad_dtype
    dx = torch.empty_like(x, dtype=gdt) if need_dx else None
    dw = torch.empty_like(weight, dtype=gdt) if need_dw else None
    db = torch.empty((2 * N,), dtype=torch.float32, device=dev) if bias else None
    lib = load()
    a, dyc, gc = _act_code(act), _code(dy.dtype, "dy"), _code(gdt, "grad_dtype")
    ws = workspace
    if ws is None:
        nbytes = lib.gdn_gated_linear_bwd_workspace(M, N, K, dyc, gc, a, int(need_dx), int(need_dw), int(bool(bias)))
        if nbytes:
            ws = _scratch(nbytes, dev)
    else:
        nbytes = _given(ws, dev)
    _on_device(lib.gdn_gated_linear_bwd, "gdn_gated_linear_bwd", dev,
               _addr(dy), _addr(x), _addr(weight), _addr(z), _addr(dx), _addr(dw), _addr(db), M, N, K, dyc, gc, a,
               _addr(ws), nbytes)
    return dx, dw, db


def _conv(name, x, weight, cu, seqs, bias, act, conv_state, update_conv_state, out):
    torch = _torch()
    dev, f32 = x.device, torch.float32
    lead, C = tuple(x.shape[:-1]), x.shape[-1]
    _need(x, "x", lead + (C,), x.dtype, dev)
    if weight.dim() != 2:
        raise ValueError(f"weight must be [C, W], got {tuple(weight.shape)}")
    W = weight.shape[1]
    _need(weight, "weight", (C, W), f32, dev)
    if bias is not None:
        _need(bias, "bias", (C,), f32, dev)
    if conv_state is not None:
        _need(conv_state, "conv_state", (seqs, W - 1, C), f32, dev)
    if act not in ("none", "silu"):
        raise ValueError(f"act must be none or silu, got {act!r}")
    if update_conv_state:
        if conv_state is None:
            raise ValueError("update_conv_state needs conv_state")
        state = conv_state
    else:
        state = torch.empty((seqs, W - 1, C), dtype=f32, device=dev) if conv_state is None else torch.empty_like(conv_state)
    y = torch.empty_like(x) if out is None else out
    if out is not None:
        _need(y, "out", lead + (C,), x.dtype, dev)
    code = _code(x.dtype, "x")
    lib = load()
    if cu is None:
        _on_device(lib.gdn_causal_conv, name, dev, _addr(x), _addr(weight), _addr(bias), _addr(conv_state), _addr(y),
                   _addr(state), lead[0], lead[1], C, W, code, _act_code(act))
    else:
        _need(cu, "cu_seqlens", (seqs + 1,), torch.int32, dev)
        _on_device(lib.gdn_causal_conv_varlen, name, dev, _addr(x), _addr(weight), _addr(bias), _addr(cu),
                   _addr(conv_state), _addr(y), _addr(state), seqs, lead[0], C, W, code, _act_code(act))
    return y, state


def gdn_causal_conv(x, weight, bias=None, act="silu", conv_state=None, update_conv_state=False, out=None):
    """Short causal convolution per channel: y_t = act(bias + sum_j weight[:, j] x_{t-W+1+j}).  x [B,T,C] bf16 or fp32;
    weight [C,W] fp32, W 2 to 4; bias [C] fp32 or None; act: none or silu; conv_state [B,W-1,C] fp32 (the inputs before
    t = 0, oldest first) or None.  Returns (y in the type of x, new conv state); with update_conv_state the new state
    overwrites conv_state.  T = 1 is one decode token."""
    if x.dim() != 3:
        raise ValueError(f"x must be [B, T, C], got {tuple(x.shape)}")
    return _conv("gdn_causal_conv", x, weight, None, x.shape[0], bias, act, conv_state, update_conv_state, out)


def gdn_causal_conv_varlen(x, weight, cu_seqlens, bias=None, act="silu", conv_state=None, update_conv_state=False,
                           out=None):
    """gdn_causal_conv over packed sequences: x [total_T,C], cu_seqlens int32 [N+1] on the device, states [N,W-1,C]."""
    if x.dim() != 2:
        raise ValueError(f"x must be [total_T, C], got {tuple(x.shape)}")
    return _conv("gdn_causal_conv_varlen", x, weight, cu_seqlens, cu_seqlens.numel() - 1, bias, act, conv_state,
                 update_conv_state, out)


_SCAN_CHANNELS = 4  # the fewest that the scan's kernels take; fewer are filled up with channels of zeros


def gdn_selective_scan_workspace(B, T, ch, N):
    return int(load().gdn_selective_scan_workspace(B, T, max(ch, _SCAN_CHANNELS) if ch > 0 else ch, N))


def gdn_selective_scan_varlen_workspace(seqs, total_T, ch, N):
    return int(load().gdn_selective_scan_varlen_workspace(seqs, total_T, max(ch, _SCAN_CHANNELS) if ch > 0 else ch, N))


def _scan_inputs(x, dt, A, B, C, D, z, dt_bias):
    """Checks what the scan and the step share; (channels, states)."""
    f32 = _torch().float32
    dev, lead, ch = x.device, tuple(x.shape[:-1]), x.shape[-1]
    if A.dim() != 2:
        raise ValueError(f"A must be [channels, N], got {tuple(A.shape)}")
    N = A.shape[1]
    _need(x, "x", lead + (ch,), x.dtype, dev)
    _need(dt, "dt", lead + (ch,), x.dtype, dev)
    _need(A, "A", (ch, N), f32, dev)
    _need(B, "B", lead + (N,), x.dtype, dev)
    _need(C, "C", lead + (N,), x.dtype, dev)
    if D is not None:
        _need(D, "D", (ch,), f32, dev)
    if z is not None:
        _need(z, "z", lead + (ch,), x.dtype, dev)
    if dt_bias is not None:
        _need(dt_bias, "dt_bias", (ch,), f32, dev)
    return ch, N


def _overlap(a, b):
    if b is None:
        return False
    a0, b0 = a.data_ptr(), b.data_ptr()
    return a0 < b0 + b.numel() * b.element_size() and b0 < a0 + a.numel() * a.element_size()


def _scan(name, x, dt, A, B, C, cu, seqs, D, z, dt_bias, h0, output_final_state, workspace, out, final_state):
    torch = _torch()
    dev, f32 = x.device, torch.float32
    ch, N = _scan_inputs(x, dt, A, B, C, D, z, dt_bias)
    if h0 is not None:
        _need(h0, "h0", (seqs, ch, N), f32, dev)
    y = torch.empty_like(x) if out is None else out
    if out is not None:
        _need(y, "out", tuple(x.shape), x.dtype, dev)
    ht = None
    if output_final_state:
        if final_state is not None:
            ht = final_state
            _need(ht, "final_state", (seqs, ch, N), f32, dev)
        else:
            ht = torch.empty((seqs, ch, N), dtype=f32, device=dev) if h0 is None else torch.empty_like(h0)
    if 0 < ch < _SCAN_CHANNELS:
        # what the call below would refuse of the given buffers, and no longer sees
        read = [x, dt, A, B, C, cu, D, z, dt_bias]
        bad = any(_overlap(y, t) for t in read + [h0, ht])
        if ht is not None:
            in_place = h0 is not None and h0.data_ptr() == ht.data_ptr()
            bad = bad or any(_overlap(ht, t) for t in read + ([] if in_place else [h0]))
        _check(int(bad), name)

        def last(t):
            return None if t is None else torch.nn.functional.pad(t, (0, _SCAN_CHANNELS - ch))

        def rows(t):
            return None if t is None else torch.nn.functional.pad(t, (0, 0, 0, _SCAN_CHANNELS - ch))

        # a given out keeps what it holds for tokens of no sequence
        wide, state = _scan(name, last(x), last(dt), rows(A), B, C, cu, seqs, last(D), last(z), last(dt_bias), rows(h0),
                            output_final_state, workspace, last(out), None)
        y.copy_(wide[..., :ch])
        if ht is not None:
            ht.copy_(state[:, :ch])
        return y, ht
    code = _code(x.dtype, "x")
    lib = load()
    T = x.shape[0] if cu is not None else x.shape[1]
    ws = workspace
    if ws is None:
        query = lib.gdn_selective_scan_workspace if cu is None else lib.gdn_selective_scan_varlen_workspace
        nbytes = query(seqs, T, ch, N)
        if nbytes:
            ws = _scratch(nbytes, dev)
    else:
        nbytes = _given(ws, dev)
    if cu is None:
        _on_device(lib.gdn_selective_scan, name, dev, _addr(x), _addr(dt), _addr(A), _addr(B), _addr(C), _addr(D),
                   _addr(z), _addr(dt_bias), _addr(h0), _addr(y), _addr(ht), seqs, T, ch, N, code, _addr(ws), nbytes)
    else:
        _need(cu, "cu_seqlens", (seqs + 1,), torch.int32, dev)
        _on_device(lib.gdn_selective_scan_varlen, name, dev, _addr(x), _addr(dt), _addr(A), _addr(B), _addr(C),
                   _addr(cu), _addr(D), _addr(z), _addr(dt_bias), _addr(h0), _addr(y), _addr(ht), seqs, T, ch, N, code,
                   _addr(ws), nbytes)
    return y, ht


def gdn_selective_scan(x, dt, A, B, C, D=None, z=None, dt_bias=None, h0=None, output_final_state=True, workspace=None,
                       out=None, final_state=None):
    """Selective state space scan: d = softplus(dt + dt_bias), h_t = exp(d A) h_{t-1} + d x B, y = (C . h + D x) silu(z).
    x, dt, z [batch,T,ch] and B, C [batch,T,N] in one type (bf16 or fp32); A [ch,N], D, dt_bias [ch] fp32 (z, D and
    dt_bias may be None); h0 [batch,ch,N] fp32 or None; N 8, 16, 32 or 64.  final_state may be h0 itself.  One to three
    channels are scanned as four, in copies filled up with zeros.  Returns (y in the type of x, final state or None)."""
    if x.dim() != 3:
        raise ValueError(f"x must be [batch, T, channels], got {tuple(x.shape)}")
    return _scan("gdn_selective_scan", x, dt, A, B, C, None, x.shape[0], D, z, dt_bias, h0, output_final_state, workspace,
                 out, final_state)


def gdn_selective_scan_varlen(x, dt, A, B, C, cu_seqlens, D=None, z=None, dt_bias=None, h0=None,
                              output_final_state=True, workspace=None, out=None, final_state=None):
    """gdn_selective_scan over packed sequences: x, dt, z [total_T,ch], B, C [total_T,N], cu_seqlens int32 [n+1] on the
    device, states [n,ch,N]."""
    if x.dim() != 2:
        raise ValueError(f"x must be [total_T, channels], got {tuple(x.shape)}")
    return _scan("gdn_selective_scan_varlen", x, dt, A, B, C, cu_seqlens, cu_seqlens.numel() - 1, D, z, dt_bias, h0,
                 output_final_state, workspace, out, final_state)


def gdn_selective_step(x, dt, A, B, C, state, D=None, z=None, dt_bias=None, out=None, state_out=None):
    """One decode token of gdn_selective_scan: x, dt, z [batch,ch], B, C [batch,N], state [batch,ch,N] fp32, updated in
    place unless state_out is given.  Returns (y [batch,ch], the new state)."""
    torch = _torch()
    if x.dim() != 2:
        raise ValueError(f"x must be [batch, channels], got {tuple(x.shape)}")
    dev, n = x.device, x.shape[0]
    ch, N = _scan_inputs(x, dt, A, B, C, D, z, dt_bias)
    _need(state, "state", (n, ch, N), torch.float32, dev)
    new = state if state_out is None else state_out
    if state_out is not None:
        _need(new, "state_out", (n, ch, N), torch.float32, dev)
    y = torch.empty_like(x) if out is None else out
    if out is not None:
        _need(y, "out", (n, ch), x.dtype, dev)
    _on_device(load().gdn_selective_step, "gdn_selective_step", dev, _addr(x), _addr(dt), _addr(A), _addr(B), _addr(C),
               _addr(D), _addr(z), _addr(dt_bias), _addr(state), _addr(new), _addr(y), n, ch, N, _code(x.dtype, "x"))
    return y, new


def clock_probe(nblocks=256, spin_us=2000, device="cuda"):
    """Enqueue the clock probe (measurement aid) on torch's current stream and
    return a device tensor [nblocks, 2] int64 of (shader cycles, 100 MHz ticks);
    read it after the stream has run: clock_MHz = 100 * cycles / ticks."""
    torch = _torch()
    out = torch.zeros((nblocks, 2), dtype=torch.int64, device=device)
    _check(load().gdn_clock_probe(_ptr(out), int(nblocks), int(spin_us), _stream(out.device)), "gdn_clock_probe")
    return out
