"""Python binding of include/gtr_ssm.h: the short causal convolution and the selective scan
(argument marshalling only; every step runs in the CUDA library).

Activations are fp16 or bf16 (one type a call), [B, N, channels] in grid order with
N = Hgrid * Wgrid, the last dimension contiguous and token rows evenly spaced: a channel
slice of a wider projection's output is taken without a copy.  A sequence that is no grid is a
1 x N grid scanned ``L2R``; one token is a 1 x 1 grid with the carried states.

Outputs and workspaces that a call allocates belong to the stream it runs on.
"""
from __future__ import annotations

import ctypes

import torch

from . import gla
from .gla import B2T, GTR_OK, L2R, R2L, T2B, GTRError, _ptr, _stream_handle, load  # noqa: F401

ACT_NONE, ACT_SILU = 0, 1
DTYPES = {torch.float16: 0, torch.bfloat16: 1}


class _Conv(ctypes.Structure):
    """gtr_conv_t"""
    _fields_ = ([(n, ctypes.c_int) for n in ("B", "Hgrid", "Wgrid", "D", "K", "direction", "dtype", "activation")]
                + [("x", ctypes.c_void_p), ("ldx", ctypes.c_longlong), ("w", ctypes.c_void_p),
                   ("bias", ctypes.c_void_p), ("init_state", ctypes.c_void_p)])


class _Ssm(ctypes.Structure):
    """gtr_ssm_t"""
    _fields_ = ([(n, ctypes.c_int) for n in ("B", "Hgrid", "Wgrid", "D", "S", "direction", "dtype", "dt_softplus")]
                + [(n, ctypes.c_void_p) for n in ("u", "dt", "Bm", "Cm", "z")]
                + [(n, ctypes.c_longlong) for n in ("ldu", "lddt", "ldb", "ldc", "ldz")]
                + [(n, ctypes.c_void_p) for n in ("A", "Dskip", "dt_bias", "init_state")])


class _SsmGrads(ctypes.Structure):
    """gtr_ssm_grads_t"""
    _fields_ = [(n, ctypes.c_void_p) for n in ("u", "dt", "Bm", "Cm", "z", "A", "Dskip", "dt_bias", "init_state")]


def _addr(t):
    return None if t is None else t.data_ptr()


def _on(stream):
    """Allocations inside belong to the stream the call runs on."""
    return torch.cuda.stream(stream)     # a no-op for None


def _device(t, name):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    cur = torch.cuda.current_device()
    if t.device.index != cur:
        raise ValueError(f"{name} is on {t.device}, but the current CUDA device is cuda:{cur}")


def _rows(t, name, shape, dtype):
    """Checks a [B, N, cols] activation; returns the elements between its token rows."""
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must be {list(shape)}, not {list(t.shape)}")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, like the other activations")
    _device(t, name)
    B, N, cols = shape
    if t.numel() == 0:
        return 0
    sb, sn, sc = t.stride()
    if cols > 1 and sc != 1:
        raise ValueError(f"{name}'s channels must be contiguous")
    ld = sn if N > 1 else (sb if B > 1 else cols)
    if ld < cols or (B > 1 and sb != N * ld):
        raise ValueError(f"{name}'s token rows must be evenly spaced and must not overlap")
    return ld


def _dense(t, name, shape, dtype, required=True):
    if t is None:
        if required:
            raise ValueError(f"{name} is required")
        return
    if tuple(t.shape) != tuple(shape) or t.dtype != dtype or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor {list(shape)}")
    _device(t, name)


def _grid(x, name, Hgrid, Wgrid):
    if x.dim() != 3:
        raise ValueError(f"{name} must be [B, N, channels]")
    if x.dtype not in DTYPES:
        raise ValueError(f"{name} must be float16 or bfloat16")
    if x.shape[1] != Hgrid * Wgrid:
        raise ValueError(f"N={x.shape[1]} does not match the grid {Hgrid}x{Wgrid}")
    _device(x, name)
    return x.shape


def _workspace(t, nbytes, device, stream):
    if nbytes == 0:
        return None, 0
    if t is None:
        with _on(stream):
            t = torch.empty(nbytes, dtype=torch.uint8, device=device)
    _device(t, "workspace")
    if not t.is_contiguous():
        raise ValueError("workspace must be contiguous")
    return t, t.numel() * t.element_size()


def _new(shape, dtype, device, stream):
    with _on(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _check(status, where):
    if status != GTR_OK:
        raise GTRError(status, where)


# ------------------------------------------------------------------ short causal convolution
def _conv(x, w, Hgrid, Wgrid, direction, bias, activation, init_state):
    B, N, D = _grid(x, "x", Hgrid, Wgrid)
    ld = _rows(x, "x", (B, N, D), x.dtype)
    if w.dim() != 2:
        raise ValueError("w must be [D, K]")
    K = w.shape[1]
    _dense(w, "w", (D, K), torch.float32)
    _dense(bias, "bias", (D,), torch.float32, required=False)
    _dense(init_state, "init_state", (B, K - 1, D), x.dtype, required=False)
    c = _Conv(B, int(Hgrid), int(Wgrid), D, K, int(direction), DTYPES[x.dtype], int(activation), _addr(x), ld,
              _addr(w), _addr(bias), _addr(init_state))
    return c, (B, N, D, K)


def gtr_causal_conv_fwd(x, w, Hgrid: int, Wgrid: int, direction: int, bias=None, activation: int = ACT_SILU,
                        init_state=None, out=None, final_state=None, stream=None):
    """Depthwise causal convolution over the scan order: act(bias + sum_j w[:, j] X[p + j]) with
    X = [init_state ; x in scan order].

    x: [B, N, D]; w: float32 [D, K], K in 2..4 (w[:, K - 1] weighs the token itself); bias:
    float32 [D] or None; init_state: the K - 1 earlier inputs, oldest first, [B, K-1, D] of x's
    type, or None for zeros; final_state: a tensor to fill (init_state itself for an in-place
    carry), True to allocate one, or None.  Returns (out, final_state)."""
    lib = load()
    c, (B, N, D, K) = _conv(x, w, Hgrid, Wgrid, direction, bias, activation, init_state)
    if out is None:
        out = _new((B, N, D), x.dtype, x.device, stream)
    _dense(out, "out", (B, N, D), x.dtype)
    if final_state is True:
        final_state = _new((B, max(K - 1, 0), D), x.dtype, x.device, stream)
    _dense(final_state, "final_state", (B, K - 1, D), x.dtype, required=False)
    _check(lib.gtr_causal_conv_fwd(ctypes.byref(c), _ptr(out), _ptr(final_state), _stream_handle(stream)),
           "gtr_causal_conv_fwd")
    return out, final_state


def causal_conv_bwd_workspace_bytes(B: int, Hgrid: int, Wgrid: int, D: int, K: int) -> int:
    """Workspace gtr_causal_conv_bwd needs (0: none, or a rejected shape)."""
    return int(load().gtr_causal_conv_bwd_workspace_bytes(B, Hgrid, Wgrid, D, K))


def gtr_causal_conv_bwd(x, w, d_out, Hgrid: int, Wgrid: int, direction: int, bias=None, activation: int = ACT_SILU,
                        init_state=None, d_final_state=None, workspace=None, grads=None, want_init_grad: bool = True,
                        stream=None):
    """Gradients of gtr_causal_conv_fwd given d_out ([B, N, D]) and d_final_state ([B, K-1, D] or
    None).  workspace: a CUDA tensor of causal_conv_bwd_workspace_bytes(...) bytes, or None to
    allocate one.  grads: (grad_x, grad_w, grad_bias, grad_init_state) to fill, or None to allocate
    them (grad_bias with a bias, grad_init_state with want_init_grad).  Returns that tuple:
    grad_x and grad_init_state of x's type, the parameters' float32."""
    lib = load()
    c, (B, N, D, K) = _conv(x, w, Hgrid, Wgrid, direction, bias, activation, init_state)
    ld = _rows(d_out, "d_out", (B, N, D), x.dtype)
    _dense(d_final_state, "d_final_state", (B, K - 1, D), x.dtype, required=False)
    if grads is None:
        new = lambda shape, t: _new(shape, t, x.device, stream)  # noqa: E731
        grads = (new((B, N, D), x.dtype), new((D, K), torch.float32),
                 None if bias is None else new((D,), torch.float32),
                 new((B, max(K - 1, 0), D), x.dtype) if want_init_grad else None)
    gx, gw, gb, gi = grads
    _dense(gx, "grad_x", (B, N, D), x.dtype)
    _dense(gw, "grad_w", (D, K), torch.float32)
    _dense(gb, "grad_bias", (D,), torch.float32, required=False)
    _dense(gi, "grad_init_state", (B, K - 1, D), x.dtype, required=False)
    ws, nbytes = _workspace(workspace, causal_conv_bwd_workspace_bytes(B, Hgrid, Wgrid, D, K), x.device, stream)
    _check(lib.gtr_causal_conv_bwd(ctypes.byref(c), _ptr(d_out), ld, _ptr(d_final_state), _ptr(gx), _ptr(gw), _ptr(gb),
                                   _ptr(gi), _ptr(ws), nbytes, _stream_handle(stream)), "gtr_causal_conv_bwd")
    return gx, gw, gb, gi


# ------------------------------------------------------------------ selective scan
def _ssm(u, dt, A, Bm, Cm, Hgrid, Wgrid, direction, D, z, dt_bias, dt_softplus, init_state):
    B, N, C = _grid(u, "u", Hgrid, Wgrid)
    if A.dim() != 2:
        raise ValueError("A must be [D, S]")
    S = A.shape[1]
    t = u.dtype
    ldu, lddt = _rows(u, "u", (B, N, C), t), _rows(dt, "dt", (B, N, C), t)
    ldb, ldc = _rows(Bm, "Bm", (B, N, S), t), _rows(Cm, "Cm", (B, N, S), t)
    ldz = 0 if z is None else _rows(z, "z", (B, N, C), t)
    _dense(A, "A", (C, S), torch.float32)
    _dense(D, "D", (C,), torch.float32, required=False)
    _dense(dt_bias, "dt_bias", (C,), torch.float32, required=False)
    _dense(init_state, "init_state", (B, C, S), torch.float32, required=False)
    m = _Ssm(B, int(Hgrid), int(Wgrid), C, S, int(direction), DTYPES[t], int(bool(dt_softplus)), _addr(u), _addr(dt),
             _addr(Bm), _addr(Cm), _addr(z), ldu, lddt, ldb, ldc, ldz, _addr(A), _addr(D), _addr(dt_bias),
             _addr(init_state))
    return m, (B, N, C, S)


def ssm_scan_fwd_workspace_bytes(B: int, Hgrid: int, Wgrid: int, D: int, S: int) -> int:
    """Workspace gtr_ssm_scan_fwd needs (0: none, or a rejected shape)."""
    return int(load().gtr_ssm_scan_fwd_workspace_bytes(B, Hgrid, Wgrid, D, S))


def gtr_ssm_scan_fwd(u, dt, A, Bm, Cm, Hgrid: int, Wgrid: int, direction: int, D=None, z=None, dt_bias=None,
                     dt_softplus: bool = True, init_state=None, out=None, final_state=None, workspace=None,
                     stream=None):
    """Selective scan: h = exp(t A) h + t u Bm, out = (Cm h + D u) silu(z) over the scan order, with
    t = softplus(dt + dt_bias) (or dt + dt_bias).

    u, dt, z: [B, N, D] (z None: no gate); Bm, Cm: [B, N, S]; A: float32 [D, S], S in 1..32; D,
    dt_bias: float32 [D] or None; init_state: float32 [B, D, S] or None; final_state: a tensor to
    fill (init_state itself for an in-place carry), True to allocate one, or None; workspace: a
    CUDA tensor of ssm_scan_fwd_workspace_bytes(...) bytes, or None to allocate one.  Returns
    (out, final_state)."""
    lib = load()
    m, (B, N, C, S) = _ssm(u, dt, A, Bm, Cm, Hgrid, Wgrid, direction, D, z, dt_bias, dt_softplus, init_state)
    if out is None:
        out = _new((B, N, C), u.dtype, u.device, stream)
    _dense(out, "out", (B, N, C), u.dtype)
    if final_state is True:
        final_state = _new((B, C, S), torch.float32, u.device, stream)
    _dense(final_state, "final_state", (B, C, S), torch.float32, required=False)
    ws, nbytes = _workspace(workspace, ssm_scan_fwd_workspace_bytes(B, Hgrid, Wgrid, C, S), u.device, stream)
    _check(lib.gtr_ssm_scan_fwd(ctypes.byref(m), _ptr(out), _ptr(final_state), _ptr(ws), nbytes,
                                _stream_handle(stream)), "gtr_ssm_scan_fwd")
    return out, final_state


def ssm_scan_bwd_workspace_bytes(B: int, Hgrid: int, Wgrid: int, D: int, S: int) -> int:
    """Workspace gtr_ssm_scan_bwd needs (0: none, or a rejected shape)."""
    return int(load().gtr_ssm_scan_bwd_workspace_bytes(B, Hgrid, Wgrid, D, S))


def gtr_ssm_scan_bwd(u, dt, A, Bm, Cm, d_out, Hgrid: int, Wgrid: int, direction: int, D=None, z=None, dt_bias=None,
                     dt_softplus: bool = True, init_state=None, d_final_state=None, workspace=None, grads=None,
                     want_init_grad: bool = True, stream=None):
    """Gradients of gtr_ssm_scan_fwd given d_out ([B, N, D]) and d_final_state (float32 [B, D, S] or
    None).  workspace: a CUDA tensor of ssm_scan_bwd_workspace_bytes(...) bytes, or None to allocate
    one.  grads: a tuple (grad_u, grad_dt, grad_A, grad_Bm, grad_Cm, grad_D, grad_z, grad_dt_bias,
    grad_init_state) to fill, or None to allocate them (those of absent inputs stay None,
    grad_init_state unless want_init_grad).  Returns that tuple: the activations' gradients of
    their type, the parameters' and the state's float32."""
    lib = load()
    m, (B, N, C, S) = _ssm(u, dt, A, Bm, Cm, Hgrid, Wgrid, direction, D, z, dt_bias, dt_softplus, init_state)
    t, f = u.dtype, torch.float32
    ld = _rows(d_out, "d_out", (B, N, C), t)
    _dense(d_final_state, "d_final_state", (B, C, S), f, required=False)
    if grads is None:
        new = lambda shape, ty: _new(shape, ty, u.device, stream)  # noqa: E731
        grads = (new((B, N, C), t), new((B, N, C), t), new((C, S), f), new((B, N, S), t), new((B, N, S), t),
                 None if D is None else new((C,), f), None if z is None else new((B, N, C), t),
                 None if dt_bias is None else new((C,), f), new((B, C, S), f) if want_init_grad else None)
    gu, gdt, gA, gB, gC, gD, gz, gt, gi = grads
    for g, name, shape, ty, req in ((gu, "grad_u", (B, N, C), t, True), (gdt, "grad_dt", (B, N, C), t, True),
                                    (gA, "grad_A", (C, S), f, True), (gB, "grad_Bm", (B, N, S), t, True),
                                    (gC, "grad_Cm", (B, N, S), t, True), (gD, "grad_D", (C,), f, False),
                                    (gz, "grad_z", (B, N, C), t, z is not None), (gt, "grad_dt_bias", (C,), f, False),
                                    (gi, "grad_init_state", (B, C, S), f, False)):
        _dense(g, name, shape, ty, required=req)
    if z is None and gz is not None:
        raise ValueError("grad_z without z")
    ws, nbytes = _workspace(workspace, ssm_scan_bwd_workspace_bytes(B, Hgrid, Wgrid, C, S), u.device, stream)
    g = _SsmGrads(_addr(gu), _addr(gdt), _addr(gB), _addr(gC), _addr(gz), _addr(gA), _addr(gD), _addr(gt), _addr(gi))
    _check(lib.gtr_ssm_scan_bwd(ctypes.byref(m), _ptr(d_out), ld, _ptr(d_final_state), ctypes.byref(g), _ptr(ws),
                                nbytes, _stream_handle(stream)), "gtr_ssm_scan_bwd")
    return grads
