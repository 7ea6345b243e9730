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

from .gla import B2T, GTR_OK, L2R, R2L, T2B, GTRError, load  # noqa: F401

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


# Checks are spelled for speed: a call of one token takes a few microseconds on the GPU, so the
# host side of a call is kept to the reads of tensor metadata that the checks need.
def _addr(t):
    return None if t is None else t.data_ptr()


def _device(t, name):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    cur = torch.cuda.current_device()
    if t.get_device() != cur:
        raise ValueError(f"{name} is on {t.device}, but the current CUDA device is cuda:{cur}")
    return cur


def _rows(t, name, shape, dtype, dev):
    """Checks a [B, N, cols] activation on device `dev`; returns the elements between its token rows."""
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, not {list(t.shape)}")
    if t.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype}, like the other activations")
    if t.get_device() != dev:
        _device(t, name)
    if t.is_contiguous():
        return shape[2]
    B, N, cols = shape
    if B == 0 or N == 0:
        return 0
    sb, sn, sc = t.stride()
    if cols > 1 and sc != 1:
        raise ValueError(f"{name}'s channels must be contiguous")
    ld = sn if N > 1 else (sb if B > 1 else cols)
    if ld < cols or (B > 1 and sb != N * ld):
        raise ValueError(f"{name}'s token rows must be evenly spaced and must not overlap")
    return ld


def _dense(t, name, shape, dtype, dev, required=True):
    if t is None:
        if required:
            raise ValueError(f"{name} is required")
        return None
    if t.shape != shape or t.dtype is not dtype or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor {list(shape)}")
    if t.get_device() != dev:
        _device(t, name)
    return t.data_ptr()


def _grid(x, name, Hgrid, Wgrid):
    if x.dim() != 3:
        raise ValueError(f"{name} must be [B, N, channels]")
    if x.dtype not in DTYPES:
        raise ValueError(f"{name} must be float16 or bfloat16")
    if x.shape[1] != Hgrid * Wgrid:
        raise ValueError(f"N={x.shape[1]} does not match the grid {Hgrid}x{Wgrid}")
    return x.shape, _device(x, name)


def _new(like, shape, dtype, stream):
    """A tensor on `like`'s device that belongs to the stream the call runs on."""
    if stream is None:
        return like.new_empty(shape, dtype=dtype)
    with torch.cuda.stream(stream):
        return like.new_empty(shape, dtype=dtype)


def _workspace(t, nbytes, like, stream):
    """(tensor, address, bytes) of the caller's workspace or a new one."""
    if nbytes == 0:
        return None, None, 0
    if t is None:
        t = _new(like, (nbytes,), torch.uint8, stream)
    else:
        _device(t, "workspace")
        if not t.is_contiguous():
            raise ValueError("workspace must be contiguous")
    return t, t.data_ptr(), t.numel() * t.element_size()


def _stream(stream):
    return torch.cuda.current_stream().cuda_stream if stream is None else stream.cuda_stream


def _check(status, where):
    if status != GTR_OK:
        raise GTRError(status, where)


# ------------------------------------------------------------------ short causal convolution
def _conv(x, w, Hgrid, Wgrid, direction, bias, activation, init_state):
    (B, N, D), dev = _grid(x, "x", Hgrid, Wgrid)
    ld = _rows(x, "x", (B, N, D), x.dtype, dev)
    if w.dim() != 2:
        raise ValueError("w must be [D, K]")
    K = w.shape[1]
    c = _Conv(B, int(Hgrid), int(Wgrid), D, K, int(direction), DTYPES[x.dtype], int(activation), x.data_ptr(), ld,
              _dense(w, "w", (D, K), torch.float32, dev), _dense(bias, "bias", (D,), torch.float32, dev, False),
              _dense(init_state, "init_state", (B, K - 1, D), x.dtype, dev, False))
    return c, (B, N, D, K), dev


def gtr_causal_conv_fwd(x, w, Hgrid: int, Wgrid: int, direction: int, bias=None, activation: int = ACT_SILU,
                        init_state=None, out=None, final_state=None, stream=None):
    """Depthwise causal convolution over the scan order: act(bias + sum_j w[:, j] X[p + j]) with
    X = [init_state ; x in scan order].

    x: [B, N, D]; w: float32 [D, K], K in 2..4 (w[:, K - 1] weighs the token itself); bias:
    float32 [D] or None; init_state: the K - 1 earlier inputs, oldest first, [B, K-1, D] of x's
    type, or None for zeros; final_state: a tensor to fill (init_state itself for an in-place
    carry), True to allocate one, or None.  Returns (out, final_state)."""
    c, (B, N, D, K), dev = _conv(x, w, Hgrid, Wgrid, direction, bias, activation, init_state)
    if out is None:
        out = _new(x, (B, N, D), x.dtype, stream)
    if final_state is True:
        final_state = _new(x, (B, max(K - 1, 0), D), x.dtype, stream)
    _check(load().gtr_causal_conv_fwd(ctypes.byref(c), _dense(out, "out", (B, N, D), x.dtype, dev),
                                      _dense(final_state, "final_state", (B, K - 1, D), x.dtype, dev, False),
                                      _stream(stream)), "gtr_causal_conv_fwd")
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
    c, (B, N, D, K), dev = _conv(x, w, Hgrid, Wgrid, direction, bias, activation, init_state)
    ld = _rows(d_out, "d_out", (B, N, D), x.dtype, dev)
    df = _dense(d_final_state, "d_final_state", (B, K - 1, D), x.dtype, dev, False)
    if grads is None:
        grads = (_new(x, (B, N, D), x.dtype, stream), _new(x, (D, K), torch.float32, stream),
                 None if bias is None else _new(x, (D,), torch.float32, stream),
                 _new(x, (B, max(K - 1, 0), D), x.dtype, stream) if want_init_grad else None)
    gx, gw, gb, gi = grads
    ws, wp, nbytes = _workspace(workspace, causal_conv_bwd_workspace_bytes(B, Hgrid, Wgrid, D, K), x, stream)
    _check(load().gtr_causal_conv_bwd(ctypes.byref(c), d_out.data_ptr(), ld, df,
                                      _dense(gx, "grad_x", (B, N, D), x.dtype, dev),
                                      _dense(gw, "grad_w", (D, K), torch.float32, dev),
                                      _dense(gb, "grad_bias", (D,), torch.float32, dev, False),
                                      _dense(gi, "grad_init_state", (B, K - 1, D), x.dtype, dev, False), wp, nbytes,
                                      _stream(stream)), "gtr_causal_conv_bwd")
    return gx, gw, gb, gi


# ------------------------------------------------------------------ selective scan
def _ssm(u, dt, A, Bm, Cm, Hgrid, Wgrid, direction, D, z, dt_bias, dt_softplus, init_state):
    (B, N, C), dev = _grid(u, "u", Hgrid, Wgrid)
    if A.dim() != 2:
        raise ValueError("A must be [D, S]")
    S = A.shape[1]
    t, f, tok, st = u.dtype, torch.float32, (B, N, C), (B, N, S)
    m = _Ssm(B, int(Hgrid), int(Wgrid), C, S, int(direction), DTYPES[t], int(bool(dt_softplus)), u.data_ptr(),
             dt.data_ptr(), Bm.data_ptr(), Cm.data_ptr(), _addr(z), _rows(u, "u", tok, t, dev),
             _rows(dt, "dt", tok, t, dev), _rows(Bm, "Bm", st, t, dev), _rows(Cm, "Cm", st, t, dev),
             0 if z is None else _rows(z, "z", tok, t, dev), _dense(A, "A", (C, S), f, dev),
             _dense(D, "D", (C,), f, dev, False), _dense(dt_bias, "dt_bias", (C,), f, dev, False),
             _dense(init_state, "init_state", (B, C, S), f, dev, False))
    return m, (B, N, C, S), dev


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
    m, (B, N, C, S), dev = _ssm(u, dt, A, Bm, Cm, Hgrid, Wgrid, direction, D, z, dt_bias, dt_softplus, init_state)
    if out is None:
        out = _new(u, (B, N, C), u.dtype, stream)
    if final_state is True:
        final_state = _new(u, (B, C, S), torch.float32, stream)
    ws, wp, nbytes = _workspace(workspace, ssm_scan_fwd_workspace_bytes(B, Hgrid, Wgrid, C, S), u, stream)
    _check(load().gtr_ssm_scan_fwd(ctypes.byref(m), _dense(out, "out", (B, N, C), u.dtype, dev),
                                   _dense(final_state, "final_state", (B, C, S), torch.float32, dev, False), wp, nbytes,
                                   _stream(stream)), "gtr_ssm_scan_fwd")
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
    m, (B, N, C, S), dev = _ssm(u, dt, A, Bm, Cm, Hgrid, Wgrid, direction, D, z, dt_bias, dt_softplus, init_state)
    t, f, tok, st = u.dtype, torch.float32, (B, N, C), (B, N, S)
    ld = _rows(d_out, "d_out", tok, t, dev)
    df = _dense(d_final_state, "d_final_state", (B, C, S), f, dev, False)
    if grads is None:
        grads = (_new(u, tok, t, stream), _new(u, tok, t, stream), _new(u, (C, S), f, stream), _new(u, st, t, stream),
                 _new(u, st, t, stream), None if D is None else _new(u, (C,), f, stream),
                 None if z is None else _new(u, tok, t, stream), None if dt_bias is None else _new(u, (C,), f, stream),
                 _new(u, (B, C, S), f, stream) if want_init_grad else None)
    gu, gdt, gA, gB, gC, gD, gz, gt, gi = grads
    if z is None and gz is not None:
        raise ValueError("grad_z without z")
    g = _SsmGrads(_dense(gu, "grad_u", tok, t, dev), _dense(gdt, "grad_dt", tok, t, dev),
                  _dense(gB, "grad_Bm", st, t, dev), _dense(gC, "grad_Cm", st, t, dev),
                  _dense(gz, "grad_z", tok, t, dev, z is not None), _dense(gA, "grad_A", (C, S), f, dev),
                  _dense(gD, "grad_D", (C,), f, dev, False), _dense(gt, "grad_dt_bias", (C,), f, dev, False),
                  _dense(gi, "grad_init_state", (B, C, S), f, dev, False))
    ws, wp, nbytes = _workspace(workspace, ssm_scan_bwd_workspace_bytes(B, Hgrid, Wgrid, C, S), u, stream)
    _check(load().gtr_ssm_scan_bwd(ctypes.byref(m), d_out.data_ptr(), ld, df, ctypes.byref(g), wp, nbytes,
                                   _stream(stream)), "gtr_ssm_scan_bwd")
    return grads
