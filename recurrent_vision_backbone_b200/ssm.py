"""Python binding of include/gtr_ssm.h: the short causal convolution and the selective scan
(every step runs in the CUDA library; the checks and the marshalling in csrc/binding.cpp).

Activations are fp16 or bf16 (one type a call), [B, N, channels] in grid order with
N = Hgrid * Wgrid, the last dimension contiguous and token rows evenly spaced: a channel
slice of a wider projection's output is taken without a copy.  A sequence that is no grid is a
1 x N grid scanned ``L2R``; one token is a 1 x 1 grid with the carried states.

Outputs and workspaces that a call allocates belong to the stream it runs on.
"""
from __future__ import annotations

import torch

from .gla import B2T, L2R, R2L, T2B, GTRError, load  # noqa: F401

ACT_NONE, ACT_SILU = 0, 1

_module = None


def _ops():
    """The extension module, beside the CUDA library (raises if it has not been built)."""
    global _module
    if _module is None:
        load()
        try:
            from . import _ops as m
        except ImportError as e:
            raise RuntimeError("the extension module is missing or was made for another torch: build it with "
                               "`python -m recurrent_vision_backbone_b200.build`") from e
        _module = m
    return _module


def _run(where, stream, *args):
    """One call of the extension module on `stream` (None: the current one)."""
    f = getattr(_ops(), where)
    if stream is None:
        r = f(*args)
    else:
        with torch.cuda.stream(stream):
            r = f(*args)
    if type(r) is int:
        raise GTRError(r, _NAMES[where])
    return r


_NAMES = {"conv_fwd": "gtr_causal_conv_fwd", "conv_bwd": "gtr_causal_conv_bwd", "scan_fwd": "gtr_ssm_scan_fwd",
          "scan_bwd": "gtr_ssm_scan_bwd", "norm_fwd": "gtr_group_norm_fwd", "norm_bwd": "gtr_group_norm_bwd"}


# ------------------------------------------------------------------ short causal convolution
def gtr_causal_conv_fwd(x, w, Hgrid: int, Wgrid: int, direction: int, bias=None, activation: int = ACT_SILU,
                        init_state=None, out=None, final_state=None, stream=None):
    """Depthwise causal convolution over the scan order: act(bias + sum_j w[:, j] X[p + j]) with
    X = [init_state ; x in scan order].

    x: [B, N, D]; w: float32 [D, K], K in 2..4 (w[:, K - 1] weighs the token itself); bias:
    float32 [D] or None; init_state: the K - 1 earlier inputs, oldest first, [B, K-1, D] of x's
    type, or None for zeros; final_state: a tensor to fill (init_state itself for an in-place
    carry), True to allocate one, or None.  Returns (out, final_state)."""
    return _run("conv_fwd", stream, x, w, bias, init_state, out, final_state, Hgrid, Wgrid, direction, activation)


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
    return _run("conv_bwd", stream, x, w, d_out, bias, init_state, d_final_state, workspace, grads, want_init_grad, Hgrid,
                Wgrid, direction, activation)


# ------------------------------------------------------------------ selective scan
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
    return _run("scan_fwd", stream, u, dt, A, Bm, Cm, D, z, dt_bias, init_state, out, final_state, workspace, Hgrid, Wgrid,
                direction, dt_softplus)


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
    return _run("scan_bwd", stream, u, dt, A, Bm, Cm, d_out, D, z, dt_bias, init_state, d_final_state, workspace, grads,
                want_init_grad, Hgrid, Wgrid, direction, dt_softplus)
