"""Python binding of include/gtr_norm.h: the channels-last group norm with an activation
(argument marshalling only; every step runs in the CUDA library)."""
from __future__ import annotations

import torch

from .gla import load
from .ssm import ACT_NONE, ACT_SILU, DTYPES, _check, _dense, _device, _new, _stream, _workspace  # noqa: F401


def _shape(x, groups, gamma, beta):
    if x.dim() < 2:
        raise ValueError("x must be [B, ..., C]")
    if x.dtype not in DTYPES or not x.is_contiguous():
        raise ValueError("x must be a contiguous float16 or bfloat16 tensor")
    dev = _device(x, "x")
    B, C = x.shape[0], x.shape[-1]
    N = 1
    for n in x.shape[1:-1]:
        N *= n
    if groups <= 0 or C == 0 or C % groups:
        raise ValueError(f"{groups} groups do not divide {C} channels")
    return B, N, C, dev, _dense(gamma, "gamma", (C,), torch.float32, dev, False), _dense(beta, "beta", (C,), torch.float32, dev, False)


def group_norm_fwd_workspace_bytes(B: int, N: int, C: int, groups: int) -> int:
    """Workspace gtr_group_norm_fwd needs (0: none, or a rejected shape)."""
    return int(load().gtr_group_norm_fwd_workspace_bytes(B, N, C, groups))


def group_norm_bwd_workspace_bytes(B: int, N: int, C: int, groups: int) -> int:
    """Workspace gtr_group_norm_bwd needs (0: none, or a rejected shape)."""
    return int(load().gtr_group_norm_bwd_workspace_bytes(B, N, C, groups))


def gtr_group_norm_fwd(x, groups: int, gamma=None, beta=None, eps: float = 1e-5, activation: int = ACT_NONE, out=None,
                       stats=None, workspace=None, stream=None):
    """act(group_norm(x) gamma + beta) over the tokens and the channels of a group, channels last.

    x: fp16 or bf16 [B, ..., C]; gamma, beta: float32 [C] or None; out: a tensor like x to fill (x
    itself for in place) or None; stats: a float32 [B, groups, 2] tensor to fill with the means and
    reciprocal deviations (the backward pass takes it) or None to allocate one; workspace: a CUDA
    tensor of group_norm_fwd_workspace_bytes(...) bytes, or None to allocate one.  Returns
    (out, stats)."""
    B, N, C, dev, gp, bp = _shape(x, groups, gamma, beta)
    if out is None:
        out = _new(x, x.shape, x.dtype, stream)
    if stats is None:
        stats = _new(x, (B, groups, 2), torch.float32, stream)
    ws, wp, nbytes = _workspace(workspace, group_norm_fwd_workspace_bytes(B, N, C, groups), x, stream)
    _check(load().gtr_group_norm_fwd(x.data_ptr(), gp, bp, B, N, C, groups, eps, DTYPES[x.dtype], int(activation),
                                     _dense(out, "out", x.shape, x.dtype, dev),
                                     _dense(stats, "stats", (B, groups, 2), torch.float32, dev), wp, nbytes,
                                     _stream(stream)), "gtr_group_norm_fwd")
    return out, stats


def gtr_group_norm_bwd(x, d_out, stats, groups: int, gamma=None, beta=None, activation: int = ACT_NONE, workspace=None,
                       grads=None, stream=None):
    """Gradients of gtr_group_norm_fwd given d_out (like x) and the stats it returned.  workspace: a
    CUDA tensor of group_norm_bwd_workspace_bytes(...) bytes, or None to allocate one.  grads:
    (grad_x, grad_gamma, grad_beta) to fill, or None to allocate them (those of absent parameters
    stay None).  Returns that tuple: grad_x of x's type, the others float32."""
    B, N, C, dev, gp, bp = _shape(x, groups, gamma, beta)
    if grads is None:
        grads = (_new(x, x.shape, x.dtype, stream), None if gamma is None else _new(x, (C,), torch.float32, stream),
                 None if beta is None else _new(x, (C,), torch.float32, stream))
    gx, gg, gb = grads
    ws, wp, nbytes = _workspace(workspace, group_norm_bwd_workspace_bytes(B, N, C, groups), x, stream)
    _check(load().gtr_group_norm_bwd(x.data_ptr(), _dense(d_out, "d_out", x.shape, x.dtype, dev),
                                     _dense(stats, "stats", (B, groups, 2), torch.float32, dev), gp, bp, B, N, C, groups,
                                     DTYPES[x.dtype], int(activation), _dense(gx, "grad_x", x.shape, x.dtype, dev),
                                     _dense(gg, "grad_gamma", (C,), torch.float32, dev, False),
                                     _dense(gb, "grad_beta", (C,), torch.float32, dev, False), wp, nbytes,
                                     _stream(stream)), "gtr_group_norm_bwd")
    return grads
