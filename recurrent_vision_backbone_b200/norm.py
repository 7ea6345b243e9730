"""Python binding of include/gtr_norm.h: the channels-last group norm with an activation (every
step runs in the CUDA library; the checks and the marshalling in csrc/binding.cpp).

Outputs and workspaces that a call allocates belong to the stream it runs on.
"""
from __future__ import annotations

from .gla import load
from .ssm import ACT_NONE, ACT_SILU, _run  # noqa: F401


def group_norm_fwd_workspace_bytes(B: int, N: int, C: int, groups: int) -> int:
    """Workspace gtr_group_norm_fwd needs (0: none, or a rejected shape)."""
    return int(load().gtr_group_norm_fwd_workspace_bytes(B, N, C, groups))


def group_norm_bwd_workspace_bytes(B: int, N: int, C: int, groups: int) -> int:
    """Workspace gtr_group_norm_bwd needs (0: none, or a rejected shape)."""
    return int(load().gtr_group_norm_bwd_workspace_bytes(B, N, C, groups))


def gtr_group_norm_fwd(x, groups: int, gamma=None, beta=None, eps: float = 1e-5, activation: int = ACT_NONE, out=None,
                       stats=None, workspace=None, stream=None):
    """act(group_norm(x) gamma + beta) over the tokens and the channels of a group, channels last (each token
    by itself: x as [tokens, C]).

    x: fp16 or bf16 [B, ..., C], contiguous; gamma, beta: float32 [C] or None; out: a tensor like x to
    fill (x itself for in place) or None; stats: a float32 [B, groups, 2] tensor to fill with the
    means and reciprocal deviations (the backward pass takes it; without any token it is left as it
    is) or None to allocate one;
    workspace: a CUDA tensor of group_norm_fwd_workspace_bytes(...) bytes, or None to allocate one.
    Returns (out, stats)."""
    return _run("norm_fwd", stream, x, gamma, beta, out, stats, workspace, groups, eps, activation)


def gtr_group_norm_bwd(x, d_out, stats, groups: int, gamma=None, beta=None, activation: int = ACT_NONE, workspace=None,
                       grads=None, stream=None):
    """Gradients of gtr_group_norm_fwd given d_out (like x) and the stats it returned.  workspace: a
    CUDA tensor of group_norm_bwd_workspace_bytes(...) bytes, or None to allocate one.  grads:
    (grad_x, grad_gamma, grad_beta) to fill, or None to allocate them (those of absent parameters
    stay None).  Returns that tuple: grad_x of x's type, the others float32."""
    return _run("norm_bwd", stream, x, d_out, stats, gamma, beta, workspace, grads, groups, activation)
