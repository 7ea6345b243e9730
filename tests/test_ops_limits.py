"""Sizes at the edge of 32-bit indices (CPU only): a row of more than 2^30 - 1 channels is refused before
anything is launched (the kernels count channels in 32 bits, up to a block's width beyond the last)."""
import ctypes

import pytest

from recurrent_vision_backbone_b200 import build, gla, norm, ssm
from tests import ops_abi

GB = 1 << 40   # fake buffers far apart; never dereferenced
BAD = gla.GTR_ERR_INVALID_ARG


@pytest.fixture(scope="module")
def lib():
    return gla.load(build.build())


@pytest.mark.parametrize("D", [1 << 30, (1 << 31) - 128, (1 << 31) - 1])
def test_too_many_channels(lib, D):
    c = ops_abi.Conv(1, 1, 1, D, 4, 0, 0, 1, GB, 0, 2 * GB, None, None)
    assert lib.gtr_causal_conv_fwd(ctypes.byref(c), 3 * GB, None, None) == BAD
    assert lib.gtr_causal_conv_bwd(ctypes.byref(c), 4 * GB, 0, None, 5 * GB, 6 * GB, None, None, 7 * GB, 1 << 39, None) == BAD
    m = ops_abi.Ssm(1, 1, 1, D, 1, 0, 0, 1, GB, 2 * GB, 3 * GB, 4 * GB, None, 0, 0, 0, 0, 0, 5 * GB, None, None, None)
    assert lib.gtr_ssm_scan_fwd(ctypes.byref(m), 6 * GB, None, 7 * GB, 1 << 39, None) == BAD
    g = ops_abi.SsmGrads(8 * GB, 9 * GB, 10 * GB, 11 * GB, None, 12 * GB, None, None, None)
    assert lib.gtr_ssm_scan_bwd(ctypes.byref(m), 13 * GB, 0, None, ctypes.byref(g), 14 * GB, 1 << 39, None) == BAD
    assert lib.gtr_group_norm_fwd(GB, None, None, 1, 1, D, 1, 1e-5, 0, 0, 2 * GB, None, 3 * GB, 1 << 39, None) == BAD
    assert lib.gtr_group_norm_bwd(GB, 2 * GB, 3 * GB, None, None, 1, 1, D, 1, 0, 0, 4 * GB, None, None, 5 * GB, 1 << 39, None) == BAD
    assert ssm.causal_conv_bwd_workspace_bytes(1, 1, 1, D, 4) == 0
    assert ssm.ssm_scan_bwd_workspace_bytes(1, 1, 1, D, 1) == 0
    assert norm.group_norm_fwd_workspace_bytes(1, 1, D, 1) == 0


def test_the_most_channels(lib):
    D = (1 << 30) - 1
    assert ssm.causal_conv_bwd_workspace_bytes(1, 1, 1, D, 4) > 0
    assert ssm.ssm_scan_bwd_workspace_bytes(1, 1, 1, D, 1) > 0
    assert norm.group_norm_fwd_workspace_bytes(1, 1, D, 1) > 0
