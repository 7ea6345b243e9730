"""Arguments of the Python binding that raise by themselves (GPU only: host tensors are refused first)."""
import pytest
import torch

from recurrent_vision_backbone_b200 import gla, ssm

pytestmark = pytest.mark.gpu


class NoTruth:
    def __bool__(self):
        raise LookupError("neither true nor false")


def test_an_error_in_a_truth_value_is_raised():
    x = torch.ones(1, 4, 8, dtype=torch.float16, device="cuda")
    b, A, w = x[..., :2].contiguous(), -torch.ones(8, 2, device="cuda"), torch.ones(8, 4, device="cuda")
    with pytest.raises(LookupError):
        ssm.gtr_causal_conv_bwd(x, w, x, 2, 2, 0, want_init_grad=NoTruth())
    with pytest.raises(LookupError):
        ssm.gtr_ssm_scan_bwd(x, x, A, b, b, x, 2, 2, 0, want_init_grad=NoTruth())
    with pytest.raises(LookupError):
        ssm.gtr_ssm_scan_fwd(x, x, A, b, b, 2, 2, 0, dt_softplus=NoTruth())
    assert gla.device_status() == gla.GTR_OK
