"""gtr_gla_device_status over the error words of all operators (GPU only): one call reports and clears
them, from whichever operator they come, and nothing that another stream's kernels record while it
runs goes unreported."""
import threading

import pytest
import torch

from recurrent_vision_backbone_b200 import gla, norm, ssm

pytestmark = pytest.mark.gpu


def operators():
    """Calls of each operator whose result leaves the fp16 range, one source file each."""
    one = lambda *s, v=1.0: torch.full(s, v, dtype=torch.float16, device="cuda")  # noqa: E731
    f32 = lambda *s, v=1.0: torch.full(s, v, device="cuda")  # noqa: E731
    x, bc = one(1, 8, 64), one(1, 8, 16, v=0.0)
    return {
        "conv": lambda: ssm.gtr_causal_conv_fwd(x, f32(64, 4), 1, 8, 0, bias=f32(64, v=1e6), activation=0),
        "scan": lambda: ssm.gtr_ssm_scan_fwd(x, x, -f32(64, 16), bc, bc, 1, 8, 0, D=f32(64, v=1e6)),
        "scan backward": lambda: ssm.gtr_ssm_scan_bwd(x, x, -f32(64, 16), bc, bc, x, 1, 8, 0, D=f32(64, v=1e6)),
        "norm": lambda: norm.gtr_group_norm_fwd(x, 4, None, f32(64, v=1e6)),
    }


def test_each_operator_and_all_at_once():
    assert gla.device_status() == gla.GTR_OK
    calls = operators()
    for name, call in calls.items():
        call()
        assert gla.device_status() == gla.GTR_ERR_RANGE, name
        assert gla.device_status() == gla.GTR_OK, name
    for call in calls.values():
        call()
    assert gla.device_status() == gla.GTR_ERR_RANGE
    assert gla.device_status() == gla.GTR_OK


def test_a_timeout_counts_more():
    assert gla.device_status() == gla.GTR_OK
    operators()["norm"]()
    assert gla.selftest_timeout(1000) == gla.GTR_OK
    assert gla.device_status() == gla.GTR_ERR_TIMEOUT
    assert gla.device_status() == gla.GTR_OK


def test_while_another_stream_runs():
    """A call that leaves the range on a stream of its own, the status asked for meanwhile from two host
    threads: it is reported once or more, by the end at the latest, and then no more."""
    call = operators()["conv"]
    call()
    assert gla.device_status() == gla.GTR_ERR_RANGE
    side, seen = torch.cuda.Stream(), []
    torch.cuda.synchronize()
    for _ in range(50):
        with torch.cuda.stream(side):
            call()
        seen.clear()
        ask = [threading.Thread(target=lambda: seen.append(gla.device_status())) for _ in range(2)]
        for t in ask:
            t.start()
        for t in ask:
            t.join()
        side.synchronize()
        seen.append(gla.device_status())
        assert set(seen) <= {gla.GTR_OK, gla.GTR_ERR_RANGE} and gla.GTR_ERR_RANGE in seen
        assert gla.device_status() == gla.GTR_OK
