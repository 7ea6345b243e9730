"""Host-side argument checks of gtr_ssm.h and gtr_norm.h (CPU only, no compute call): every case
is one the library rejects before it touches the device, so the fake pointers are never
dereferenced."""
import ctypes

import pytest

from recurrent_vision_backbone_b200 import build, gla, norm, ssm
from tests import ops_abi

MB = 1 << 24   # fake buffers 16 MiB apart
BAD, UNSUP = gla.GTR_ERR_INVALID_ARG, gla.GTR_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    return gla.load(build.build())


def P(x):
    return None if x is None else x * MB if x < 64 else x


def conv(x=1, w=2, bias=3, init=4, B=2, H=8, W=8, D=64, K=4, direction=0, dtype=0, act=1, ldx=0):
    return ops_abi.Conv(B, H, W, D, K, direction, dtype, act, P(x), ldx, P(w), P(bias), P(init))


CONV_BAD = [(dict(B=0), BAD), (dict(D=0), BAD), (dict(H=-1), BAD), (dict(direction=4), BAD), (dict(dtype=2), BAD),
            (dict(act=2), BAD), (dict(K=0), BAD), (dict(K=1), UNSUP), (dict(K=5), UNSUP), (dict(x=None), BAD),
            (dict(w=None), BAD), (dict(x=MB + 1), BAD), (dict(w=2 * MB + 8), BAD), (dict(bias=3 * MB + 4), BAD),
            (dict(init=4 * MB + 1), BAD), (dict(ldx=63), BAD), (dict(ldx=-64), BAD), (dict(H=1 << 15, W=1 << 15), BAD),
            (dict(B=1 << 20, H=1 << 12, W=1 << 12), BAD)]


@pytest.mark.parametrize("bad,code", CONV_BAD + [
    (dict(out=None), BAD), (dict(out=1), BAD), (dict(out=MB + 4096), BAD), (dict(out=4), BAD), (dict(fin=5), BAD),
    (dict(fin=4 * MB + 64), BAD), (dict(out=5 * MB + 1), BAD)])
def test_conv_forward_refusals(lib, bad, code):
    bad = dict(bad)
    out, fin = bad.pop("out", 5), bad.pop("fin", 6)
    c = conv(**bad)
    assert lib.gtr_causal_conv_fwd(ctypes.byref(c), P(out), P(fin), None) == code


@pytest.mark.parametrize("bad,code", CONV_BAD + [
    (dict(dy=None), BAD), (dict(ld=5), BAD), (dict(gx=None), BAD), (dict(gw=None), BAD), (dict(gx=5), BAD),
    (dict(gw=8 * MB + 4), BAD), (dict(gb=8 * MB + 16), BAD), (dict(gi=1), BAD), (dict(ws=None), BAD),
    (dict(wsb=64), BAD), (dict(ws=5), BAD), (dict(ws=11 * MB + 8), BAD), (dict(ws=7), BAD)])
def test_conv_backward_refusals(lib, bad, code):
    bad = dict(bad)
    a = {k: bad.pop(k, v) for k, v in dict(dy=5, ld=0, df=6, gx=7, gw=8, gb=9, gi=10, ws=11, wsb=1 << 22).items()}
    c = conv(**bad)
    assert lib.gtr_causal_conv_bwd(ctypes.byref(c), P(a["dy"]), a["ld"], P(a["df"]), P(a["gx"]), P(a["gw"]), P(a["gb"]),
                                   P(a["gi"]), P(a["ws"]), a["wsb"], None) == code


def scan(u=1, dt=2, Bm=3, Cm=4, z=5, A=6, D=7, bias=8, init=9, B=2, H=64, W=64, C=64, S=16, direction=0, dtype=0,
         softplus=1, ldu=0, lddt=0, ldb=0, ldc=0, ldz=0):
    return ops_abi.Ssm(B, H, W, C, S, direction, dtype, softplus, P(u), P(dt), P(Bm), P(Cm), P(z), ldu, lddt, ldb, ldc, ldz,
                    P(A), P(D), P(bias), P(init))


SCAN_BAD = [(dict(B=0), BAD), (dict(C=-1), BAD), (dict(W=-1), BAD), (dict(direction=-1), BAD), (dict(dtype=-1), BAD),
            (dict(softplus=2), BAD), (dict(S=0), BAD), (dict(S=33), UNSUP), (dict(u=None), BAD), (dict(dt=None), BAD),
            (dict(Bm=None), BAD), (dict(Cm=None), BAD), (dict(A=None), BAD), (dict(z=5 * MB + 1), BAD),
            (dict(A=6 * MB + 4), BAD), (dict(D=7 * MB + 8), BAD), (dict(bias=8 * MB + 2), BAD),
            (dict(init=9 * MB + 8), BAD), (dict(ldu=1), BAD), (dict(lddt=-1), BAD), (dict(ldb=15), BAD),
            (dict(ldc=1), BAD), (dict(ldz=63), BAD), (dict(H=1 << 16, W=1 << 15), BAD),
            (dict(B=1 << 30, H=1 << 6, W=1 << 6), BAD), (dict(ldu=1 << 60), BAD)]


@pytest.mark.parametrize("bad,code", SCAN_BAD + [
    (dict(out=None), BAD), (dict(out=1), BAD), (dict(out=5), BAD), (dict(out=9), BAD), (dict(fin=10), BAD),
    (dict(fin=9 * MB + 16), BAD), (dict(fin=11 * MB + 8), BAD), (dict(ws=None), BAD), (dict(wsb=256), BAD),
    (dict(ws=2), BAD), (dict(ws=12 * MB + 4), BAD)])
def test_scan_forward_refusals(lib, bad, code):
    bad = dict(bad)
    a = {k: bad.pop(k, v) for k, v in dict(out=10, fin=11, ws=12, wsb=1 << 23).items()}
    m = scan(**bad)
    assert lib.gtr_ssm_scan_fwd(ctypes.byref(m), P(a["out"]), P(a["fin"]), P(a["ws"]), a["wsb"], None) == code


@pytest.mark.parametrize("bad,code", SCAN_BAD + [
    (dict(grads=None), BAD), (dict(gu=None), BAD), (dict(gz=None), BAD), (dict(gA=None), BAD), (dict(gu=1), BAD),
    (dict(gB=20), BAD), (dict(gA=24 * MB + 4), BAD), (dict(gi=9), BAD), (dict(dy=None), BAD), (dict(ld=7), BAD),
    (dict(df=27 * MB + 8), BAD), (dict(ws=None), BAD), (dict(wsb=1024), BAD), (dict(ws=3), BAD), (dict(ws=30 * MB + 2), BAD)])
def test_scan_backward_refusals(lib, bad, code):
    bad = dict(bad)
    base = dict(dy=18, ld=0, df=19, gu=20, gdt=21, gB=22, gC=23, gz=33, gA=24, gD=25, gt=26, gi=29, ws=30, wsb=1 << 25,
                grads=1)
    a = {k: bad.pop(k, v) for k, v in base.items()}
    m = scan(**bad)
    g = ops_abi.SsmGrads(P(a["gu"]), P(a["gdt"]), P(a["gB"]), P(a["gC"]), P(a["gz"]), P(a["gA"]), P(a["gD"]), P(a["gt"]), P(a["gi"]))
    assert lib.gtr_ssm_scan_bwd(ctypes.byref(m), P(a["dy"]), a["ld"], P(a["df"]), ctypes.byref(g) if a["grads"] else None,
                                P(a["ws"]), a["wsb"], None) == code


NORM_BAD = [dict(B=-1), dict(N=-1), dict(C=0), dict(G=0), dict(G=7), dict(dtype=3), dict(act=-1), dict(x=None),
            dict(x=MB + 1), dict(gamma=2 * MB + 4), dict(beta=3 * MB + 8), dict(ws=None), dict(wsb=128),
            dict(ws=9 * MB + 4), dict(ws=1), dict(N=1 << 30), dict(B=1 << 16, C=1 << 15)]


@pytest.mark.parametrize("bad", NORM_BAD + [dict(eps=-1e-5), dict(eps=float("nan")), dict(eps=float("inf")),
                                            dict(out=None), dict(out=MB + 32), dict(out=2), dict(st=1), dict(st=6 * MB + 4)])
def test_norm_forward_refusals(lib, bad):
    a = dict(x=1, gamma=2, beta=3, B=2, N=100, C=64, G=4, eps=1e-5, dtype=0, act=0, out=5, st=6, ws=9, wsb=1 << 20)
    a.update(bad)
    assert lib.gtr_group_norm_fwd(P(a["x"]), P(a["gamma"]), P(a["beta"]), a["B"], a["N"], a["C"], a["G"], a["eps"],
                                  a["dtype"], a["act"], P(a["out"]), P(a["st"]), P(a["ws"]), a["wsb"], None) == BAD


@pytest.mark.parametrize("bad", NORM_BAD + [dict(dy=None), dict(st=None), dict(gx=None), dict(gx=1), dict(gx=4), dict(gg=5),
                                            dict(gg=7 * MB + 4), dict(gb=7 * MB + 16)])
def test_norm_backward_refusals(lib, bad):
    a = dict(x=1, gamma=2, beta=3, dy=4, st=5, B=2, N=100, C=64, G=4, dtype=0, act=0, gx=6, gg=7, gb=8, ws=9, wsb=1 << 20)
    a.update(bad)
    assert lib.gtr_group_norm_bwd(P(a["x"]), P(a["dy"]), P(a["st"]), P(a["gamma"]), P(a["beta"]), a["B"], a["N"], a["C"],
                                  a["G"], a["dtype"], a["act"], P(a["gx"]), P(a["gg"]), P(a["gb"]), P(a["ws"]), a["wsb"],
                                  None) == BAD


def test_workspace_queries(lib):
    assert ssm.ssm_scan_fwd_workspace_bytes(256, 1, 1, 2048, 16) == 0      # single tokens need none
    assert ssm.ssm_scan_fwd_workspace_bytes(1, 128, 128, 1024, 16) > 0
    assert ssm.ssm_scan_fwd_workspace_bytes(1, 0, 5, 64, 16) == 0
    assert ssm.ssm_scan_fwd_workspace_bytes(1, 4, 4, 64, 33) == 0
    assert ssm.ssm_scan_bwd_workspace_bytes(1, 1, 1, 64, 16) > 0
    assert ssm.ssm_scan_bwd_workspace_bytes(0, 1, 1, 64, 16) == 0
    assert ssm.causal_conv_bwd_workspace_bytes(1, 4, 4, 64, 5) == 0
    assert ssm.causal_conv_bwd_workspace_bytes(1, 4, 4, 64, 4) > 0
    assert norm.group_norm_fwd_workspace_bytes(1, 4, 64, 5) == 0
    assert norm.group_norm_bwd_workspace_bytes(1, 0, 64, 4) == 0


def test_bindings_refuse_host_tensors(lib):
    import torch
    x = torch.zeros(1, 4, 64, dtype=torch.float16)
    f = lambda *s: torch.zeros(s)  # noqa: E731
    b = torch.zeros(1, 4, 16, dtype=torch.float16)
    with pytest.raises(ValueError):
        ssm.gtr_causal_conv_fwd(x, f(64, 4), 2, 2, 0)
    with pytest.raises(ValueError):
        ssm.gtr_causal_conv_bwd(x, f(64, 4), x, 2, 2, 0)
    with pytest.raises(ValueError):
        ssm.gtr_ssm_scan_fwd(x, x, f(64, 16), b, b, 2, 2, 0)
    with pytest.raises(ValueError):
        ssm.gtr_ssm_scan_bwd(x, x, f(64, 16), b, b, x, 2, 2, 0)
    with pytest.raises(ValueError):
        norm.gtr_group_norm_fwd(x, 4)
    with pytest.raises(ValueError):
        norm.gtr_group_norm_bwd(x, x, f(1, 4, 2), 4)


def test_headers_compile_as_c(tmp_path):
    import os
    import subprocess
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    src = tmp_path / "t.c"
    src.write_text('#include "gtr_ssm.h"\n#include "gtr_norm.h"\n'
                   "int main(void){ gtr_conv_t c; gtr_ssm_t m; return (int)(sizeof(c) + sizeof(m)) * 0 + (int)GTR_F16; }\n")
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-I", os.path.join(root, "include"), str(src), "-o",
                    str(tmp_path / "t")], check=True)
