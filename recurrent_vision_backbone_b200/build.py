"""Build the CUDA library in-tree, recurrent_vision_backbone_b200/libgtr_gla.so, and the
extension module that hands it torch tensors, recurrent_vision_backbone_b200/_ops.so.

The library needs nvcc alone and serves the C ABI by itself; the module (for ``ssm`` and ``norm``) is
left out, with a note, where torch, g++ or Python's headers are missing.

Compiles the csrc/*.cu sources for sm_100a only (nvcc cross-compiles without a GPU):
    python -m recurrent_vision_backbone_b200.build [--verbose]
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
import sysconfig
import tempfile

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
SOURCES = [os.path.join(CSRC, n) for n in ("gtr_gla.cu", "causal_conv.cu", "ssm_scan.cu", "ssm_scan_bwd.cu", "group_norm.cu")]
DEPS = SOURCES + [os.path.join(CSRC, n) for n in ("sm100_ptx.cuh", "gla_fwd_span.cuh", "gla_fwd_pipe.cuh", "swiglu_gate.cuh", "gla_bwd.cuh",
                                                  "ops_common.cuh", "ops_errors.h", "causal_conv.cuh", "ssm_scan.cuh", "ssm_scan_bwd.cuh",
                                                  "ssm_host.cuh")]
DEPS += [os.path.join(ROOT, "include", n) for n in ("gtr_gla.h", "gtr_swiglu.h", "gtr_gla_bwd.h", "gtr_ops.h", "gtr_ssm.h",
                                                    "gtr_norm.h")]
LIB = os.path.join(HERE, "libgtr_gla.so")
BINDING_SOURCE = os.path.join(CSRC, "binding.cpp")
BINDING_DEPS = [BINDING_SOURCE] + [os.path.join(ROOT, "include", n) for n in ("gtr_gla.h", "gtr_ops.h", "gtr_ssm.h", "gtr_norm.h")]
BINDING = os.path.join(HERE, "_ops.so")


def nvcc_path() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def nvcc_cmd(out: str = LIB, extra=(), inputs=None) -> list:
    """The command that compiles and links `inputs` (all sources by default) into `out`."""
    return [nvcc_path(), "-gencode", "arch=compute_100a,code=sm_100a", "-lineinfo", "-O3",
            "-std=c++17", "--shared", "-Xcompiler", "-fPIC", "-I", os.path.join(ROOT, "include"),
            *extra, *(SOURCES if inputs is None else inputs), "-o", out, "-lcudart"]


def compile_cmd(src: str, obj: str, extra=()) -> list:
    """The command that compiles one source (the options of nvcc_cmd)."""
    return [nvcc_path(), "-gencode", "arch=compute_100a,code=sm_100a", "-lineinfo", "-O3",
            "-std=c++17", "-Xcompiler", "-fPIC", "-I", os.path.join(ROOT, "include"), *extra,
            "-c", src, "-o", obj]


def binding_missing() -> str | None:
    """What the extension module needs and this machine lacks, or None."""
    try:
        import torch  # noqa: F401
    except ImportError:
        return "torch"
    if shutil.which("g++") is None:
        return "g++"
    if not os.path.exists(os.path.join(sysconfig.get_paths()["include"], "Python.h")):
        return "Python.h"
    return None


def binding_cmd(out: str) -> list:
    """The command that compiles the extension module against the installed torch and links it to
    the CUDA library beside it."""
    import torch
    base = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(nvcc_path()))
    inc = [os.path.join(ROOT, "include"), os.path.join(base, "include"),
           os.path.join(base, "include", "torch", "csrc", "api", "include"), os.path.join(cuda, "include"),
           sysconfig.get_paths()["include"]]
    return ["g++", "-O2", "-std=c++17", "-shared", "-fPIC", *(a for i in inc for a in ("-I", i)), BINDING_SOURCE, "-o", out,
            "-L", HERE, "-l:libgtr_gla.so", "-L", os.path.join(base, "lib"), "-ltorch_python", "-ltorch", "-ltorch_cpu",
            "-lc10", "-lc10_cuda", "-Wl,-rpath,$ORIGIN"]


def is_stale(out: str = LIB, deps=None) -> bool:
    if not os.path.exists(out):
        return True
    t = os.path.getmtime(out)
    return any(os.path.getmtime(d) > t for d in (DEPS if deps is None else deps))


def binding_version() -> str:
    """What the extension module is compiled against (kept beside it)."""
    import torch
    return f"torch {torch.__version__}, Python {sys.version}\n"


def binding_is_stale() -> bool:
    """Whether the extension module is missing, older than its sources or made for another torch or Python."""
    if is_stale(BINDING, BINDING_DEPS) or not os.path.exists(BINDING + ".version"):
        return True
    with open(BINDING + ".version") as f:
        return f.read() != binding_version()


def build(force: bool = False, verbose: bool = False) -> str:
    if force or is_stale():
        extra = ["-Xptxas", "-v"] if verbose else []
        tmp = LIB + ".tmp"
        with tempfile.TemporaryDirectory() as work:   # the sources side by side, then one link
            objs = [os.path.join(work, os.path.basename(s) + ".o") for s in SOURCES]
            procs = [subprocess.Popen(compile_cmd(s, o, extra)) for s, o in zip(SOURCES, objs)]
            codes = [p.wait() for p in procs]
            if any(codes):
                raise subprocess.CalledProcessError(max(codes, key=abs), "nvcc")
            subprocess.run(nvcc_cmd(tmp, inputs=objs), check=True)
        os.replace(tmp, LIB)
    missing = binding_missing()
    if missing is not None:
        print(f"{os.path.basename(BINDING)} not built: {missing} is missing (the ssm and norm modules need it)",
              file=sys.stderr)
    elif force or binding_is_stale():
        tmp = BINDING + ".tmp"
        subprocess.run(binding_cmd(tmp), check=True)
        os.replace(tmp, BINDING)
        with open(BINDING + ".version", "w") as f:
            f.write(binding_version())
    return LIB


if __name__ == "__main__":
    print(build(force=True, verbose="--verbose" in sys.argv))
