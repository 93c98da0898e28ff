"""Build libmoedisp.so (gfx950) from csrc/ with hipcc, in-tree, and the Python
binding's argument checks (_checks.so) with the host compiler."""
from __future__ import annotations

import os
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(HERE, "libmoedisp.so")
SOURCES = ["capi.hip", "layout.hip", "notify.hip", "dispatch.hip", "decode.hip", "combine.hip", "util.hip",
           "capi_experts.hip", "expert_gemm.hip", "expert_wgrad.hip", "expert_gemm_bf16.hip",
           "expert_wgrad_bf16.hip", "expert_gemm_w4.hip", "swiglu.hip", "balance.hip", "router.hip"]

HIPCC_FLAGS = [
    "--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC", "-shared",
    # no packed fp32 instructions in device code
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall", "-Wno-unused-command-line-argument",
]


def hipcc() -> str:
    rocm = os.environ.get("ROCM_PATH", "/opt/rocm")
    return os.path.join(rocm, "bin", "hipcc")


def build(out: str = LIB, extra_flags=(), verbose: bool = False) -> str:
    srcs = [os.path.join(CSRC, s) for s in SOURCES]
    tmp = out + ".tmp"
    cmd = [hipcc(), *HIPCC_FLAGS, *extra_flags, "-I", INCLUDE, "-I", CSRC, "-o", tmp, *srcs]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.run(cmd, check=True)
    os.replace(tmp, out)
    return out


CHECKS = os.path.join(HERE, "_checks.so")


def build_checks(out: str = CHECKS, verbose: bool = False) -> str | None:
    """The binding works without it, more slowly: where the host compiler or
    torch's headers are missing this says so, takes away what an earlier build
    left, and returns None."""
    try:
        return _build_checks(out, verbose)
    except (ImportError, AttributeError, OSError, subprocess.CalledProcessError) as e:
        print(f"{os.path.basename(out)} was not built ({e}): the binding checks its arguments in Python", file=sys.stderr)
        for left in (out, out + ".tmp"):
            if os.path.exists(left):
                os.remove(left)
        return None


def _build_checks(out: str, verbose: bool) -> str:
    import torch
    from torch.utils import cpp_extension
    inc = [f"-I{p}" for p in [sysconfig.get_paths()["include"], *cpp_extension.include_paths()]]
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = out + ".tmp"
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}",
           f'-DMOEDISP_BUILT_FOR="{torch.version.__version__} {torch.version.git_version}"', *inc, "-o", tmp,
           os.path.join(CSRC, "checks.cpp"), f"-L{lib}", "-ltorch_python", "-ltorch_cpu", "-ltorch", "-lc10",
           f"-Wl,-rpath,{lib}"]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.run(cmd, check=True)
    os.replace(tmp, out)
    return out


if __name__ == "__main__":
    print(build(verbose=True))
    print(build_checks(verbose=True))
