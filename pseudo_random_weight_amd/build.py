"""Build the HIP library libseedmm.so for gfx950 and the Python module _binding in-tree.

    python -m pseudo_random_weight_amd.build
"""
from __future__ import annotations

import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
SO = os.path.join(HERE, "libseedmm.so")
BINDING = os.path.join(HERE, "_binding.so")
SOURCES = [os.path.join(CSRC, "seedmm.hip"), os.path.join(CSRC, "search.hip"),
           os.path.join(CSRC, "expert_cache.hip"), os.path.join(CSRC, "dense.hip"),
           os.path.join(CSRC, "i8_gemv.hip"), os.path.join(CSRC, "moe_rows.hip")]
HEADERS = [os.path.join(CSRC, "seed_decode.hpp"), os.path.join(CSRC, "moe_layer.hpp"),
           os.path.join(CSRC, "device_rows.hpp"),
           os.path.join(ROOT, "include", "seedmm.h")]

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
ARCH = "gfx950"
FLAGS = [
    "-O3", "-std=c++17", "-fPIC", "-shared", f"--offload-arch={ARCH}",
    # no packed fp32 instructions in any device code
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-I", os.path.join(ROOT, "include"),
    "-Wno-unused-command-line-argument",
    # keep per-thread arrays in registers (the LDS budget belongs to the kernels' tiles)
    "-mllvm", "-disable-promote-alloca-to-lds",
]


def _run(cmd, out, verbose):
    tmp = out + ".tmp"
    cmd = [*cmd, "-o", tmp]
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        sys.stderr.write(res.stdout + res.stderr)
        raise RuntimeError(f"{os.path.basename(cmd[0])} failed building {os.path.basename(out)}")
    os.replace(tmp, out)


def binding_command() -> list:
    """The host compiler's command for _binding (argument checks on torch's tensors)."""
    import sysconfig

    import torch
    from torch.utils.cpp_extension import include_paths
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    inc = [*include_paths(), sysconfig.get_paths()["include"], "/opt/rocm/include"]
    return ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-w", "-D__HIP_PLATFORM_AMD__=1",
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
            *(f"-I{d}" for d in inc), os.path.join(CSRC, "binding.cpp"), f"-L{lib}",
            f"-Wl,-rpath,{lib}", "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_hip"]


def build(verbose: bool = False) -> str:
    _run([HIPCC, *FLAGS, *SOURCES], SO, verbose)
    _run(binding_command(), BINDING, verbose)
    return SO


if __name__ == "__main__":
    print(build(verbose=True))
