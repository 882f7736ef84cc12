"""AddressSanitizer + UBSan build of the host code of the 8-bit experts (no GPU needed), run
on its argument checks and size functions by tests/sanitize/experts8_driver.cpp."""
import os

import pytest

from test_sanitize import CLANGXX, CSRC, HERE, HIPCC, ROOT, SAN_ENV, _run


@pytest.mark.skipif(not (os.path.exists(HIPCC) and os.path.exists(CLANGXX)),
                    reason="the ROCm compilers are needed")
def test_experts8_host_code_under_address_and_undefined_sanitizers(tmp_path):
    objs = []
    for src in ("seedmm.hip", "i8_gemv.hip", "moe_rows.hip"):
        obj = str(tmp_path / (src + ".o"))
        # host code instrumented; device code compiled as usual (never run here)
        _run([HIPCC, "-c", "-O1", "-g", "-std=c++17", "--offload-arch=gfx950",
              "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
              "-mllvm", "-disable-promote-alloca-to-lds",
              "-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
              "-Xarch_host", "-fno-omit-frame-pointer", "-Xarch_host", "-fno-sanitize-recover=all",
              "-I", os.path.join(ROOT, "include"), os.path.join(CSRC, src), "-o", obj], 900)
        objs.append(obj)
    exe = str(tmp_path / "experts8_driver")
    _run([CLANGXX, "-O1", "-g", "-std=c++17", "-fsanitize=address,undefined",
          "-fno-omit-frame-pointer", "-fno-sanitize-recover=all",
          "-I", os.path.join(ROOT, "include"), os.path.join(HERE, "experts8_driver.cpp"), *objs,
          "-L/opt/rocm/lib", "-lamdhip64", "-Wl,-rpath,/opt/rocm/lib", "-o", exe], 300)
    assert "clean" in _run([exe], 300, SAN_ENV)
