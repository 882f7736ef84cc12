"""Which kernels the calls of the 8-bit experts launch, asked on the CPU: the library's host code
linked with launch functions that note a kernel's name (tests/sanitize/experts8_choice_driver.cpp).
The GPU tests' cases take the kernels that they are meant for, and every kernel has one."""
import os
import subprocess

import pytest

import test_gpu_experts8 as base
import test_gpu_experts8_kernels as named
import test_gpu_experts8_paths as paths
from test_sanitize import CLANGXX, CSRC, HERE, HIPCC, ROOT, _run

pytestmark = pytest.mark.skipif(not (os.path.exists(HIPCC) and os.path.exists(CLANGXX)),
                                reason="the ROCm compilers are needed")
TYPE = {"f32": 0, "bf16": 1, "i8": 2}


@pytest.fixture(scope="module")
def driver(tmp_path_factory):
    d = tmp_path_factory.mktemp("choice")
    objs = []
    for src in ("i8_gemv.hip", "moe_rows.hip"):
        objs.append(str(d / (src + ".o")))
        _run([HIPCC, "-c", "-O1", "-std=c++17", "--offload-arch=gfx950", "--offload-host-only",
              "-I", os.path.join(ROOT, "include"), os.path.join(CSRC, src), "-o", objs[-1]], 300)
    exe = str(d / "driver")
    # the kernels' own code is left out
    _run([CLANGXX, "-O1", "-std=c++17", "-D__HIP_PLATFORM_AMD__=1", "-I/opt/rocm/include",
          os.path.join(HERE, "experts8_choice_driver.cpp"), *objs,
          "-Wl,--unresolved-symbols=ignore-all", "-o", exe], 300)
    return exe


def ask(driver, queries):
    """(all kernels, for each query its [(kernel, workgroups)])"""
    r = subprocess.run([driver], input="".join(q + "\n" for q in queries), capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stderr[-2000:]
    lines = r.stdout.split("\n")
    assert len(lines) == len(queries) + 2
    split = [[(k[:k.rindex(" ")], int(k[k.rindex(" "):])) for k in line.split("\t")[1:]] for line in lines[1:-1]]
    return set(lines[0].split("\t")[1:]), split


def gemv(N, M, K, E=None, ldx=None, ldy=None, s="f32", y="f32", w_offset=0, x_offset=0):
    return (f"gemv {E or 1} {int(E is not None)} {N} {M} {K} {ldx or K} {ldy or M} {TYPE[s]} {TYPE[y]} "
            f"{w_offset} {x_offset}")


def named_cases():
    """(kernel, query) of test_gpu_experts8_kernels"""
    out = [(k, gemv(N, M, K, s=s, y=y)) for k, N, M, K in named.ONE for s, y in named.TYPES]
    for i, (k, counts, behind, M, K) in enumerate(named.MANY):
        s, y = named.many_types(i)
        out.append((k, gemv(sum(counts) + behind, M, K, E=len(counts), s=s, y=y)))
    return out


def gemv_cases():
    """the product's calls of the other GPU tests"""
    out = [gemv(N, M, K, s=t, y=t) for N, M, K in base.SIZES for t in ("f32", "bf16")]
    out += [gemv(sum(c) + b, M, K, E=len(c), ldy=M + 2, s=t, y=t) for c, b, M, K in base.GROUPS for t in ("f32", "bf16")]
    for N, M, K in paths.FEW + paths.MID + paths.WIDE:
        for more in (0, 4, 8, 3):
            s, y = ("f32", "bf16")[(N + more // 4) % 2], ("bf16", "f32")[(N + M + more // 4) % 2]
            out.append(gemv(N, M, K + more, s=s, y=y))
    for i, (c, b, M, K) in enumerate(paths.GROUPED):
        for more in (0, 4, 1):
            s, y = ("f32", "bf16")[i % 2], ("bf16", "f32")[(i // 2 + more) % 2]
            out.append(gemv(sum(c) + b, M, K + more, E=len(c), ldy=M + 2, s=s, y=y))
    return out


def test_named_cases_take_their_kernels(driver):
    cases = named_cases()
    for (kernel, query), took in zip(cases, ask(driver, [q for _, q in cases])[1]):
        assert [k[:len(kernel)] for k, _ in took] == [kernel], (kernel, query, took)


def test_every_kernel_of_the_product_has_a_case(driver):
    every, took = ask(driver, gemv_cases() + [q for _, q in named_cases()])
    every = {k for k in every if k.startswith("k_i8")}
    assert len(every) > 30
    assert every == {k for t in took for k, _ in t}


def test_every_kernel_of_the_rows_has_a_case(driver):
    q = [f"sort {T} {k} {E} {H} {TYPE[x]}" for T, k, E, _ in base.ROUTES for x, H in (("bf16", 64), ("f32", 37), ("i8", 100))]
    q += [f"unsort {T} {k} {H} {TYPE[r]} {TYPE[y]}" for T, k, _, H in base.BACK for r in ("f32", "bf16") for y in ("f32", "bf16")]
    q += [f"grad {T} {k} {H} {TYPE[y]} {TYPE[r]}" for T, k, _, H in base.BACK for r in ("f32", "bf16") for y in ("f32", "bf16")]
    wide = [(1, 1), (64, 512), (65, 513), (20, 2048), (9, 2055), (5, 4100), (4, 8192), (3, 8200)]    # test_swiglu's
    codes = [(7, 5), (64, 1024), (30, 513), (9, 2049), (5, 4096), (3, 8191), (2, 9000)]              # test_swiglu_codes'
    q += [f"swiglu {N} {I} {TYPE[x]} {TYPE[o]}" for N, I in wide for x in ("bf16", "f32") for o in ("bf16", "f32")]
    q += [f"swiglu {N} {I} {TYPE[x]} {TYPE['i8']}" for N, I in codes for x in ("bf16", "f32")]
    every, took = ask(driver, q)
    every = {k for k in every if not k.startswith("k_i8")}
    assert len(every) > 20
    assert every == {k for t in took for k, _ in t}


def test_grids_that_hip_takes(driver):
    """The largest calls: no grid of more than 2^22 workgroups of 256 threads, and all tiles in them."""
    _, took = ask(driver, [gemv(1 << 30, 1 << 30, 1), gemv(1 << 30, 128, 64, E=4096), gemv(1, 1 << 30, 64),
                           gemv(1 << 30, 64, 65), "swiglu 1000000000 64 1 1", "sort 1000000 8 100 64 1"][1:])
    for t in took:
        assert t and all(0 < n <= 1 << 22 for _, n in t), t[:3]
    assert sum(n for _, n in took[1]) >= (1 << 30) // 64


# calls on both sides of a rule, and the kernel that is faster there
BORDERS = [
    (gemv(33, 4090, 4096), "k_i8_rows<2, 2"), (gemv(33, 4130, 4096), "k_i8_rows<2, 4"),      # 256 and 260 workgroups
    (gemv(96, 2720, 4096), "k_i8_rows<2, 2"), (gemv(61, 4500, 4150), "k_i8_rows<2, 4"),
    (gemv(1536, 8192, 1024), "k_i8_mid<2, 2"), (gemv(1536, 8192, 2048), "k_i8_wide"),        # 192 tiles
    (gemv(1792, 8192, 1024), "k_i8_wide"), (gemv(2304, 8192, 512), "k_i8_mid<2, 2"),         # 224, 288
    (gemv(2304, 8192, 4096), "k_i8_wide"), (gemv(3584, 8192, 512), "k_i8_wide"),             # 288, 448
    (gemv(200, 800, 4096, E=4), "k_i8_rows<2, 2"), (gemv(120, 1900, 4096, E=2), "k_i8_rows<2, 4"),
]


def test_rules_at_their_borders(driver):
    for (query, kernel), took in zip(BORDERS, ask(driver, [q for q, _ in BORDERS])[1]):
        assert [k[:len(kernel)] for k, _ in took] == [kernel], (query, kernel, took)
