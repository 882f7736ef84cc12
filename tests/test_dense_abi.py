"""CPU checks of the dense operators around the routed layer: every refusal of their C calls
and of their Python binding, before anything is launched (no GPU needed)."""
import ctypes

import pytest

F = 0x100000   # aligned address that is never dereferenced: validation fails first
F32, BF16, I8 = 0, 1, 2


@pytest.fixture(scope="module")
def sm():
    from pseudo_random_weight_amd import seedmm
    return seedmm


def q4(sm, w=F, s=F, b=F, sd=BF16, group=64, x=F, xd=BF16, ldx=128, xs=None, y=F, yd=F32, ldy=16,
       M=16, K=128, N=1, ws=F, wsb=1 << 40):
    return sm.lib().seedmm_q4_gemv(w, s, b, sd, group, x, xd, ldx, xs, y, yd, ldy, M, K, N, ws, wsb, None)


@pytest.mark.parametrize("kw,expect", [
    (dict(group=16), -1), (dict(group=0), -1), (dict(group=256, K=256, ldx=256), -1),
    (dict(K=96), -1), (dict(K=96, group=128), -1),
    (dict(M=-1), -1), (dict(K=-64), -1), (dict(N=-1), -1),
    (dict(M=(1 << 30) + 1, ldy=(1 << 30) + 1), -1), (dict(K=(1 << 30) + 64, ldx=(1 << 30) + 64), -1),
    (dict(N=(1 << 30) + 1), -1),
    (dict(ldx=127), -1), (dict(ldy=15), -1),
    (dict(sd=I8), -1), (dict(yd=I8), -1), (dict(xd=3), -1), (dict(sd=-1), -1),
    (dict(w=None), -1), (dict(s=None), -1), (dict(b=None), -1), (dict(x=None), -1), (dict(y=None), -1),
    (dict(xd=I8), -1), (dict(xs=F), -1),
    (dict(w=F + 8), -2), (dict(x=F + 8), -2), (dict(s=F + 1), -2), (dict(b=F + 2, sd=F32), -2),
    (dict(y=F + 2), -2), (dict(y=F + 1, yd=BF16), -2), (dict(xd=I8, xs=F + 2), -2),
    (dict(N=2, ldx=132), -2), (dict(N=2, xd=F32, ldx=130), -2), (dict(N=2, xd=I8, xs=F, ldx=136), -2),
    (dict(N=17, K=2048, ldx=2048, ws=None), -3), (dict(N=17, K=2048, ldx=2048, wsb=100), -3),
    (dict(N=6, xd=F32, ws=None), -3), (dict(N=17, K=2048, ldx=2048, xd=I8, xs=F, ws=None, wsb=0), -3),
    (dict(N=17, K=2048, ldx=2048, ws=F + 8), -2),
    (dict(M=0, ldy=0, w=None, y=None), 0), (dict(N=0, x=None, y=None), 0),
])
def test_q4_gemv_refusals(sm, kw, expect):
    assert q4(sm, **kw) == expect


def test_q4_workspace_sizes(sm):
    f = sm.lib().seedmm_q4_workspace_bytes
    assert [f(BF16, 64, 100, 2048, n) for n in (0, 1, 16)] == [0, 0, 0]
    assert f(F32, 64, 100, 2048, 5) == 0 and f(F32, 64, 100, 2048, 6) >= 3 * 6 * 2048 * 2
    # partial sums of at least two splits; laid-out rows of a prompt
    assert f(BF16, 64, 100, 2048, 17) >= 2 * 17 * 100 * 4 and f(I8, 64, 100, 2048, 17) >= 2 * 17 * 100 * 4
    assert f(BF16, 64, 100, 64, 17) == 0
    assert f(BF16, 64, 8192, 2048, 4096) >= 4096 * 2048 * 2
    assert f(BF16, 48, 100, 2048, 17) == 0 and f(BF16, 64, -1, 2048, 17) == 0
    assert f(BF16, 64, 100, 2049, 17) == 0 and f(BF16, 64, 0, 2048, 17) == 0
    assert f(BF16, 64, 1 << 20, 1 << 20, 1 << 20) >= 2 ** 41    # no 32-bit size


def norm(sm, x=F, xd=BF16, ldx=64, d=F, dd=F32, ldd=64, w=F, wd=BF16, eps=1e-6, res=F, ldr=64,
         out=F, od=BF16, ldo=64, sc=None, N=2, H=64):
    return sm.lib().seedmm_add_norm(x, xd, ldx, d, dd, ldd, w, wd, eps, res, ldr, out, od, ldo, sc,
                                    N, H, None)


@pytest.mark.parametrize("kw,expect", [
    (dict(N=-1), -1), (dict(H=-1), -1), (dict(ldx=63), -1), (dict(ldd=63), -1), (dict(ldr=63), -1),
    (dict(ldo=63), -1), (dict(xd=I8), -1), (dict(dd=I8), -1), (dict(wd=I8), -1), (dict(od=3), -1),
    (dict(eps=-1e-6), -1), (dict(eps=float("nan")), -1), (dict(eps=float("inf")), -1),
    (dict(od=I8), -1), (dict(sc=F), -1), (dict(x=None), -1), (dict(out=None), -1),
    (dict(x=F + 1), -2), (dict(x=F + 2, xd=F32), -2), (dict(d=F + 2), -2), (dict(w=F + 1), -2),
    (dict(res=F + 1), -2), (dict(out=F + 1), -2), (dict(od=I8, sc=F + 2), -2),
    (dict(N=0, x=None, out=None, res=None), 0), (dict(H=0, x=None, out=None), 0),
])
def test_add_norm_refusals(sm, kw, expect):
    assert norm(sm, **kw) == expect


def route(sm, lg=F, dt=F32, ldl=16, bias=None, score=0, T=2, E=16, k=4, ids=F, w=F):
    return sm.lib().seedmm_route(lg, dt, ldl, bias, score, T, E, k, ids, w, None)


@pytest.mark.parametrize("kw,expect", [
    (dict(T=-1), -1), (dict(E=0), -1), (dict(E=4097, ldl=4097), -1), (dict(k=0), -1), (dict(k=17), -1),
    (dict(E=100, ldl=100, k=65), -1), (dict(T=1 << 25, E=100, ldl=100, k=64), -1), (dict(ldl=15), -1),
    (dict(dt=I8), -1), (dict(score=2), -1), (dict(bias=F), -1), (dict(lg=None), -1),
    (dict(ids=None), -1), (dict(w=None), -1),
    (dict(lg=F + 2), -2), (dict(lg=F + 1, dt=BF16), -2), (dict(score=1, bias=F + 1), -2),
    (dict(ids=F + 2), -2), (dict(w=F + 2), -2), (dict(T=0, lg=None, ids=None, w=None), 0),
])
def test_route_refusals(sm, kw, expect):
    assert route(sm, **kw) == expect


def make_block(sm, **kw):
    m = sm.SeedMat(F, F, F, F)
    v = dict(norm_weight=F, router_weight=F, router_scales=F, router_biases=F, router_bias=None,
             p4mask=None, gate=m, up=m, down=m, eps=1e-6, norm_dtype=BF16, router_dtype=BF16,
             group=64, score=0, top_k=2, E=8, H=64, I=32, P=4)
    v.update(kw)
    b = sm.SeedBlock()
    for k, x in v.items():
        setattr(b, k, x)
    return b


def run_block(sm, b, r=F, rd=BF16, d=F, dd=F32, y=F, ids=None, w=None, T=4, ws=F, wsb=None, st=None,
              side=None):
    L = sm.lib()
    if wsb is None:
        wsb = max(L.seedmm_moe_block_workspace_bytes(ctypes.byref(b), T), 1)
    return L.seedmm_moe_block(ctypes.byref(b), r, rd, d, dd, y, ids, w, T, ws, wsb, st,
                              None if side is None else ctypes.byref(side))


@pytest.mark.parametrize("bkw,kw,expect", [
    (dict(P=5), {}, -1), (dict(P=0), {}, -1), (dict(P=4, p4mask=F), {}, -1), (dict(top_k=9), {}, -1),
    (dict(top_k=0), {}, -1), (dict(E=0), {}, -1), (dict(H=72), {}, -1), (dict(group=48), {}, -1),
    (dict(I=12), {}, -1), (dict(score=3), {}, -1), (dict(router_bias=F), {}, -1),
    (dict(eps=-1.0), {}, -1), (dict(norm_dtype=I8), {}, -1), (dict(router_dtype=I8), {}, -1),
    (dict(router_weight=None), {}, -1), (dict(router_scales=None), {}, -1),
    ({}, dict(T=-1, wsb=1 << 20), -1), ({}, dict(rd=I8), -1), ({}, dict(dd=I8), -1),
    ({}, dict(r=None), -1), ({}, dict(y=None), -1),
    ({}, dict(r=F + 2), -2), ({}, dict(d=F + 4), -2), ({}, dict(y=F + 4), -2), ({}, dict(ids=F + 2), -2),
    ({}, dict(ws=F + 4), -2), (dict(router_weight=F + 4), {}, -2), (dict(norm_weight=F + 2), {}, -2),
    ({}, dict(ws=None), -3), ({}, dict(wsb=64), -3),
    ({}, dict(T=0, r=None, y=None, ws=None), 0),
])
def test_moe_block_refusals(sm, bkw, kw, expect):
    assert run_block(sm, make_block(sm, **bkw), **kw) == expect


def test_moe_block_refuses_a_missing_expert_stream_and_a_bad_side(sm):
    for name in ("gate", "up", "down"):
        assert run_block(sm, make_block(sm, **{name: sm.SeedMat(F, None, F, F)})) == -1
    b = make_block(sm)
    assert run_block(sm, b, side=sm.SeedSide(F + 256, None, F), st=F) == -1
    assert run_block(sm, b, side=sm.SeedSide(F, F, F), st=F) == -1
    L = sm.lib()
    assert L.seedmm_moe_block(None, F, BF16, None, 0, F, None, None, 4, F, 1 << 20, None, None) == -1
    assert L.seedmm_moe_block_workspace_bytes(None, 4) == 0
    assert L.seedmm_moe_block_workspace_bytes(ctypes.byref(make_block(sm, top_k=0)), 4) == 0
    small = L.seedmm_moe_block_workspace_bytes(ctypes.byref(b), 4)
    assert small >= L.seedmm_moe_workspace_bytes(4, 2, 8, 64, 32) + 4 * 64 * 2 + 4 * 8 * 4 + 2 * 4 * 2 * 4
    assert L.seedmm_moe_block_workspace_bytes(ctypes.byref(b), 400) > small


def test_binding_refuses_cpu_tensors_and_bad_shapes(sm):
    import torch
    x = torch.zeros(2, 64, dtype=torch.bfloat16)
    with pytest.raises(TypeError, match="x must be a CUDA"):
        sm.add_norm(x)
    with pytest.raises(TypeError, match="x must be a CUDA"):
        sm.q4_gemv({}, x, 16, 64)
    with pytest.raises(TypeError, match="x must be a CUDA"):
        sm.q4_gemv({"weight": x, "scales": x, "biases": x}, x, 16, 64, y=x)
    with pytest.raises(TypeError, match="x must be a CUDA"):
        sm.add_norm(x, out=x)
    with pytest.raises(TypeError, match="logits must be a CUDA"):
        sm.route(x, 4, ids=x, w=x)
    with pytest.raises(TypeError, match="logits must be a CUDA"):
        sm.route(torch.zeros(2, 16), 4)
    with pytest.raises(TypeError, match="logits must be a CUDA"):
        sm.route(None, 4)


def test_binding_module_counts_arguments(sm):
    for f in (sm._binding.q4_gemv, sm._binding.add_norm, sm._binding.route):
        with pytest.raises(TypeError, match="arguments are needed"):
            f(None)


def test_moe_block_refuses_too_many_tokens_before_its_first_launch(sm):
    """The product takes 2^30 - 64 tokens; a block of more may not have added delta to r when
    it says so (a launch would give -4 here)."""
    b = make_block(sm, top_k=1, H=64, I=32)
    for T in (1 << 30, (1 << 30) - 63):
        assert run_block(sm, b, T=T, wsb=1 << 62) == -1


def test_the_library_imports_without_the_dense_binding(tmp_path):
    """Callers of the seed-coded products need libseedmm.so alone: a package without _binding.so
    (or with one that another torch was built for) imports, answers, and names the file at
    the first dense call."""
    import os
    import subprocess
    import sys

    import pseudo_random_weight_amd as pkg
    here, there = os.path.dirname(pkg.__file__), tmp_path / "pseudo_random_weight_amd"
    there.mkdir()
    for f in os.listdir(here):
        if f.endswith(".py") or f == "libseedmm.so":
            os.symlink(os.path.join(here, f), there / f)
    code = """
import torch
from pseudo_random_weight_amd import seedmm as sm
assert sm.moe_workspace_bytes(4, 2, 8, 64, 32) > 0 and sm.q4_workspace_bytes(torch.float32, 64, 100, 2048, 6) > 0
x = torch.zeros(2, 8)
for call in (lambda: sm.route(x, 2, ids=x, w=x), lambda: sm.add_norm(x, out=x), lambda: sm._binding,
             lambda: sm.q4_gemv({"weight": x, "scales": x, "biases": x}, x, 16, 64, y=x)):
    try:
        call()
    except ImportError as e:
        assert "_binding" in str(e)
    else:
        raise SystemExit("a dense call without its module")
print("imported")
"""
    run = [sys.executable, "-c", code]
    env = dict(os.environ, PYTHONPATH=str(tmp_path))
    for text in (None, b"no library"):
        if text:
            (there / "_binding.so").write_bytes(text)
        res = subprocess.run(run, cwd=tmp_path, env=env, capture_output=True, text=True, timeout=300)
        assert "imported" in res.stdout, res.stderr


@pytest.mark.parametrize("kw,expect", [
    (dict(ldr=72), -1), (dict(ldx=72), -1), (dict(ldx=72, ldr=72, d=F + 1, dd=F32), -2),
    (dict(ldr=72, N=1, d=F + 1), -2), (dict(ldr=72, res=F + 0x1000, d=F + 1), -2),
])
def test_add_norm_in_place_takes_one_row_stride(sm, kw, expect):
    """x as residual with another row stride would write rows that others still read.  (-2, of
    a misaligned delta, stands for a call that passes this check.)"""
    assert norm(sm, **kw) == expect
