"""CPU checks of the operators of 8-bit experts: every refusal of their C calls and of their
Python binding, before anything is launched, and the sizes of their workspaces (no GPU
needed)."""
import pytest

F = 0x100000   # aligned address that is never dereferenced: validation fails first
F32, BF16, I8 = 0, 1, 2


@pytest.fixture(scope="module")
def sm():
    from pseudo_random_weight_amd import seedmm
    return seedmm


def gemv(sm, w=F, s=F, sd=F32, E=1, off=None, x=F, ldx=64, xs=F, y=F, yd=F32, ldy=16, M=16, K=64, N=2):
    return sm.lib().seedmm_i8_gemv(w, s, sd, E, off, x, ldx, xs, y, yd, ldy, M, K, N, None)


@pytest.mark.parametrize("kw,expect", [
    (dict(M=-1), -1), (dict(K=-1), -1), (dict(N=-1), -1), (dict(M=(1 << 30) + 1, ldy=1 << 31), -1),
    (dict(N=(1 << 30) + 1), -1), (dict(K=131072, ldx=131072), -1), (dict(E=0, off=F), -1),
    (dict(E=4097, off=F), -1), (dict(E=2), -1), (dict(ldx=63), -1), (dict(ldy=15), -1),
    (dict(sd=I8), -1), (dict(sd=-1), -1), (dict(yd=I8), -1), (dict(yd=3), -1),
    (dict(w=None), -1), (dict(s=None), -1), (dict(x=None), -1), (dict(xs=None), -1), (dict(y=None), -1),
    (dict(s=F + 2), -2), (dict(s=F + 1, sd=BF16), -2), (dict(xs=F + 2), -2), (dict(off=F + 2), -2),
    (dict(y=F + 2), -2), (dict(y=F + 1, yd=BF16), -2),
    (dict(M=0, ldy=0, w=None, s=None, y=None), 0), (dict(N=0, x=None, xs=None, y=None), 0),
])
def test_i8_gemv_refusals(sm, kw, expect):
    assert gemv(sm, **kw) == expect


def sort(sm, ids=F, T=4, k=2, E=8, x=F, xd=BF16, ldx=64, xs=None, rows=F, ldr=64, rs=None, H=64, off=F,
         inv=F, ws=F, wsb=1 << 40):
    return sm.lib().seedmm_moe_sort(ids, T, k, E, x, xd, ldx, xs, rows, ldr, rs, H, off, inv, ws, wsb, None)


@pytest.mark.parametrize("kw,expect", [
    (dict(T=-1), -1), (dict(k=0), -1), (dict(k=65), -1), (dict(T=1 << 26, k=64), -1), (dict(E=0), -1),
    (dict(E=4097), -1), (dict(H=-1), -1), (dict(H=(1 << 30) + 1, ldx=1 << 31, ldr=1 << 31), -1),
    (dict(ldx=63), -1), (dict(ldr=63), -1), (dict(xd=3), -1), (dict(xd=-1), -1),
    (dict(xs=F), -1), (dict(rs=F), -1), (dict(ids=None), -1), (dict(x=None), -1), (dict(rows=None), -1),
    (dict(off=None), -1), (dict(off=None, T=0), -1), (dict(inv=None), -1),
    (dict(ids=F + 2), -2), (dict(off=F + 2), -2), (dict(inv=F + 2), -2), (dict(x=F + 1), -2),
    (dict(rows=F + 1), -2), (dict(x=F + 2, xd=F32), -2), (dict(xs=F + 2, rs=F), -2), (dict(xs=F, rs=F + 2), -2),
    (dict(T=4096, k=8, ws=None), -3), (dict(T=4096, k=8, wsb=100), -3), (dict(T=4096, k=8, ws=F + 8), -2),
])
def test_moe_sort_refusals(sm, kw, expect):
    assert sort(sm, **kw) == expect


def test_moe_sort_workspace_sizes(sm):
    f = sm.moe_sort_workspace_bytes
    assert [f(*a) for a in ((0, 8, 100), (1, 8, 100), (64, 8, 100))] == [0, 0, 0]
    # counts of every chunk of at most 1024 pairs and their sums
    for T, k, E in ((4096, 8, 100), (16384, 16, 512), (100, 64, 4096), (3000, 1, 1)):
        assert f(T, k, E) >= ((T * k + 1023) // 1024 + 1) * E * 4
    assert f(-1, 8, 100) == 0 and f(4, 0, 100) == 0 and f(4, 65, 100) == 0 and f(4, 8, 0) == 0
    assert f(1 << 26, 64, 8) == 0 and f(4, 8, 4097) == 0
    assert f((1 << 31) // 64 - 1, 64, 4096) >= 2 ** 34      # no 32-bit size


def unsort(sm, rows=F, rd=BF16, ldr=64, n=8, inv=F, w=F, y=F, yd=F32, ldy=64, T=4, k=2, H=64):
    return sm.lib().seedmm_moe_unsort(rows, rd, ldr, n, inv, w, y, yd, ldy, T, k, H, None)


@pytest.mark.parametrize("kw,expect", [
    (dict(T=-1), -1), (dict(k=0), -1), (dict(k=65), -1), (dict(T=1 << 26, k=64), -1), (dict(H=-1), -1),
    (dict(H=(1 << 30) + 1, ldr=1 << 31, ldy=1 << 31), -1), (dict(n=-1), -1), (dict(ldr=63), -1),
    (dict(ldy=63), -1), (dict(rd=I8), -1), (dict(yd=I8), -1), (dict(rows=None), -1), (dict(inv=None), -1),
    (dict(y=None), -1), (dict(rows=F + 1), -2), (dict(rows=F + 2, rd=F32), -2), (dict(y=F + 2), -2),
    (dict(y=F + 1, yd=BF16), -2), (dict(inv=F + 2), -2), (dict(w=F + 2), -2),
    (dict(T=0, rows=None, inv=None, w=None, y=None), 0), (dict(H=0, rows=None, inv=None, y=None), 0),
])
def test_moe_unsort_refusals(sm, kw, expect):
    assert unsort(sm, **kw) == expect


def grad(sm, dy=F, dd=F32, ldd=64, rows=F, rd=BF16, ldr=64, n=8, inv=F, w=F, dr=2 * F, ldg=64, dw=F, T=4,
         k=2, H=64):
    return sm.lib().seedmm_moe_unsort_grad(dy, dd, ldd, rows, rd, ldr, n, inv, w, dr, ldg, dw, T, k, H, None)


@pytest.mark.parametrize("kw,expect", [
    (dict(T=-1), -1), (dict(k=0), -1), (dict(k=65), -1), (dict(T=1 << 26, k=64), -1), (dict(H=-1), -1),
    (dict(H=(1 << 30) + 1, ldr=1 << 31, ldd=1 << 31, ldg=1 << 31), -1), (dict(n=-1), -1),
    (dict(ldd=63), -1), (dict(ldr=63), -1), (dict(ldg=63), -1), (dict(dd=I8), -1), (dict(rd=I8), -1),
    (dict(dy=None), -1), (dict(rows=None), -1), (dict(inv=None), -1), (dict(w=None), -1),
    (dict(dr=None, dw=None), -1), (dict(dr=F, ldg=128), -1), (dict(dr=F, ldg=128, ldr=128, dy=F + 2), -2),
    (dict(dy=F + 2), -2), (dict(dy=F + 1, dd=BF16), -2), (dict(rows=F + 1), -2), (dict(dr=2 * F + 1), -2),
    (dict(inv=F + 2), -2), (dict(w=F + 2), -2), (dict(dw=F + 2), -2),
    (dict(T=0, dy=None, rows=None, inv=None, w=None, dr=None, dw=None), 0), (dict(H=0, dw=None), 0),
])
def test_moe_unsort_grad_refusals(sm, kw, expect):
    assert grad(sm, **kw) == expect


def swiglu(sm, g=F, gd=BF16, ldg=64, o=F, od=BF16, ldo=32, sc=None, count=None, N=2, I=32):
    return sm.lib().seedmm_swiglu(g, gd, ldg, o, od, ldo, sc, count, N, I, None)


@pytest.mark.parametrize("kw,expect", [
    (dict(N=-1), -1), (dict(I=-1), -1), (dict(I=(1 << 29) + 1, ldg=1 << 31, ldo=1 << 30), -1),
    (dict(ldg=63), -1), (dict(ldo=31), -1), (dict(gd=I8), -1), (dict(od=3), -1), (dict(od=I8), -1),
    (dict(sc=F), -1), (dict(g=None), -1), (dict(o=None), -1), (dict(g=F + 1), -2), (dict(g=F + 2, gd=F32), -2),
    (dict(o=F + 1), -2), (dict(o=F + 2, od=F32), -2), (dict(od=I8, sc=F + 2), -2), (dict(count=F + 2), -2),
    (dict(N=0, g=None, o=None), 0), (dict(I=0, g=None, o=None), 0),
])
def test_swiglu_refusals(sm, kw, expect):
    assert swiglu(sm, **kw) == expect


def layer(sm, ids=F, w=F, T=4, k=2, x=F, xs=F, y=F, E=8, H=64, I=32, gu=None, dn=None, ws=F, wsb=None):
    L = sm.lib()
    if wsb is None:
        wsb = L.seedmm_moe_i8_workspace_bytes(T, k, E, H, I)
    m = sm.I8Mat(F, F, F32)
    return L.seedmm_moe_i8(ids, w, T, k, x, xs, y, E, H, I, gu or m, dn or m, ws, wsb, None)


@pytest.mark.parametrize("kw,expect", [
    (dict(T=-1), -1), (dict(k=0), -1), (dict(k=65), -1), (dict(E=0), -1), (dict(E=4097), -1), (dict(H=0), -1),
    (dict(I=0), -1), (dict(H=131072), -1), (dict(I=131072), -1), (dict(T=(1 << 29) + 1, k=2), -1),
    (dict(ids=None), -1), (dict(w=None), -1), (dict(x=None), -1), (dict(xs=None), -1), (dict(y=None), -1),
    (dict(ids=F + 2), -2), (dict(w=F + 2), -2), (dict(xs=F + 2), -2), (dict(y=F + 2), -2),
    (dict(ws=F + 8), -2), (dict(ws=None), -3), (dict(wsb=64), -3),
    (dict(T=0, ids=None, w=None, x=None, xs=None, y=None, ws=None), 0),
])
def test_moe_i8_refusals(sm, kw, expect):
    assert layer(sm, **kw) == expect


def test_moe_i8_refuses_bad_matrices(sm):
    for bad, e in (((None, F, F32), -1), ((F, None, F32), -1), ((F, F, I8), -1), ((F, F + 2, F32), -2),
                   ((F, F + 1, BF16), -2)):
        assert layer(sm, gu=sm.I8Mat(*bad)) == e and layer(sm, dn=sm.I8Mat(*bad)) == e


def test_moe_i8_workspace_sizes(sm):
    f = sm.moe_i8_workspace_bytes
    for T, k, E, H, I in ((1, 8, 100, 2048, 1024), (4096, 8, 100, 2048, 1024), (7, 3, 5, 100, 30)):
        P = T * k
        assert f(T, k, E, H, I) >= P * H + P * max(2 * I, H) * 2 + P * I + 12 * P + sm.moe_sort_workspace_bytes(T, k, E)
    assert f(1, 8, 100, 0, 1024) == 0 and f(1, 0, 100, 2048, 1024) == 0 and f(-1, 8, 100, 2048, 1024) == 0
    assert f(1 << 27, 8, 100, 131071, 131071) > 2 ** 48


def test_binding_refuses_cpu_tensors_and_counts_arguments(sm):
    import torch
    x8, ids = torch.zeros(2, 64, dtype=torch.int8), torch.zeros(2, 4, dtype=torch.int32)
    xf, sc = torch.zeros(2, 64), torch.zeros(2)
    for call, name in (
            (lambda: sm.i8_gemv({"weight": x8, "scales": sc}, x8, sc, 16, 64), "x"),
            (lambda: sm.i8_gemv({"weight": x8, "scales": sc}, x8, sc, 16, 64, y=xf), "x"),
            (lambda: sm.moe_sort(xf, ids, 8), "topk_ids"),
            (lambda: sm.moe_sort(xf, ids, 8, rows=xf, offsets=ids, inverse=ids), "x"),
            (lambda: sm.moe_unsort(xf, ids), "inverse"), (lambda: sm.moe_unsort(xf, ids, y=xf), "rows"),
            (lambda: sm.moe_unsort_grad(xf, xf, ids, xf), "rows"),
            (lambda: sm.moe_unsort_grad(xf, xf, ids, xf, drows=xf, dw=xf), "rows"),
            (lambda: sm.swiglu(xf), "gate_up"), (lambda: sm.swiglu(xf, out=xf), "gate_up"),
            (lambda: sm.moe_i8(ids, xf, x8, sc, 8, 64, 32, {}, {}), "x"),
            (lambda: sm.moe_i8(ids, xf, x8, sc, 8, 64, 32, {"weight": x8, "scales": sc},
                               {"weight": x8, "scales": sc}, y=xf), "x")):
        with pytest.raises(TypeError, match=f"{name} must be a CUDA"):
            call()
    for f in ("i8_gemv", "moe_sort", "moe_unsort", "moe_unsort_grad", "swiglu", "moe_i8", "init_experts"):
        with pytest.raises(TypeError, match="arguments are needed"):
            getattr(sm._binding, f)(None)
