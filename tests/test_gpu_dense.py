"""GPU tests of the dense operators around the routed layer (seedmm_q4_gemv, seedmm_add_norm,
seedmm_route, seedmm_moe_block) against their formulas in 64 bits.

Tolerances, with u = 2^-24 the unit roundoff of fp32:
- 4-bit product: every product of a code and an activation is exact, sums are fp32.  With
  S = sum_k (|s| (q + 32) + |b|) |x| (the terms, the code's offset of 16 and its removal), an
  element is off by at most 8 sqrt(K) u S (the summation bound used for the other products),
  plus the output's rounding (bf16: 2^-8 of the value).
- norm: the mean of H squares is off by at most (sqrt(H) + 4) u relative, the root by half of
  that; the sum, two products, division and root add 8 u; plus the output's rounding.
- 8 bits: the value over the scale is off by the norm's error, at most 127 times it in codes,
  and the rounding to a code by half a code.
- router weights: exp of a difference d is off by (|d| + 4) u; the sum of at most 64 terms and
  the quotient add 8 u.  Chosen experts are equal.
"""
import math
import sys

import numpy as np
import pytest

import synth

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
DT = {}


def say(*a):
    print("[case]", *a, file=sys.stderr, flush=True)


@pytest.fixture(scope="module")
def sm():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    from pseudo_random_weight_amd import seedmm
    DT.update(f32=torch.float32, bf16=torch.bfloat16, i8=torch.int8)
    return seedmm


def gen(seed):
    import torch
    g = torch.Generator(device="cpu")
    g.manual_seed(seed)
    return g


# ---- 4-bit product --------------------------------------------------------------------

def q4_case(N, M, K, group, x, s, seed):
    """CPU tensors: weight words, scales, biases, activation rows (and their 8-bit scales)."""
    import torch
    g = gen(seed)
    w = torch.randint(-2 ** 31, 2 ** 31, (M, K // 8), generator=g, dtype=torch.int64).to(torch.int32)
    sc = (0.01 * torch.randn(M, K // group, generator=g)).to(DT[s])
    bi = (0.05 * torch.randn(M, K // group, generator=g)).to(DT[s])
    xv = torch.randn(N, K, generator=g) * torch.exp(torch.randn(K, generator=g))
    xs = None
    if x == "i8":
        xs = 0.01 + torch.rand(N, generator=g)
        xv = torch.randint(-128, 128, (N, K), generator=g).to(torch.int8)
    else:
        xv = xv.to(DT[x])
    return w, sc, bi, xv, xs


def q4_ref(w, sc, bi, xv, xs, group):
    """(y, S) in 64 bits."""
    import torch
    M, K = w.shape[0], w.shape[1] * 8
    q = torch.stack([(w.to(torch.int64) >> (4 * i)) & 15 for i in range(8)], dim=2).view(M, K).double()
    s = sc.double().repeat_interleave(group, dim=1)
    b = bi.double().repeat_interleave(group, dim=1)
    x = xv.double() if xs is None else xv.double() * xs.double()[:, None]
    return x @ (q * s + b).t(), x.abs() @ (s.abs() * (q + 32) + b.abs()).t()


def q4_bound(ref, S, K, y):
    return 8 * math.sqrt(K) * U * S + (2.0 ** -8 if y == "bf16" else U) * ref.abs() + 1e-37


def to_mat(w, sc, bi):
    import torch
    return {"weight": w.cuda().view(torch.uint32), "scales": sc.cuda(), "biases": bi.cuda()}


def check_q4(sm, N, M, K, group, x, s, y, seed):
    import torch
    say("q4", N, M, K, group, x, s, y)
    w, sc, bi, xv, xs = q4_case(N, M, K, group, x, s, seed)
    out = sm.q4_gemv(to_mat(w, sc, bi), xv.cuda(), M, K, group,
                     x_scale=None if xs is None else xs.cuda(), y_dtype=DT[y])
    torch.cuda.synchronize()
    assert out.shape == (N, M) and out.dtype == DT[y]
    ref, S = q4_ref(w, sc, bi, xv, xs, group)
    err = (out.cpu().double() - ref).abs()
    assert bool((err <= q4_bound(ref, S, K, y)).all()), float((err / q4_bound(ref, S, K, y)).max())


@pytest.mark.parametrize("x", ["bf16", "i8", "f32"])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("N,M,K", [
    (1, 1, 128), (1, 16, 128), (1, 17, 2048), (1, 100, 2048 + 128), (1, 257, 1024 - 128),
    (2, 33, 384), (4, 64, 1152), (5, 48, 640), (6, 15, 512), (15, 40, 768), (16, 128, 1024),
    (17, 130, 1280), (33, 65, 256), (64, 64, 512), (65, 200, 896), (130, 129, 384), (300, 70, 256),
])
def test_q4_gemv(sm, x, group, N, M, K):
    check_q4(sm, N, M, K, group, x, "bf16", "f32", 1)


@pytest.mark.parametrize("x", ["bf16", "i8", "f32"])
@pytest.mark.parametrize("s,y", [("f32", "f32"), ("f32", "bf16"), ("bf16", "bf16")])
@pytest.mark.parametrize("N,M,K,group", [(1, 50, 96, 32), (3, 21, 192, 64), (40, 90, 1088, 64), (20, 40, 32, 32),
                                         (200, 150, 160, 32), (1, 130, 4160, 64), (9, 300, 8320, 128)])
def test_q4_gemv_types(sm, x, s, y, N, M, K, group):
    check_q4(sm, N, M, K, group, x, s, y, 2)


@pytest.mark.parametrize("N,M,K,group", [(1, 4000, 16384, 64), (16, 1000, 16384, 32), (70, 500, 12288, 128),
                                         (1, 40000, 256, 64), (1025, 260, 320, 64), (512, 1024, 2048, 64)])
@pytest.mark.parametrize("x", ["bf16", "i8", "f32"])
def test_q4_gemv_long(sm, x, N, M, K, group):
    check_q4(sm, N, M, K, group, x, "bf16", "f32", 3)


@pytest.mark.parametrize("x", ["bf16", "i8", "f32"])
@pytest.mark.parametrize("N", [1, 7, 20, 150])
def test_q4_rows_apart_leave_the_rest(sm, x, N):
    """Activation rows and output rows with gaps: the gaps are not read into the result and
    not written; a vector [K] gives a vector [M]; nothing past the last row is touched."""
    import torch
    M, K, group = 75, 320, 64
    w, sc, bi, xv, xs = q4_case(N, M, K, group, x, "bf16", 4)
    wide = torch.full((N + 2, K + 64), 100, dtype=DT[x])
    wide[:N, :K] = xv
    y = torch.full((N + 3, M + 13), 7.0, device="cuda")
    mat = to_mat(w, sc, bi)
    xsd = None if xs is None else xs.cuda()
    out = sm.q4_gemv(mat, wide.cuda()[:N, :K], M, K, group, x_scale=xsd, y=y[:N, :M])
    torch.cuda.synchronize()
    ref, S = q4_ref(w, sc, bi, xv, xs, group)
    assert bool(((out.cpu().double() - ref).abs() <= q4_bound(ref, S, K, "f32")).all())
    assert bool((y[:, M:] == 7.0).all()) and bool((y[N:] == 7.0).all())
    v = sm.q4_gemv(mat, xv[0].cuda(), M, K, group, x_scale=xsd)
    torch.cuda.synchronize()
    assert v.shape == (M,)
    assert bool(((v.cpu().double() - ref[0]).abs() <= q4_bound(ref, S, K, "f32")[0]).all())


@pytest.mark.parametrize("x", ["bf16", "f32"])
@pytest.mark.parametrize("N", [3, 40, 140])
def test_q4_a_bad_row_stays_alone(sm, x, N):
    import torch
    M, K, group = 60, 256, 64
    w, sc, bi, xv, _ = q4_case(N, M, K, group, x, "bf16", 5)
    mat = to_mat(w, sc, bi)
    good = sm.q4_gemv(mat, xv.cuda(), M, K, group)
    bad = xv.clone()
    bad[1, 7], bad[2, 200] = math.nan, math.inf
    got = sm.q4_gemv(mat, bad.cuda(), M, K, group)
    torch.cuda.synchronize()
    assert not bool(torch.isfinite(got[1:3]).any())
    keep = [n for n in range(N) if n not in (1, 2)]
    assert bool((got[keep] == good[keep]).all())


def test_q4_extreme_activations(sm):
    """fp32 activations over the whole range: the three parts of a value stay exact."""
    import torch
    M, K, group = 32, 64, 64
    w, sc, bi, xv, _ = q4_case(6, M, K, group, "f32", "f32", 6)
    xv = torch.stack([xv[0] * 1e30, xv[1] * 1e-30, xv[2].sign() * (1 + 2.0 ** -23), xv[3] * 1e-3,
                      torch.zeros(K), xv[5]])
    got = sm.q4_gemv(to_mat(w, sc, bi), xv.cuda(), M, K, group)
    torch.cuda.synchronize()
    ref, S = q4_ref(w, sc, bi, xv, None, group)
    assert bool(((got.cpu().double() - ref).abs() <= q4_bound(ref, S, K, "f32")).all())


@pytest.mark.parametrize("x", ["bf16", "i8", "f32"])
def test_q4_zero_sizes(sm, x):
    import torch
    w, sc, bi, xv, xs = q4_case(4, 20, 128, 64, x, "bf16", 7)
    mat = to_mat(w, sc, bi)
    xsd = None if xs is None else xs.cuda()
    y = torch.full((4, 24), 5.0, device="cuda")
    sm.q4_gemv(mat, xv.cuda(), 20, 0, 64, x_scale=xsd, y=y[:, :20])
    torch.cuda.synchronize()
    assert bool((y[:, :20] == 0).all()) and bool((y[:, 20:] == 5.0).all())
    assert sm.q4_gemv(mat, xv[:0].cuda(), 20, 128, 64, x_scale=xsd).shape == (0, 20)


def test_q4_matrix_beyond_32_bit_bytes(sm):
    """A matrix of more than 2^31 bytes of codes: rows at its end."""
    import torch
    K, group = 65536, 128
    M = 65536 + 24
    g = torch.Generator(device="cuda")
    g.manual_seed(8)
    w = torch.empty(M, K // 8, dtype=torch.int32, device="cuda")
    w.random_(-2 ** 31, 2 ** 31 - 1, generator=g)
    sc = 0.01 * torch.randn(M, K // group, generator=g, device="cuda")
    bi = 0.05 * torch.randn(M, K // group, generator=g, device="cuda")
    assert w.numel() * 4 > 2 ** 31
    mat = {"weight": w.view(torch.uint32), "scales": sc, "biases": bi}
    for N in (1, 40):
        say("q4 beyond 2^31 bytes", N)
        x = torch.randn(N, K, generator=g, device="cuda").to(torch.bfloat16)
        got = sm.q4_gemv(mat, x, M, K, group)
        torch.cuda.synchronize()
        for rows in (slice(0, 3), slice(M - 9, M)):
            ref, S = q4_ref(w[rows].cpu(), sc[rows].cpu(), bi[rows].cpu(), x.cpu(), None, group)
            assert bool(((got[:, rows].cpu().double() - ref).abs() <= q4_bound(ref, S, K, "f32")).all())


def test_q4_same_bits_again_and_on_another_stream(sm):
    import torch
    for (N, M, K, x) in [(1, 500, 2048, "bf16"), (30, 300, 1024, "i8"), (300, 300, 512, "bf16")]:
        w, sc, bi, xv, xs = q4_case(N, M, K, 64, x, "bf16", 9)
        mat, xd, xsd = to_mat(w, sc, bi), xv.cuda(), None if xs is None else xs.cuda()
        a = sm.q4_gemv(mat, xd, M, K, 64, x_scale=xsd)
        st = torch.cuda.Stream()
        st.wait_stream(torch.cuda.current_stream())
        b = sm.q4_gemv(mat, xd, M, K, 64, x_scale=xsd, stream=st)
        st.synchronize()
        torch.cuda.synchronize()
        assert bool((a == b).all())


# ---- norm -----------------------------------------------------------------------------

def norm_case(N, H, x, delta, weight, seed):
    import torch
    g = gen(seed)
    xv = (3 * torch.randn(N, H, generator=g)).to(DT[x])
    d = None if delta is None else torch.randn(N, H, generator=g).to(DT[delta])
    w = None if weight is None else (1 + 0.3 * torch.randn(H, generator=g)).to(DT[weight])
    return xv, d, w


def norm_ref(xv, d, w, eps):
    r = xv.double() if d is None else xv.double() + d.double()
    v = r / ((r * r).mean(dim=1, keepdim=True) + eps).sqrt()
    return r, v if w is None else v * w.double()


def norm_tol(H):
    return (0.5 * (math.sqrt(H) + 4) + 8) * U


def check_norm(out, sc, res, xv, d, w, eps, out_dt, res_dt):
    import torch
    H = xv.shape[1]
    r, v = norm_ref(xv, d, w, eps)
    tol = norm_tol(H)
    if out_dt == "i8":
        top = v.abs().amax(dim=1)
        s = sc.cpu().double()
        assert bool(((s - top / 127).abs() <= (tol + 2 * U) * top / 127 + 2.0 ** -126).all())
        codes = out.cpu().double()
        assert bool((codes.abs() <= 127).all())
        assert bool(((codes * s[:, None] - v).abs() <= (0.5 + 127 * (2 * tol + 4 * U)) * s[:, None]).all())
    else:
        rnd = 2.0 ** -8 if out_dt == "bf16" else U
        assert bool(((out.cpu().double() - v).abs() <= (tol + rnd * (1 + tol)) * v.abs() + 1e-37).all())
        assert sc is None
    if d is not None:
        rnd = (2.0 ** -8 if res_dt == "bf16" else 0) + U * 1.01
        assert bool(((res.cpu().double() - r).abs() <= rnd * r.abs() + 1e-37).all())


@pytest.mark.parametrize("x,delta,weight,out", [
    ("bf16", "f32", "bf16", "bf16"), ("bf16", "bf16", "bf16", "i8"), ("f32", "f32", "f32", "f32"),
    ("f32", "bf16", None, "i8"), ("bf16", None, "f32", "f32"), ("f32", None, None, "bf16"),
    ("f32", "f32", "bf16", "bf16"), ("bf16", "f32", "f32", "i8"),
])
@pytest.mark.parametrize("N,H", [(1, 1), (1, 7), (3, 8), (2, 63), (5, 64), (1, 2048), (4, 2047), (33, 256),
                                 (2, 520), (1, 7168), (3, 7167), (2, 16384), (1, 16385), (2, 40000),
                                 (1, 100003), (1030, 72)])
def test_add_norm(sm, x, delta, weight, out, N, H):
    import torch
    say("norm", N, H, x, delta, weight, out)
    xv, d, w = norm_case(N, H, x, delta, weight, 11)
    c = lambda t: None if t is None else t.cuda()
    xd = c(xv)
    o, sc, res = sm.add_norm(xd, c(w), delta=c(d), eps=1e-5, out_dtype=DT[out])
    torch.cuda.synchronize()
    assert o.dtype == DT[out] and (res is xd) == (d is None)
    assert bool((xd.cpu() == xv).all())
    check_norm(o, sc, res, xv, d, w, 1e-5, out, x)


@pytest.mark.parametrize("x", ["bf16", "f32"])
@pytest.mark.parametrize("H", [65, 256, 2048, 20000])
@pytest.mark.parametrize("out", ["bf16", "i8", "f32"])
def test_add_norm_in_place_and_rows_apart(sm, x, H, out):
    """The residual updated in place, rows of every operand apart by gaps that stay as they
    were and start off 16 bytes, and the same bits as the plain call."""
    import torch
    N = 5
    xv, d, w = norm_case(N, H, x, "f32", "bf16", 12)
    xw = torch.full((N + 1, H + 3), 9.0, dtype=DT[x], device="cuda")
    dw = torch.full((N, H + 1), 9.0, device="cuda")
    ow = torch.full((N + 1, H + 5), 9, dtype=DT[out], device="cuda")
    xw[:N, 1:H + 1] = xv.cuda()
    dw[:, :H] = d.cuda()
    xr = xw[:N, 1:H + 1]
    o, sc, res = sm.add_norm(xr, w.cuda(), delta=dw[:, :H], residual=xr, out=ow[:N, 3:H + 3])
    torch.cuda.synchronize()
    assert res is xr
    check_norm(o, sc, res, xv, d, w, 1e-6, out, x)
    assert bool((xw[:N, 0] == 9).all()) and bool((xw[:N, H + 1:] == 9).all()) and bool((xw[N] == 9).all())
    assert bool((ow[:N, :3] == 9).all()) and bool((ow[:N, H + 3:] == 9).all()) and bool((ow[N] == 9).all())


def test_add_norm_edge_rows(sm):
    """Rows of zeros, one large value, tiny values, an infinity, a NaN; eps 0."""
    import torch
    for H in (48, 2048, 30000):
        x = torch.zeros(7, H)
        x[1, 5] = 1e15
        x[2] = 1e-18
        x[3, H - 1] = math.inf
        x[4, 0] = math.nan
        x[5] = -1e-12
        x[6] = torch.linspace(-3, 3, H)
        o, sc, _ = sm.add_norm(x.cuda(), out_dtype=torch.int8)
        f, none, _ = sm.add_norm(x.cuda(), out_dtype=torch.float32)
        torch.cuda.synchronize()
        assert none is None
        for n in (0, 1, 2, 5, 6):
            check_norm(o[n:n + 1], sc[n:n + 1], None, x[n:n + 1], None, None, 1e-6, "i8", "f32")
            check_norm(f[n:n + 1], None, None, x[n:n + 1], None, None, 1e-6, "f32", "f32")
        assert bool((o[0] == 0).all()) and float(sc[0]) == 2.0 ** -126
        for n in (3, 4):
            assert math.isnan(float(sc[n])) and bool((o[n] == 0).all())
        assert bool(torch.isnan(f[4]).all())
        one = sm.add_norm(x[6:].cuda(), eps=0.0, out_dtype=torch.float32)[0]
        torch.cuda.synchronize()
        check_norm(one, None, None, x[6:], None, None, 0.0, "f32", "f32")


def test_add_norm_empty_and_vector(sm):
    import torch
    x = torch.randn(0, 64, device="cuda")
    o, sc, res = sm.add_norm(x, out_dtype=torch.int8)
    assert o.shape == (0, 64) and sc.shape == (0,) and res is x
    xv, d, w = norm_case(1, 333, "bf16", "f32", "bf16", 13)
    o, _, res = sm.add_norm(xv[0].cuda(), w.cuda(), delta=d[0].cuda())
    torch.cuda.synchronize()
    assert o.shape == (333,) and res.shape == (333,)
    check_norm(o[None], None, res[None], xv, d, w, 1e-6, "bf16", "bf16")


def test_norm_codes_through_the_product(sm):
    """The 8-bit rows go to the 4-bit product: its result is the product of the values that
    the codes stand for, and near the bf16 path's."""
    import torch
    N, H, M = 9, 512, 70
    xv, d, w = norm_case(N, H, "bf16", "f32", "bf16", 14)
    wq, sc, bi, _, _ = q4_case(1, M, H, 64, "bf16", "bf16", 15)
    mat = to_mat(wq, sc, bi)
    o, s, _ = sm.add_norm(xv.cuda(), w.cuda(), delta=d.cuda(), out_dtype=torch.int8)
    y = sm.q4_gemv(mat, o, M, H, 64, x_scale=s)
    torch.cuda.synchronize()
    ref, S = q4_ref(wq, sc, bi, o.cpu(), s.cpu(), 64)
    assert bool(((y.cpu().double() - ref).abs() <= q4_bound(ref, S, H, "f32")).all())
    # each activation is off by half a code at most
    _, v = norm_ref(xv, d, w, 1e-6)
    full, _ = q4_ref(wq, sc, bi, v, None, 64)
    half = (0.5 + 127 * (2 * norm_tol(H) + 4 * U)) * s.cpu().double()[:, None]
    q = torch.stack([(wq.to(torch.int64) >> (4 * i)) & 15 for i in range(8)], dim=2).view(M, H).double()
    W = q * sc.double().repeat_interleave(64, 1) + bi.double().repeat_interleave(64, 1)
    assert bool(((ref - full).abs() <= half * W.abs().sum(dim=1)[None] + 1e-12).all())


# ---- router ---------------------------------------------------------------------------

def route_ref(lg, k, score, bias):
    lg = lg.astype(np.float64)
    with np.errstate(over="ignore", invalid="ignore"):
        p = 1 / (1 + np.exp(-lg))
        key = lg if score == "softmax" else p + (0 if bias is None else bias.astype(np.float64))
    off = ~(lg > -np.inf) | ~(key > -np.inf)
    key = np.where(off, -np.inf, key)
    T, E = lg.shape
    ids = np.empty((T, k), dtype=np.int32)
    w = np.zeros((T, k))
    for t in range(T):
        order = sorted(range(E), key=lambda e: (bool(off[t, e]), -key[t, e], e))[:k]
        ids[t] = order
        ok = ~off[t, order]
        if ok.any():
            sel = lg[t, order]
            if score == "softmax":
                top = sel[ok].max()
                v = np.array([(1.0 if s == top else math.exp(s - top)) if o else 0.0 for s, o in zip(sel, ok)])
            else:
                v = np.where(ok, p[t, order], 0.0)
            w[t] = v / v.sum() if v.sum() > 0 else 0.0
    return ids, w


def check_route(sm, lg, k, score, bias=None):
    import torch
    ids, w = sm.route(lg.cuda(), k, bias=None if bias is None else bias.cuda(), score=score)
    torch.cuda.synchronize()
    ri, rw = route_ref(lg.float().numpy(), k, score, None if bias is None else bias.numpy())
    assert np.array_equal(ids.cpu().numpy(), ri)
    lf = lg.float().numpy().astype(np.float64)
    sel = np.take_along_axis(lf, ri.astype(np.int64), axis=1)
    fin = np.where(np.isfinite(sel), sel, 0.0)
    span = np.abs(fin - fin.max(axis=1, keepdims=True)) if score == "softmax" else 0.0
    assert np.all(np.abs(w.cpu().numpy() - rw) <= (2 * span + 16) * U * rw + 1e-37)


@pytest.mark.parametrize("score", ["softmax", "sigmoid", "sigmoid+bias"])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 100, 8), (3, 8, 8), (5, 63, 3), (7, 64, 64), (9, 65, 1),
                                   (64, 100, 8), (33, 129, 17), (20, 257, 4), (257, 512, 10), (6, 1000, 32),
                                   (5, 2049, 64), (4, 4096, 64), (1500, 100, 8)])
def test_route(sm, score, dt, T, E, k):
    import torch
    say("route", score, dt, T, E, k)
    g = gen(21)
    lg = torch.randn(T, E, generator=g).to(DT[dt])
    bias = 0.1 * torch.randn(E, generator=g) if score.endswith("bias") else None
    check_route(sm, lg, k, score.split("+")[0], bias)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,k", [(5, 5), (64, 8), (100, 8), (200, 20), (512, 8), (4096, 9)])
def test_route_ties_masks_and_infinities(sm, score, E, k):
    """Equal logits (all, and in few classes), -0 beside 0, rows with fewer experts left than
    slots, with none, with NaN, with +inf, and logits far apart."""
    import torch
    g = gen(22)
    rows = [torch.zeros(E), torch.randint(0, 3, (E,), generator=g).float(),
            torch.where(torch.arange(E) % 2 == 0, torch.tensor(-0.0), torch.tensor(0.0)),
            torch.full((E,), -math.inf), torch.full((E,), math.nan)]
    r = torch.full((E,), -math.inf)
    r[E // 2] = 1.0
    r[E - 1] = 2.0
    rows.append(r)
    r = torch.randn(E, generator=g)
    r[::3] = -math.inf
    r[1::4] = math.nan
    rows.append(r)
    r = torch.randn(E, generator=g)
    r[E - 1] = math.inf
    rows.append(r)
    r = torch.randn(E, generator=g)
    r[1:4] = math.inf
    rows.append(r)
    rows.append(torch.randn(E, generator=g) * 1e4)
    rows.append(torch.randn(E, generator=g) * 1e-4)
    rows.append(torch.full((E,), -3e38))
    check_route(sm, torch.stack(rows), k, score)
    if score == "sigmoid":
        b = 0.1 * torch.randn(E, generator=g)
        b[0], b[E // 3] = -math.inf, math.nan
        check_route(sm, torch.stack(rows), k, score, b)


def test_route_rows_apart_and_outputs(sm):
    """Logit rows with a gap; given outputs are written, only in front of their rows' end."""
    import torch
    g = gen(23)
    wide = torch.randn(40, 117, generator=g)
    ids = torch.full((41, 6), -7, dtype=torch.int32, device="cuda")
    w = torch.full((41, 6), -7.0, device="cuda")
    got = sm.route(wide.cuda()[:, 9:109], 6, ids=ids[:40], w=w[:40])
    torch.cuda.synchronize()
    ri, rw = route_ref(wide[:, 9:109].numpy(), 6, "softmax", None)
    assert np.array_equal(got[0].cpu().numpy(), ri)
    assert np.allclose(got[1].cpu().numpy(), rw, rtol=1e-5, atol=0)
    assert bool((ids[40] == -7).all()) and bool((w[40] == -7).all())
    assert sm.route(torch.empty(0, 10, device="cuda"), 3)[0].shape == (0, 3)


def test_binding_refusals_on_gpu_tensors(sm):
    import torch
    x = torch.zeros(2, 64, dtype=torch.bfloat16, device="cuda")
    mat = {"weight": torch.zeros(16 * 8, dtype=torch.int32, device="cuda").view(torch.uint32),
           "scales": torch.zeros(16, device="cuda"), "biases": torch.zeros(16, device="cuda")}
    with pytest.raises(ValueError, match="K = 60"):
        sm.q4_gemv(mat, x, 16, 60)
    with pytest.raises(ValueError, match="weight has"):
        sm.q4_gemv(mat, x, 17, 64)
    with pytest.raises(ValueError, match="x rows hold"):
        sm.q4_gemv(mat, x, 8, 128)
    with pytest.raises(TypeError, match="one type"):
        sm.q4_gemv(dict(mat, biases=mat["biases"].bfloat16()), x, 16, 64)
    with pytest.raises(TypeError, match="x_scale"):
        sm.q4_gemv(mat, x.to(torch.int8), 16, 64)
    with pytest.raises(ValueError, match="x_scale"):
        sm.q4_gemv(mat, x, 16, 64, x_scale=torch.ones(2, device="cuda"))
    with pytest.raises(ValueError, match="y must hold"):
        sm.q4_gemv(mat, x, 16, 64, y=torch.empty(2, 15, device="cuda"))
    with pytest.raises(TypeError, match="weight must be one of"):
        sm.q4_gemv(dict(mat, weight=mat["weight"].view(torch.int32)), x, 16, 64)
    with pytest.raises(sm.SeedmmError) as e:    # rows that do not start on 16 bytes
        sm.q4_gemv(mat, torch.zeros(2, 68, dtype=torch.bfloat16, device="cuda")[:, :64], 16, 64)
    assert e.value.status == sm.EALIGN
    with pytest.raises(ValueError, match="delta"):
        sm.add_norm(x, delta=x[:1])
    for bad in (x[:1].expand(2, 64), torch.zeros(64, 2, dtype=torch.bfloat16, device="cuda").t(),
                torch.zeros(2, 128, dtype=torch.bfloat16, device="cuda")[:, ::2]):
        with pytest.raises(ValueError, match="distinct rows"):
            sm.add_norm(x, delta=bad)
    with pytest.raises(ValueError, match="row-major"):
        sm.add_norm(x, delta=x[None], residual=x)
    with pytest.raises(ValueError, match="workspace"):
        sm.q4_gemv(mat, x, 16, 64, workspace=torch.zeros(64))
    with pytest.raises(sm.SeedmmError) as e:
        sm.q4_gemv(mat, x.repeat(20, 1).float(), 16, 64, workspace=torch.zeros(64, device="cuda"))
    assert e.value.status == sm.EWORKSPACE
    with pytest.raises(ValueError, match="T..E"):
        sm.route(torch.zeros(8, device="cuda"), 2)
    with pytest.raises(TypeError, match="logits must be one of"):
        sm.route(torch.zeros(2, 8, dtype=torch.float64, device="cuda"), 2)
    with pytest.raises(ValueError, match="residual"):
        sm.add_norm(x, delta=x, residual=torch.empty(2, 64, device="cuda"))
    with pytest.raises(ValueError, match="int8"):
        sm.add_norm(x, scale=torch.empty(2, device="cuda"))
    with pytest.raises(ValueError, match="weight has"):
        sm.add_norm(x, torch.ones(63, device="cuda"))
    with pytest.raises(ValueError, match="top_k"):
        sm.route(torch.zeros(2, 8, device="cuda"), 9)
    with pytest.raises(ValueError, match="score"):
        sm.route(torch.zeros(2, 8, device="cuda"), 2, score="none")
    with pytest.raises(sm.SeedmmError) as e:
        sm.route(torch.zeros(2, 8, device="cuda"), 2, bias=torch.zeros(8, device="cuda"))
    assert e.value.status == sm.EINVAL


# ---- the layer on the residual stream --------------------------------------------------

def seed_dev(m):
    import torch
    return {"seeds": torch.from_numpy(m["seeds"].view(np.int16).copy()).view(torch.uint16).cuda(),
            "coefs": torch.from_numpy(m["coefs"].view(np.int16).copy()).view(torch.uint16).cuda(),
            "codes": torch.from_numpy(m["codes"].copy()).cuda(),
            "exp_bias": torch.from_numpy(m["exp_bias"].copy()).cuda()}


def block_case(sm, E, H, I, P, k, score, seed, group=64):
    import torch
    base = synth.config_seed(40 + seed)
    g, u = (synth.seed_matrix(base, f"blk.{n}", I, H, P, E) for n in ("g", "u"))
    d = synth.seed_matrix(base, "blk.d", H, I, P, E)
    w, sc, bi, _, _ = q4_case(1, E, H, group, "bf16", "bf16", seed)
    nw = (1 + 0.2 * torch.randn(H, generator=gen(seed))).to(torch.bfloat16)
    rb = 0.05 * torch.randn(E, generator=gen(seed + 1)) if score == "sigmoid" else None
    blk = sm.MoeBlock(E, H, I, P, k, seed_dev(g), seed_dev(u), seed_dev(d), to_mat(w, sc, bi), group,
                      norm_weight=nw.cuda(), eps=1e-5, score=score,
                      router_bias=None if rb is None else rb.cuda())
    return blk, (g, u, d), (w, sc, bi), nw, rb


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,H,I,P,k", [(1, 16, 256, 128, 4, 4), (5, 16, 256, 128, 4, 4),
                                         (40, 8, 192, 64, 3, 2), (1, 100, 2048, 1024, 4, 8),
                                         (600, 8, 128, 64, 4, 2)])
def test_block_is_its_calls(sm, score, T, E, H, I, P, k):
    """The block equals add_norm, q4_gemv, route and moe called one after the other, bit for
    bit, over two layers whose second takes the first's output as its delta."""
    import torch
    say("block", score, T, E, H, I, P, k)
    blk, (g, u, d), (w, sc, bi), nw, rb = block_case(sm, E, H, I, P, k, score, 1)
    mats, mat = [seed_dev(m) for m in (g, u, d)], to_mat(w, sc, bi)
    r0 = torch.randn(T, H, generator=gen(3)).to(torch.bfloat16).cuda()
    rbd = None if rb is None else rb.cuda()
    ra, y = r0.clone(), None
    got = []
    for _ in range(2):
        ids = torch.full((T, k), -1, dtype=torch.int32, device="cuda")
        wt = torch.full((T, k), -1.0, device="cuda")
        y = blk.moe(ra, delta=y, ids=ids, w=wt)
        got.append((y, ids, wt))
    rc, y = r0.clone(), None
    for yg, ig, wg in got:
        x, _, _ = sm.add_norm(rc, nw.cuda(), delta=y, eps=1e-5, residual=None if y is None else rc)
        lg = sm.q4_gemv(mat, x, E, H, 64)
        ids, wt = sm.route(lg, k, bias=rbd, score=score)
        y = sm.moe(ids, wt, x, E, H, I, P, *mats, check_ids=True)
        torch.cuda.synchronize()
        assert bool((ids == ig).all()) and bool((wt == wg).all()) and bool((y == yg).all())
    assert bool((rc == ra).all())


def test_block_against_the_oracle(sm, oracle):
    """The block from its inputs to its output in 64 bits: the norm, the router's logits and
    the choice from their formulas, the experts from the CPU reference on the bf16 rows."""
    import torch
    T, E, H, I, P, k = 6, 16, 256, 128, 4, 4
    blk, (g, u, d), (w, sc, bi), nw, _ = block_case(sm, E, H, I, P, k, "softmax", 2)
    xv, dl, _ = norm_case(T, H, "f32", "bf16", None, 5)
    r = xv.cuda()
    ids = torch.empty(T, k, dtype=torch.int32, device="cuda")
    wt = torch.empty(T, k, device="cuda")
    y = blk.moe(r, delta=dl.cuda(), ids=ids, w=wt)
    torch.cuda.synchronize()
    rr, v = norm_ref(xv, dl, nw, 1e-5)
    assert bool(((r.cpu().double() - rr).abs() <= 1.01 * U * rr.abs()).all())
    xb = v.to(torch.bfloat16)
    lg, _ = q4_ref(w, sc, bi, xb, None, 64)
    gap = lg.sort(dim=1, descending=True).values
    assert float((gap[:, :k] - gap[:, 1:k + 1]).min()) > 1e-3    # no choice hangs on a rounding
    ri, rw = route_ref(lg.numpy(), k, "softmax", None)
    assert np.array_equal(ids.cpu().numpy(), ri)
    ref = oracle.moe(ri, rw.astype(np.float32), xb.float().numpy(), E, H, I, P, g, u, d)
    err = np.linalg.norm(y.cpu().numpy() - ref) / np.linalg.norm(ref)
    assert err <= 1e-2, err


@pytest.mark.parametrize("T", [1, 12])
def test_block_graph_replays_match_eager(sm, T):
    """A captured block (two layers in a row, with the caller's second stream), replayed with
    eager work of its own between the replays, gives the eager bits each time."""
    import torch
    E, H, I, P, k = 16, 256, 128, 4, 4
    blk, _, _, _, _ = block_case(sm, E, H, I, P, k, "sigmoid", 3)
    side = sm.SideStream()
    r = torch.zeros(T, H, dtype=torch.bfloat16, device="cuda")
    bufs = [torch.empty(T, H, device="cuda") for _ in range(2)]
    ws = [torch.empty(blk.workspace_bytes(T), dtype=torch.uint8, device="cuda") for _ in range(2)]

    def step(rt, b, w, sd):
        blk.moe(rt, y=b[0], workspace=w[0], side=sd)
        blk.moe(rt, delta=b[0], y=b[1], workspace=w[1], side=sd)

    start = [torch.randn(T, H, generator=gen(30 + i)).to(torch.bfloat16).cuda() for i in range(4)]
    step(r, bufs, ws, side)      # first use outside the capture
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(r, bufs, ws, side)
    for s in start:
        re = s.clone()
        be = [torch.empty_like(b) for b in bufs]
        step(re, be, [torch.empty_like(w) for w in ws], None)
        torch.cuda.synchronize()
        r.copy_(s)
        graph.replay()
        torch.cuda.synchronize()
        assert bool((r == re).all()) and bool((bufs[0] == be[0]).all()) and bool((bufs[1] == be[1]).all())


def test_block_mixed_pack(sm):
    import torch
    T, E, H, I, k = 7, 8, 128, 64, 3
    Ps = [4, 3, 3, 4, 4, 3, 4, 3]
    base = synth.config_seed(44)
    g, u = (synth.seed_matrix_mixed(base, f"bm.{n}", I, H, Ps) for n in ("g", "u"))
    d = synth.seed_matrix_mixed(base, "bm.d", H, I, Ps)
    w, sc, bi, _, _ = q4_case(1, E, H, 32, "bf16", "f32", 6)
    mats, mat = [seed_dev(m) for m in (g, u, d)], to_mat(w, sc, bi)
    blk = sm.MoeBlock(E, H, I, 4, k, *mats, mat, 32, Ps=Ps)
    r = torch.randn(T, H, generator=gen(7)).cuda()
    y = blk.moe(r)
    x, _, same = sm.add_norm(r)
    ids, wt = sm.route(sm.q4_gemv(mat, x, E, H, 32), k)
    ref = sm.moe_mixed(ids, wt, x, E, H, I, sm.p4_mask(Ps, "cuda"), *mats, Ps=Ps)
    torch.cuda.synchronize()
    assert same is r and bool((y == ref).all())
    assert blk.moe(r[:0]).shape == (0, H)


def test_captured_operators_replay_like_eager(sm):
    """q4_gemv (few tokens, many tokens, K split), add_norm and route captured with buffers of
    the caller's, replayed with eager work of their own in between: every replay's bits are
    the eager call's on the inputs of the moment."""
    import torch
    for (N, M, K, xt) in [(1, 100, 2048, "bf16"), (16, 70, 512, "f32"), (40, 300, 4096, "bf16"),
                          (600, 260, 320, "i8")]:
        say("captured", N, M, K, xt)
        w, sc, bi, xv, xs = q4_case(N, M, K, 64, xt, "bf16", 31)
        mat, x, xsd = to_mat(w, sc, bi), xv.cuda(), None if xs is None else xs.cuda()
        y = torch.empty(N, M, device="cuda")
        nb = sm.q4_workspace_bytes(DT[xt], 64, M, K, N)
        ws = torch.empty(max(nb, 16), dtype=torch.uint8, device="cuda")
        hid = torch.randn(N, M, device="cuda")
        out, res = torch.empty(N, M, dtype=torch.int8, device="cuda"), torch.empty(N, M, device="cuda")
        scale = torch.empty(N, device="cuda")
        k = min(8, M)
        ids, wt = torch.empty(N, k, dtype=torch.int32, device="cuda"), torch.empty(N, k, device="cuda")

        def step():
            sm.q4_gemv(mat, x, M, K, 64, x_scale=xsd, y=y, workspace=ws)
            sm.add_norm(hid, delta=y, out=out, scale=scale, residual=res)
            sm.route(y, k, ids=ids, w=wt)
        step()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        for r in range(4):
            _, _, _, nx, _ = q4_case(N, M, K, 64, xt, "bf16", 40 + r)
            x.copy_(nx.cuda())
            ye = sm.q4_gemv(mat, x, M, K, 64, x_scale=xsd)          # its own workspace
            oe, se, re = sm.add_norm(hid, delta=ye, out_dtype=torch.int8)
            ie, we = sm.route(ye, k)
            ws.fill_(255)
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            for a, b in ((y, ye), (out, oe), (scale, se), (res, re), (ids, ie), (wt, we)):
                assert bool((a == b).all())


def test_concurrent_threads_and_streams(sm):
    """Four host threads at once, each with its own stream and workspace: every product, norm
    and choice equals the single-thread call bit for bit."""
    import threading

    import torch
    cases = []
    for i, (N, M, K, xt) in enumerate([(1, 500, 2048, "bf16"), (33, 200, 1024, "i8"),
                                       (300, 257, 640, "bf16"), (9, 300, 512, "f32")]):
        w, sc, bi, xv, xs = q4_case(N, M, K, 64, xt, "bf16", 50 + i)
        mat, x, xsd = to_mat(w, sc, bi), xv.cuda(), None if xs is None else xs.cuda()
        y = sm.q4_gemv(mat, x, M, K, 64, x_scale=xsd)
        cases.append((mat, x, xsd, M, K, y, sm.add_norm(y, out_dtype=torch.int8)[:2], sm.route(y, 8)))
    torch.cuda.synchronize()
    bad = []

    def work(i):
        mat, x, xsd, M, K, y, (o, s), (ids, wt) = cases[i]
        st = torch.cuda.Stream()
        try:
            for _ in range(16):
                y2 = sm.q4_gemv(mat, x, M, K, 64, x_scale=xsd, stream=st)
                o2, s2, _ = sm.add_norm(y2, out_dtype=torch.int8, stream=st)
                i2, w2 = sm.route(y2, 8, stream=st)
                st.synchronize()
                if not all(bool((a == b).all()) for a, b in ((y, y2), (o, o2), (s, s2), (ids, i2), (wt, w2))):
                    bad.append(i)
        except Exception as e:    # reported by the assertion below
            bad.append((i, repr(e)))
    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad, bad


def test_router_with_many_experts_near_the_choice(sm):
    """Scores so close that fp32 cannot order them (sigmoids of logits a unit apart in the
    last place, and all beyond 20 where they differ by less than 2^-24), in numbers below
    and above the 64 that are compared at once."""
    import torch
    for E in (40, 90, 300, 1000):
        for k in (1, 8, 33):
            base = torch.full((3, E), 0.25)
            step = torch.arange(E).flip(0).float() * 2.0 ** -24
            lg = torch.stack([base[0] + step * 2, 20 + step * 2.0 ** 5, base[2]])
            lg[2, ::3] = lg[2, ::3] + 2.0 ** -25
            check_route(sm, lg, min(k, E), "sigmoid")
            check_route(sm, lg, min(k, E), "sigmoid", (torch.arange(E) % 5).float() * 2.0 ** -20)
            check_route(sm, lg, min(k, E), "softmax")
