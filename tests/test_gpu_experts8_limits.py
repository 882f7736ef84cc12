"""GPU tests of the operators of 8-bit experts at the borders of what their documentation
promises: rounding, what is read and written, many experts, and replays with other routings."""
import math
import sys

import numpy as np
import pytest

from test_gpu_experts8 import codes, dt, gen, layer_inputs, order, product, routing, same, scales, sizes_to_offsets, \
    swiglu64

pytestmark = pytest.mark.gpu


def say(*a):
    print("[case]", *a, file=sys.stderr, flush=True)


@pytest.fixture(scope="module")
def sm():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    from pseudo_random_weight_amd import seedmm
    return seedmm


# ---- SwiGLU's rounding -------------------------------------------------------------------------

@pytest.mark.parametrize("I", [256, 1024, 4000, 8000, 16384])
def test_swiglu_rounds_its_quotient_once(sm, I):
    """Gates of 4 .. 8 times a power of two: half a step of fp32 for the sum 1 + e, half a step for the
    quotient, and exp's step (2 half steps at most) times e / (1 + e) <= e^-4 = 0.0184: 2.04 half
    steps.  A quotient made of a reciprocal and a product has one rounding more."""
    import torch
    say("swiglu rounding", I)
    g = gen(I)
    N = (1 << 20) // I
    gu = torch.empty(N, 2 * I, device="cuda")
    gu[:, :I] = 4 + 4 * torch.rand(N, I, generator=g, device="cuda")
    gu[:, I:] = torch.tensor([1.0, -0.5, 4.0, 2.0 ** -20], device="cuda")[torch.randint(0, 4, (N, I), generator=g, device="cuda")]
    got, want = sm.swiglu(gu, out_dtype=torch.float32)[0].double(), swiglu64(gu)
    off = float(((got - want) / want).abs().max()) * 2.0 ** 24
    assert off <= 2.04, off


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("u", [1.0, -1e20, 1e30, 3e38])
def test_swiglu_of_gates_whose_exp_is_not_normal(sm, u, out):
    """exp(g) below 2^-126 is off by 2^-149 at most; so are its product with g and g's with the
    quotient, before they meet u.  The rest as in test_swiglu: 8 half steps, the output's, and half
    of the output's smallest number."""
    import torch
    g = torch.linspace(-112, -80, 4001, device="cuda")
    gu = torch.stack([g, torch.full_like(g, u)]).t().contiguous()
    got, want = sm.swiglu(gu, out_dtype=dt(out))[0][:, 0].double(), swiglu64(gu)[:, 0]
    half = 8 * 2.0 ** -24 + (2.0 ** -8 if out == "bf16" else 0.0)
    tiny = 2.0 ** -149 * (4 + g.double().abs()) * (1 + abs(u)) + (2.0 ** -134 if out == "bf16" else 0.0)
    assert bool(((got - want).abs() <= 1.01 * half * want.abs() + tiny).all())
    inf = torch.tensor([[-math.inf, u], [math.nan, u], [1.0, math.inf]], device="cuda")
    got = sm.swiglu(inf, out_dtype=dt(out))[0][:, 0]
    assert bool(got[:2].isnan().all()) and float(got[2]) == math.inf


# ---- the last channels of a tile ---------------------------------------------------------------

@pytest.mark.parametrize("N,M,K", [(2100, 7168, 32), (300, 4096, 64), (300, 4096, 65)])   # tiles of 256, of 128, of odd rows
@pytest.mark.parametrize("y", ["f32", "bf16"])
def test_last_channels_of_a_tile(sm, N, M, K, y):
    """Rows end at each place of a 16-byte piece, at the borders of 32, 64 and 128 channels, and on any
    element of y; the columns behind stay."""
    import torch
    g = gen(N + K)
    w, x = codes(g, M + 256, K), codes(g, N, K)
    ws, xs = scales(g, M + 256), scales(g, N)
    whole = product(x, xs, w, ws, y)
    for tail in (1, 2, 3, 4, 5, 6, 7, 8, 9, 31, 33, 63, 65, 95, 100, 127, 129, 135, 191, 250, 255):
        say("last channels", N, M + tail, K, y)
        m = M + tail
        for start in (0, 1):
            yb = torch.full((start + N * (m + 3),), 7.0, device="cuda", dtype=dt(y))
            out = yb[start:].view(N, m + 3)
            sm.i8_gemv({"weight": w[:m], "scales": ws[:m]}, x, xs, m, K, y=out[:, :m])
            same(out[:, :m], whole[:, :m])
            assert bool((out[:, m:] == 7).all()) and bool((yb[:start] == 7).all())


# ---- rows of fewer than 16 columns -------------------------------------------------------------

@pytest.mark.parametrize("K", range(18))
def test_rows_of_few_columns(sm, K):
    """Every length below a 16-byte piece and the first above, rows on any byte, whole and partial
    tiles, one matrix and many: codes behind a row's end belong to the next row and do not count."""
    import torch
    say("few columns", K)
    g = gen(K)
    for N, M in ((1, 1), (1, 70), (64, 64), (130, 200), (65, 63)):
        for ldx, offset in ((K, 0), (K + 5, 3)):
            x = codes(g, N * ldx + 16)[offset:offset + N * ldx].view(N, ldx)[:, :K]
            w = codes(g, M * K + 16)[offset:offset + M * K].view(M, K)
            xs, ws = scales(g, N), scales(g, M)
            same(sm.i8_gemv({"weight": w, "scales": ws}, x, xs, M, K), product(x, xs, w, ws, "f32"))
    counts = [0, 3, 0, 130, 1] * 60
    E, M, N = len(counts), 66, sum(counts) + 4
    w, x, ws, xs = codes(g, E, M, K), codes(g, N, K), scales(g, E, M), scales(g, N)
    out = torch.full((N, M), 3.0, device="cuda")
    sm.i8_gemv({"weight": w, "scales": ws}, x, xs, M, K, y=out, offsets=sizes_to_offsets(counts))
    e = torch.repeat_interleave(torch.arange(E, device="cuda"), torch.tensor(counts, device="cuda"))
    live = N - 4
    d = (w[e].double() * x[:live, None].double()).sum(dim=2)
    same(out[:live], d.float() * xs[:live, None] * ws[e])
    assert bool((out[live:] == 3).all())


# ---- offsets of any values ---------------------------------------------------------------------

WRONG = [lambda N: [0, N // 10, 2 ** 31 - 1, N // 20, N // 2, N], lambda N: [-2 ** 31, 2 * N // 5, N // 5, N, N, 3],
         lambda N: [N - 1, N + 1, 3 * N, N // 2, 0, N], lambda N: [0, N, 0, N, 0, N], lambda N: [-5, -4, -3, -2, -1, -1],
         lambda N: [-9, N // 3, N // 3, N + 7, 2 * N, 2 ** 31 - 1], lambda N: [N // 4, N // 4 + 1, N // 2, N // 2, N - 2, N - 1],
         lambda N: [N, N // 2, N // 3, N // 4, N // 5, 0]]


@pytest.mark.parametrize("N,K", [(20, 144), (100, 128), (400, 144), (400, 145), (1500, 144), (9000, 148), (9000, 163), (300, 15)])
@pytest.mark.parametrize("case", range(len(WRONG)))
def test_wrong_offsets_give_wrong_rows_only(sm, N, K, case):
    """Values are taken as the nearer end of [0, N].  Runs that do not overlap are exact; a row that
    several experts claim holds values of theirs or its old ones; a row of none stays.  Around x, its
    scales, the weights and y lie other codes, NaN and marks: a row read beside them would show."""
    import torch
    say("wrong offsets", N, K, case)
    g = gen(N + K)
    M, E, pad = 640, 5, 300
    x = codes(g, N + 2 * pad, K)[pad:pad + N]
    xsb = torch.full((N + 2 * pad,), math.nan, device="cuda")
    xs = xsb[pad:pad + N]
    xs.copy_(scales(g, N))
    w, ws = codes(g, E + 2, M, K)[1:-1], scales(g, E, M)
    off = WRONG[case](N)
    yb = torch.full((N + 2 * pad, M), 5.0, device="cuda")
    sm.i8_gemv({"weight": w, "scales": ws}, x, xs, M, K, y=yb[pad:pad + N],
               offsets=torch.tensor(off, dtype=torch.int32, device="cuda"))
    ends = [min(max(v, 0), N) for v in off]
    runs = [(e, a, b) for e, (a, b) in enumerate(zip(ends, ends[1:])) if a < b]
    claims = torch.zeros(N, dtype=torch.int32, device="cuda")
    for _, a, b in runs:
        claims[a:b] += 1
    y = yb[pad:pad + N]
    fits = (y == 5) & (claims != 1)[:, None]
    for e, a, b in runs:
        fits[a:b] |= y[a:b] == product(x[a:b], xs[a:b], w[e], ws[e], "f32")
    if sum(b - a for _, a, b in runs) > N:         # more tiles than there can be: some of them may be left out
        fits |= y == 5
    assert bool(fits.all())
    assert bool((yb[:pad] == 5).all()) and bool((yb[pad + N:] == 5).all())


# ---- bytes beside the tensors --------------------------------------------------------------------

@pytest.mark.parametrize("N,M,K", [(1, 100, 2049), (1, 33, 16), (16, 64, 258), (40, 130, 511), (300, 6600, 65), (1000, 3200, 71)])
@pytest.mark.parametrize("offset", [1, 2, 3])
def test_bytes_beside_the_rows_do_not_count(sm, N, M, K, offset):
    """Weights and x on any byte, x as a whole and with rows apart: whatever stands in front of them,
    behind them and between the rows, the bits are the same."""
    import torch
    say("bytes beside", N, M, K, offset)
    g = gen(N + K + offset)
    for ldx in (K, K + 3):
        x, w, xs, ws = codes(g, N, K), codes(g, M, K), scales(g, N), scales(g, M)
        want = product(x, xs, w, ws, "f32")
        for beside in (0, 127, -128, None):
            xb, wb = codes(g, N * ldx + 8), codes(g, M * K + 8)
            if beside is not None:
                xb.fill_(beside)
                wb.fill_(beside)
            xv, wv = xb[offset:offset + N * ldx].view(N, ldx)[:, :K], wb[4 - offset:4 - offset + M * K].view(M, K)
            xv.copy_(x)
            wv.copy_(w)
            same(sm.i8_gemv({"weight": wv, "scales": ws}, xv, xs, M, K), want)


# ---- captured calls with another routing at each replay ------------------------------------------

@pytest.mark.parametrize("T,k,E,H,I", [(3, 4, 9, 200, 72),          # sorted in one launch
                                       (70, 4, 9, 200, 72), (900, 4, 9, 204, 72),       # by chunks, summed directly
                                       (2500, 8, 600, 48, 32),      # by chunks, summed once for all
                                       (1600, 2, 5, 160, 96)])      # tiles of 256 rows
def test_replays_with_other_routings(sm, T, k, E, H, I):
    """The order, the offsets, the number of rows that exist and the tiles' experts are new at each
    replay: random ones, all slots dropped, all tokens at one expert, none dropped.  Outputs and scratch
    hold other values before it."""
    import torch
    say("replays", T, k, E, H, I)
    ids, w, x, xs, gu, dn = layer_inputs(T, k, E, H, I, 0.2, T)
    bf, f32, i8, i32 = torch.bfloat16, torch.float32, torch.int8, torch.int32
    shapes = {"rows": ((T * k, H), i8), "scale": ((T * k,), f32), "off": ((E + 1,), i32), "inv": ((T, k), i32),
              "a": ((T * k, 2 * I), bf), "h": ((T * k, I), i8), "hs": ((T * k,), f32), "d": ((T * k, H), f32),
              "y": ((T, H), f32), "dr": ((T * k, H), f32), "dw": ((T, k), f32), "layer": ((T, H), f32)}
    n_ws = sm.moe_sort_workspace_bytes(T, k, E)

    def buffers():
        b = {n: torch.empty(s, dtype=t, device="cuda") for n, (s, t) in shapes.items()}
        b["sort_ws"] = torch.empty(n_ws, dtype=torch.uint8, device="cuda") if n_ws else None
        b["layer_ws"] = torch.empty(sm.moe_i8_workspace_bytes(T, k, E, H, I), dtype=torch.uint8, device="cuda")
        return b

    def poison(b, v):
        for t in b.values():
            if t is not None:
                t.fill_(v)

    def run(b):
        sm.moe_sort(x, ids, E, x_scale=xs, rows=b["rows"], row_scale=b["scale"], offsets=b["off"], inverse=b["inv"],
                    workspace=b["sort_ws"])
        sm.i8_gemv(gu, b["rows"], b["scale"], 2 * I, H, y=b["a"], offsets=b["off"])
        sm.swiglu(b["a"], out=b["h"], scale=b["hs"], count=b["off"][E:])
        sm.i8_gemv(dn, b["h"], b["hs"], H, I, y=b["d"], offsets=b["off"])
        sm.moe_unsort(b["d"], b["inv"], w, y=b["y"])
        sm.moe_unsort_grad(b["y"], b["d"], b["inv"], w, drows=b["dr"], dw=b["dw"])
        sm.moe_i8(ids, w, x, xs, E, H, I, gu, dn, y=b["layer"], workspace=b["layer_ws"])

    got, want = buffers(), buffers()
    st, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    run(got)
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        run(got)
        st.synchronize()
        with torch.cuda.graph(graph, stream=st):
            run(got)
    one = torch.full((T, k), E // 2, dtype=i32, device="cuda")
    for i, new in enumerate([routing(1, T, k, E, 0.5), torch.full_like(ids, -1), one, routing(2, T, k, E, 0.0),
                             torch.where(one > 0, torch.full_like(one, E + 3), one), routing(3, T, k, E, 0.9), one.clone()]):
        ids.copy_(new)
        poison(got, 77)
        poison(want, 99)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        run(want)
        inv, off = order(new, E)
        assert np.array_equal(got["off"].cpu().numpy(), off) and np.array_equal(got["inv"].cpu().numpy(), inv), i
        live = int(off[-1])
        for n in ("off", "inv", "y", "dw", "layer"):
            same(got[n], want[n])
        for n in ("rows", "scale", "a", "h", "hs", "d", "dr"):
            same(got[n][:live], want[n][:live])
            assert bool((got[n][live:] == 77).all()) and bool((want[n][live:] == 99).all()), (i, n)
        gone = torch.from_numpy((inv < 0).all(axis=1)).cuda()
        assert bool((got["layer"][gone] == 0).all())
        if live:
            same(got["rows"][torch.from_numpy(inv[inv >= 0]).cuda()], x.repeat_interleave(k, dim=0)[torch.from_numpy((inv >= 0).ravel()).cuda()])


# ---- the layer's bf16 rows -----------------------------------------------------------------------

@pytest.mark.parametrize("T,k,E,H,I", [(1, 8, 100, 512, 256), (64, 8, 100, 512, 256), (900, 4, 9, 200, 72)])
def test_layer_rows_cost_half_a_step_of_bf16(sm, T, k, E, H, I):
    """The five calls with fp32 rows behind the down product: the layer differs from them by half a
    step of bf16 (2^-8) of each slot's row at most, and both sums' k half steps of fp32."""
    import torch
    say("layer's rows", T, k, E, H, I)
    ids, w, x, xs, gu, dn = layer_inputs(T, k, E, H, I, 0.1, T)
    rows, rs, off, inv = sm.moe_sort(x, ids, E, x_scale=xs)
    a = sm.i8_gemv(gu, rows, rs, 2 * I, H, y_dtype=torch.bfloat16, offsets=off)
    h, hs = sm.swiglu(a, out_dtype=torch.int8, count=off[E:])
    d = sm.i8_gemv(dn, h, hs, H, I, y_dtype=torch.float32, offsets=off)
    sizes = sm.moe_unsort(d.abs(), inv, w).double()             # w >= 0
    y, y32 = sm.moe_i8(ids, w, x, xs, E, H, I, gu, dn), sm.moe_unsort(d, inv, w)
    assert bool(((y.double() - y32.double()).abs() <= sizes * (2.0 ** -8 + 3 * k * 2.0 ** -24)).all())


# ---- gradients -----------------------------------------------------------------------------------

def test_gradients_through_a_function_of_the_callers(sm):
    """The calls record no graph; a torch.autograd.Function made of them has the plain form's gradients.
    Whole numbers, so that both are exact."""
    import torch
    T, k, E, H = 40, 3, 7, 96
    g = gen(5)
    ids = routing(5, T, k, E, 0.3)

    class Mix(torch.autograd.Function):          # sort, then back with weights
        @staticmethod
        def forward(ctx, x, w):
            rows, _, _, inv = sm.moe_sort(x, ids, E)
            ctx.save_for_backward(rows, inv, w)
            return sm.moe_unsort(rows, inv, w)

        @staticmethod
        def backward(ctx, dy):
            rows, inv, w = ctx.saved_tensors
            drows, dw = sm.moe_unsort_grad(dy.contiguous(), rows, inv, w)
            return sm.moe_unsort(drows, inv), dw

    x = torch.randint(-9, 10, (T, H), generator=g, device="cuda").float().requires_grad_()
    w = torch.randint(-4, 5, (T, k), generator=g, device="cuda").float().requires_grad_()
    dy = torch.randint(-9, 10, (T, H), generator=g, device="cuda").float()
    live = ((ids >= 0) & (ids < E)).float()
    want = torch.autograd.grad((x * (w * live).sum(dim=1, keepdim=True) * dy).sum(), (x, w))
    got = torch.autograd.grad((Mix.apply(x, w) * dy).sum(), (x, w))
    same(got[0], want[0])
    same(got[1], want[1])
    rows, _, _, inv = sm.moe_sort(x, ids, E)
    assert not rows.requires_grad and not sm.moe_unsort(rows, inv, w).requires_grad
    assert not sm.swiglu(x)[0].requires_grad
