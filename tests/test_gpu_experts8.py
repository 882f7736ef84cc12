"""GPU tests of the operators of 8-bit experts against their definitions in 64 bits or whole
numbers: the product of 8-bit integers (one matrix, and one an expert), rows sorted by expert
and back with their gradients, the SwiGLU step, and the routed layer made of them."""
import math
import sys

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

TYPES = {"f32": "float32", "bf16": "bfloat16", "i8": "int8"}


def say(*a):
    print("[case]", *a, file=sys.stderr, flush=True)


@pytest.fixture(scope="module")
def sm():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    from pseudo_random_weight_amd import seedmm
    return seedmm


def dt(name):
    import torch
    return getattr(torch, TYPES[name])


def gen(seed):
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def codes(g, *shape):
    import torch
    return torch.randint(-128, 128, shape, generator=g, device="cuda", dtype=torch.int8)


def scales(g, *shape, kind="f32"):
    import torch
    return (0.001 + 0.01 * torch.rand(*shape, generator=g, device="cuda")).to(dt(kind))


def product(x, xs, w, s, kind):
    """The product's definition: an exact sum (64-bit floats hold it), rounded to fp32, times the
    row's scale, times the channel's, rounded to y's type."""
    import torch
    if x.shape[0] == 0:
        return torch.empty(0, w.shape[0], device="cuda", dtype=dt(kind))
    d = torch.zeros(x.shape[0], w.shape[0], dtype=torch.float64, device="cuda")
    if x.shape[1]:
        d = torch.mm(x.double(), w.double().t().contiguous())
    return (d.to(torch.float32) * xs[:, None] * s.float()).to(dt(kind))


def same(a, b):
    """Equal bits, NaN with any payload."""
    import torch
    assert a.shape == b.shape and a.dtype == b.dtype
    ok = (a == b) | ((a != a) & (b != b))
    if not bool(ok.all()):
        at = (~ok).nonzero()[0].tolist()
        raise AssertionError(f"{int((~ok).sum())} of {ok.numel()} differ, first at {at}: "
                             f"{a[tuple(at)].item()} and {b[tuple(at)].item()}")


# ---- the product -------------------------------------------------------------------------

SIZES = [(1, 1, 1), (1, 16, 64), (1, 100, 2048), (1, 257, 1000), (1, 4096, 4100), (2, 33, 127), (3, 64, 128),
         (4, 130, 129), (5, 17, 4099), (8, 512, 1024), (15, 100, 513), (16, 256, 2048), (17, 31, 640),
         (31, 129, 100), (32, 2048, 2048), (33, 65, 4111), (61, 517, 4150), (64, 128, 256), (65, 300, 200),
         (100, 1000, 1000), (127, 255, 384), (128, 512, 777), (129, 513, 2048), (200, 64, 16), (256, 256, 256),
         (257, 1030, 1100), (300, 100, 3001), (512, 2048, 512), (700, 511, 129), (1025, 770, 900),
         (2048, 1024, 640), (4096, 96, 15), (7, 5, 0), (300, 300, 0), (300, 40, 17), (1, 70000, 32)]


@pytest.mark.parametrize("N,M,K", SIZES)
@pytest.mark.parametrize("s,y", [("f32", "f32"), ("bf16", "bf16")])
def test_product(sm, N, M, K, s, y):
    say("product", N, M, K, s, y)
    g = gen(N * 7919 + M * 31 + K)
    w, x = codes(g, M, K), codes(g, N, K)
    ws, xs = scales(g, M, kind=s), scales(g, N)
    got = sm.i8_gemv({"weight": w, "scales": ws}, x, xs, M, K, y_dtype=dt(y))
    same(got, product(x, xs, w, ws, y))


@pytest.mark.parametrize("N,M,K", [(1, 100, 200), (3, 70, 333), (16, 64, 256), (40, 130, 511), (130, 300, 640),
                                   (300, 257, 1000), (600, 520, 2080)])
@pytest.mark.parametrize("offset", [0, 1, 2, 8, 13])
def test_product_strides_and_alignment(sm, N, M, K, offset):
    """Rows anywhere, other elements left as they were."""
    import torch
    say("product strides", N, M, K, offset)
    g = gen(N + M + K + offset)
    for ldx, ldy in ((K, M), (K + 5, M + 3), (K + 16 - K % 16, M + 8)):
        xb = codes(g, N * ldx + 64)
        x = xb[offset:offset + N * ldx].view(N, ldx)[:, :K]
        wb = codes(g, M * K + 64)
        w = wb[offset:offset + M * K].view(M, K)
        yb = torch.full((N * ldy + 64,), 7.0, device="cuda", dtype=torch.bfloat16)
        y = yb[offset:offset + N * ldy].view(N, ldy)
        xs, ws = scales(g, N + 3)[3:], scales(g, M + 1)[1:]
        sm.i8_gemv({"weight": w, "scales": ws}, x, xs, M, K, y=y[:, :M])
        want = torch.full_like(yb, 7.0)
        want[offset:offset + N * ldy].view(N, ldy)[:, :M] = product(x, xs, w, ws, "bf16")
        same(yb, want)


@pytest.mark.parametrize("N", [1, 20, 200])
def test_product_largest_sums(sm, N):
    """-128 times -128 over the longest rows is 2^31 - 2^14."""
    import torch
    K, M = 131071, 40
    x = torch.full((N, K), -128, dtype=torch.int8, device="cuda")
    w = torch.full((M, K), -128, dtype=torch.int8, device="cuda")
    w[1::2] = 127
    one = torch.ones(max(N, M), device="cuda")
    y = sm.i8_gemv({"weight": w, "scales": one[:M]}, x, one[:N], M, K)
    want = torch.full((N, M), float(np.float32(16384 * K)), device="cuda")
    want[:, 1::2] = float(np.float32(-128 * 127 * K))
    same(y, want)


@pytest.mark.parametrize("N", [1, 30, 300])
def test_product_scales_without_value(sm, N):
    """A scale of NaN or infinity gives a row or a column without value and no other."""
    import torch
    g = gen(5)
    M, K = 70, 200
    w, x, ws, xs = codes(g, M, K), codes(g, N, K), scales(g, M), scales(g, N)
    ws[3], xs[N // 2], ws[69] = math.nan, math.inf, -math.inf
    y = sm.i8_gemv({"weight": w, "scales": ws}, x, xs, M, K)
    same(y, product(x, xs, w, ws, "f32"))
    xs[0] = math.nan      # as add_norm's row without value: codes 0
    x[0] = 0
    y = sm.i8_gemv({"weight": w, "scales": ws}, x, xs, M, K)
    assert bool(y[0].isnan().all())
    same(y[1:], product(x, xs, w, ws, "f32")[1:])


def sizes_to_offsets(counts):
    import torch
    return torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device="cuda")


GROUPS = [
    ([1], 0, 64, 128), ([0, 0, 0], 5, 20, 64), ([3, 0, 1, 0, 0, 7], 0, 100, 200), ([1] * 8, 0, 2048, 2048),
    ([0] * 40 + [1, 1] + [0] * 58, 3, 130, 513), ([5] * 100, 0, 96, 300), ([64, 64, 64], 0, 128, 128),
    ([65, 0, 63, 129, 1], 0, 200, 1000), ([300, 10, 0, 257], 20, 260, 520), ([16, 17, 15, 33, 31], 1, 48, 2100),
    ([700], 4, 300, 640), ([0, 700, 0], 0, 513, 129), ([40] * 70, 2, 33, 65), ([1000, 2, 500], 0, 1024, 2048),
    ([2] * 130 + [0] * 30 + [90], 0, 40, 100), ([128] * 6 + [256, 512], 0, 512, 256), ([9, 4], 0, 6, 0),
]


@pytest.mark.parametrize("case", range(len(GROUPS)))
@pytest.mark.parametrize("y", ["f32", "bf16"])
def test_grouped_product(sm, case, y):
    import torch
    counts, behind, M, K = GROUPS[case]
    E, N = len(counts), sum(counts) + behind
    say("grouped", case, E, N, M, K, y)
    g = gen(case)
    w, x, ws, xs = codes(g, E, M, K), codes(g, N, K), scales(g, E, M, kind=y), scales(g, N)
    out = torch.full((N, M + 2), 3.0, device="cuda", dtype=dt(y))
    sm.i8_gemv({"weight": w, "scales": ws}, x, xs, M, K, y=out[:, :M], offsets=sizes_to_offsets(counts))
    want = torch.full_like(out, 3.0)
    at = 0
    for e, n in enumerate(counts):
        want[at:at + n, :M] = product(x[at:at + n], xs[at:at + n], w[e], ws[e], y)
        at += n
    same(out, want)


def test_grouped_product_of_4096_experts(sm):
    import torch
    g = gen(9)
    E, M, K = 4096, 24, 48
    counts = torch.randint(0, 4, (E,), generator=g, device="cuda").cpu().numpy()
    counts[::3] = 0
    counts[4000] = 70
    N = int(counts.sum())
    w, x, ws, xs = codes(g, E, M, K), codes(g, N, K), scales(g, E, M), scales(g, N)
    y = sm.i8_gemv({"weight": w, "scales": ws}, x, xs, M, K, offsets=sizes_to_offsets(counts))
    e = torch.from_numpy(np.repeat(np.arange(E), counts)).cuda()
    d = (w[e].double() * x[:, None].double()).sum(dim=2)
    same(y, d.to(torch.float32) * xs[:, None] * ws[e])


def test_grouped_product_keeps_to_its_rows_with_wrong_offsets(sm):
    """Values outside of [0, N], falling ones and overlapping ones: nothing around y is written,
    nothing outside of x is read (the guards hold codes that would change a right row)."""
    import torch
    g = gen(10)
    N, M, K = 100, 64, 128
    for off in ([0, 10, 2 ** 31 - 1, 5], [-2 ** 31, 40, 20, 100], [90, 101, 300, 50], [0, 100, 0, 100],
                [-5, -3, -2, -1]):
        off = torch.tensor(off, dtype=torch.int32, device="cuda")
        w, x, ws, xs = codes(g, 3, M, K), codes(g, N, K), scales(g, 3, M), scales(g, N)
        yb = torch.full((N + 200, M), 5.0, device="cuda")
        sm.i8_gemv({"weight": w, "scales": ws}, x, xs, M, K, y=yb[100:100 + N], offsets=off)
        torch.cuda.synchronize()
        assert bool((yb[:100] == 5).all()) and bool((yb[100 + N:] == 5).all())


def test_a_row_does_not_depend_on_its_batch(sm):
    import torch
    g = gen(11)
    N, M, K = 600, 300, 1000
    w, x, ws, xs = codes(g, M, K), codes(g, N, K), scales(g, M), scales(g, N)
    mat = {"weight": w, "scales": ws}
    whole = sm.i8_gemv(mat, x, xs, M, K)
    for n in (1, 2, 5, 17, 40, 130, 300):
        same(sm.i8_gemv(mat, x[100:100 + n].contiguous(), xs[100:100 + n].contiguous(), M, K), whole[100:100 + n])
    one = sm.i8_gemv(mat, x[5], xs[5:6], M, K)
    assert one.shape == (M,)
    same(one, whole[5])


# ---- rows sorted by expert and back -------------------------------------------------------

def routing(seed, T, k, E, dropped=0.0, distinct=True):
    import torch
    r = np.random.default_rng(seed)
    if distinct and k <= E:
        ids = np.argsort(r.random((T, E)) + 0.3 * r.random(E), axis=1)[:, :k].astype(np.int64)
    else:
        ids = r.integers(0, E, (T, k))
    if dropped:
        gone = r.random((T, k)) < dropped
        ids[gone] = r.choice([-1, E, E + 5, -2 ** 31, 2 ** 31 - 1], size=int(gone.sum()))
    return torch.from_numpy(ids.astype(np.int32)).cuda()


def order(ids, E):
    """(inverse, offsets) by the definition, on the host."""
    flat = ids.cpu().numpy().astype(np.int64).ravel()
    live = (flat >= 0) & (flat < E)
    place = np.full(flat.size, -1)
    by = np.lexsort((np.nonzero(live)[0], flat[live]))
    place[np.nonzero(live)[0][by]] = np.arange(by.size)
    counts = np.bincount(flat[live], minlength=E)
    return place.reshape(ids.shape), np.concatenate([[0], np.cumsum(counts)])


ROUTES = [(1, 1, 1, 0.0), (1, 8, 100, 0.0), (1, 64, 64, 0.5), (2, 3, 5, 0.0), (7, 2, 300, 0.3), (64, 8, 100, 0.0),
          (100, 4, 7, 0.2), (33, 13, 512, 0.1), (256, 8, 64, 0.0), (257, 8, 64, 0.0), (500, 5, 20, 1.0),
          (700, 3, 4096, 0.1), (1000, 6, 100, 0.3), (64, 40, 50, 0.0), (2000, 1, 3, 0.0), (3000, 8, 100, 0.1),
          (129, 64, 128, 0.2), (5000, 7, 1, 0.5), (2048, 1, 9, 0.0), (2049, 1, 9, 0.0)]


@pytest.mark.parametrize("T,k,E,dropped", ROUTES)
@pytest.mark.parametrize("x,H", [("bf16", 64), ("f32", 37), ("i8", 100), ("i8", 7), ("bf16", 1030)])
def test_sort(sm, T, k, E, dropped, x, H):
    import torch
    say("sort", T, k, E, dropped, x, H)
    g = gen(T + k + E)
    ids = routing(T * k + E, T, k, E, dropped, distinct=T % 2 == 0 or k == 64)
    inv, off = order(ids, E)
    xs = None
    if x == "i8":
        xr, xs = codes(g, T, H), scales(g, T)
    else:
        xr = torch.randn(T, H, generator=g, device="cuda").to(dt(x))
    rows = torch.full((T * k + 2, H + 3), 5, device="cuda", dtype=dt(x))
    rs = None if xs is None else torch.full((T * k,), 9.0, device="cuda")
    got, sc, o, i = sm.moe_sort(xr, ids, E, x_scale=xs, rows=rows[:, :H], row_scale=rs)
    assert np.array_equal(o.cpu().numpy(), off) and np.array_equal(i.cpu().numpy(), inv)
    want = torch.full_like(rows, 5)
    t, s = np.nonzero(inv >= 0)
    place = torch.from_numpy(inv[t, s]).cuda()
    want[place, :H] = xr[torch.from_numpy(t).cuda()]
    assert torch.equal(rows, want)
    if xs is not None:
        ws = torch.full_like(rs, 9.0)
        ws[place] = xs[torch.from_numpy(t).cuda()]
        assert sc is rs and torch.equal(rs, ws)


@pytest.mark.parametrize("x", ["bf16", "i8"])
@pytest.mark.parametrize("offset", [0, 1, 3])
def test_sort_alignment(sm, x, offset):
    import torch
    T, k, E, H = 50, 4, 9, 333
    ids = routing(3, T, k, E)
    xb = codes(gen(1), T * (H + offset) + 16).to(dt(x))
    xr = xb[offset:offset + T * (H + offset)].view(T, H + offset)[:, :H]
    rows = torch.zeros(T * k * (H + 1) + 16, device="cuda", dtype=dt(x))[offset:offset + T * k * (H + 1)].view(T * k, H + 1)
    sm.moe_sort(xr, ids, E, rows=rows[:, :H])
    inv = torch.from_numpy(order(ids, E)[0]).cuda()
    for s in range(k):
        assert torch.equal(rows[inv[:, s], :H], xr)
    assert bool((rows[:, H] == 0).all())


def test_sort_of_no_tokens_and_of_no_columns(sm):
    import torch
    ids = torch.zeros(0, 4, dtype=torch.int32, device="cuda")
    _, _, off, inv = sm.moe_sort(torch.zeros(0, 8, device="cuda"), ids, 300)
    assert off.tolist() == [0] * 301 and inv.shape == (0, 4)
    ids = routing(4, 30, 2, 6, 0.2)
    rows, _, off, inv = sm.moe_sort(torch.zeros(30, 0, device="cuda"), ids, 6)
    i, o = order(ids, 6)
    assert np.array_equal(inv.cpu().numpy(), i) and np.array_equal(off.cpu().numpy(), o) and rows.shape == (60, 0)


BACK = [(1, 1, 1, 1), (1, 8, 100, 2048), (3, 2, 5, 7), (64, 8, 100, 512), (65, 3, 9, 513), (100, 9, 20, 130),
        (40, 64, 70, 300), (200, 5, 11, 2049), (17, 16, 40, 7167), (9, 17, 30, 64)]


def back_inputs(T, k, E, H, rows, dropped, seed):
    """Sorted rows with infinities and NaN in the rows that no slot names, weights without value
    in the slots without a row."""
    import torch
    g = gen(seed)
    ids = routing(seed, T, k, E, dropped)
    inv = torch.from_numpy(order(ids, E)[0].astype(np.int32)).cuda()
    r = (torch.randn(T * k, H, generator=g, device="cuda") * 2).to(dt(rows))
    w = torch.rand(T, k, generator=g, device="cuda") - 0.3
    named = torch.zeros(T * k, dtype=torch.bool, device="cuda")
    named[inv[inv >= 0].long()] = True
    r[~named] = math.nan
    w[inv < 0] = math.inf
    return g, inv, r, w


@pytest.mark.parametrize("T,k,E,H", BACK)
@pytest.mark.parametrize("rows,y", [("bf16", "f32"), ("f32", "f32"), ("f32", "bf16"), ("bf16", "bf16")])
@pytest.mark.parametrize("weighted,dropped", [(True, 0.3), (False, 0.0), (True, 1.0)])
def test_unsort(sm, T, k, E, H, rows, y, weighted, dropped):
    """k products and sums in fp32 are off by k 2^-24 of the sum of their sizes, to first order
    (1.01 covers the rest), and the result by half a step of its type."""
    import torch
    say("unsort", T, k, E, H, rows, y, weighted, dropped)
    _, inv, r, w = back_inputs(T, k, E, H, rows, dropped, T + k + H)
    yb = torch.full((T, H + 1), 7.0, device="cuda", dtype=dt(y))
    sm.moe_unsort(r, inv, w if weighted else None, y=yb[:, :H])
    want = torch.zeros(T, H, dtype=torch.float64, device="cuda")
    size = torch.zeros_like(want)
    for s in range(k):
        at = inv[:, s] >= 0
        v = r[inv[at, s].long()].double() * (w[at, s].double()[:, None] if weighted else 1.0)
        want[at] += v
        size[at] += v.abs()
    bound = 1.01 * k * 2.0 ** -24 * size
    if y == "bf16":
        bound = bound + 2.0 ** -8 * (want.abs() + bound)
    off = (yb[:, :H].double() - want).abs()
    assert bool((off <= bound).all()), float((off - bound).max())
    assert bool((yb[:, H] == 7).all())


def test_unsort_skips_places_outside_of_the_rows(sm):
    import torch
    r = torch.ones(6, 40, device="cuda")
    inv = torch.tensor([[0, 6, -1], [2 ** 31 - 1, 5, -2 ** 31], [7, -5, 100]], dtype=torch.int32, device="cuda")
    y = sm.moe_unsort(r, inv)
    assert y[:, 0].tolist() == [1.0, 1.0, 0.0] and bool((y == y[:, :1]).all())
    drows = torch.full_like(r, 4.0)
    _, dw = sm.moe_unsort_grad(torch.ones(3, 40, device="cuda"), r, inv, torch.full((3, 3), 2.0, device="cuda"),
                               drows=drows)
    assert dw.tolist() == [[40.0, 0, 0], [0, 40.0, 0], [0, 0, 0]]
    assert drows[:, 0].tolist() == [2.0, 4, 4, 4, 4, 2.0]


def grad_reference(dy, r, inv, w):
    import torch
    T, k = inv.shape
    dw = torch.zeros(T, k, dtype=torch.float64, device="cuda")
    size = torch.zeros_like(dw)
    drows = {}
    for s in range(k):
        at = inv[:, s] >= 0
        p = r[inv[at, s].long()].double() * dy[at].double()
        dw[at, s], size[at, s] = p.sum(dim=1), p.abs().sum(dim=1)
        drows[s] = (at, inv[at, s].long(), w[at, s].double()[:, None] * dy[at].double())
    return dw, size, drows


@pytest.mark.parametrize("T,k,E,H", BACK)
@pytest.mark.parametrize("rows,y", [("bf16", "f32"), ("f32", "bf16"), ("f32", "f32"), ("bf16", "bf16")])
@pytest.mark.parametrize("dropped", [0.0, 0.3])
def test_unsort_grad(sm, T, k, E, H, rows, y, dropped):
    """dw: a thread adds up at most 8 ceil(H / 512) products, then 6 sums over a wave and 3 over
    waves, each off by 2^-24 of the sum of sizes.  drows: one fp32 product, then the row's type."""
    import torch
    say("unsort grad", T, k, E, H, rows, y, dropped)
    g, inv, r, w = back_inputs(T, k, E, H, rows, dropped, T + k + H)
    dy = torch.randn(T, H, generator=g, device="cuda").to(dt(y))
    db = torch.full((T * k, H + 5), 3.0, device="cuda", dtype=dt(rows))
    _, dw = sm.moe_unsort_grad(dy, r, inv, w, drows=db[:, :H])
    want, size, drows = grad_reference(dy, r, inv, w)
    steps = 8 * math.ceil(H / 512) + 9
    off = (dw.double() - want).abs()
    assert bool((off <= 1.01 * steps * 2.0 ** -24 * size).all())
    assert bool((dw[inv < 0] == 0).all())
    named = torch.zeros(T * k, dtype=torch.bool, device="cuda")
    half = 2.0 ** -24 + (2.0 ** -8 if rows == "bf16" else 0.0)
    for s, (_, place, v) in drows.items():
        got = db[place, :H].double()
        assert bool(((got - v).abs() <= 1.01 * half * v.abs() + 2.0 ** -149).all())
        named[place] = True
    assert bool((db[~named] == 3).all()) and bool((db[:, H:] == 3).all())


def test_gradients_are_the_differences(sm):
    """The loss sum(dy * unsort(rows, w)) is linear in each row and in each weight: a change of
    one of them by a whole number changes it by that number times the gradient (small whole
    numbers: every sum is exact)."""
    import torch
    g = gen(21)
    T, k, E, H = 6, 3, 4, 40
    ids = routing(21, T, k, E, 0.2)
    x = torch.randint(-8, 9, (T, H), generator=g, device="cuda").float()
    dy = torch.randint(-8, 9, (T, H), generator=g, device="cuda").float()
    w = torch.randint(-4, 5, (T, k), generator=g, device="cuda").float()
    rows, _, _, inv = sm.moe_sort(x, ids, E, rows=torch.zeros(T * k, H, device="cuda"))
    drows, dw = sm.moe_unsort_grad(dy, rows, inv, w, drows=torch.zeros_like(rows))
    loss = lambda r, v: float((dy.double() * sm.moe_unsort(r, inv, v).double()).sum())  # noqa: E731
    base = loss(rows, w)
    for t, s in ((0, 0), (1, 2), (5, 1), (3, 0)):
        v = w.clone()
        v[t, s] += 2
        assert loss(rows, v) - base == 2 * float(dw[t, s])
    for p, h in ((0, 0), (4, 39), (9, 17), (T * k - 1, 3)):
        r = rows.clone()
        r[p, h] += 4
        assert loss(r, w) - base == 4 * float(drows[p, h])
    # the gradient of moe_sort: dx of sum(rows * drows)
    dx = sm.moe_unsort(drows, inv)
    for t, h in ((0, 5), (2, 0), (5, 39)):
        x2 = x.clone()
        x2[t, h] += 2
        r2 = sm.moe_sort(x2, ids, E, rows=torch.zeros_like(rows))[0]
        assert float(((r2 - rows).double() * drows.double()).sum()) == 2 * float(dx[t, h])


def test_unsort_grad_in_place(sm):
    import torch
    for T, k, H in ((30, 8, 700), (30, 20, 64)):
        g, inv, r, w = back_inputs(T, k, 50, H, "bf16", 0.2, 5)
        dy = torch.randn(T, H, generator=g, device="cuda")
        apart, dw = sm.moe_unsort_grad(dy, r, inv, w, drows=r.clone())
        over = r.clone()
        got, dw2 = sm.moe_unsort_grad(dy, over, inv, w, drows=over)
        same(got, apart)
        same(dw2, dw)


# ---- SwiGLU ------------------------------------------------------------------------------

def swiglu64(gu):
    import torch
    g, u = gu.double().chunk(2, dim=1)
    return g * torch.sigmoid(g) * u


@pytest.mark.parametrize("N,I", [(1, 1), (1, 1024), (3, 7), (64, 512), (65, 513), (20, 2048), (9, 2055), (5, 4100),
                                 (4, 8192), (3, 8200), (2, 20001), (513, 30)])
@pytest.mark.parametrize("x,out", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32"), ("f32", "bf16")])
def test_swiglu(sm, N, I, x, out):
    """exp is off by a step (2^-23) at most, which e / (1 + e) only makes smaller; the sum, the
    quotient and the products by half a step each: 6 half steps of fp32 for g >= 0 and 8 for g < 0
    (exp enters twice), then half a step of the output's type.  Below fp32's normal numbers an
    error of 2^-149 times what multiplies it stays."""
    import torch
    say("swiglu", N, I, x, out)
    g = gen(N + I)
    gu = (torch.randn(N, 2 * I + 3, generator=g, device="cuda") * 4).to(dt(x))
    gu[:, ::11] *= 20
    got = torch.full((N, I + 2), 7.0, device="cuda", dtype=dt(out))
    o, sc = sm.swiglu(gu[:, :2 * I], out=got[:, :I])
    assert sc is None
    want = swiglu64(gu[:, :2 * I])
    half = 8 * 2.0 ** -24 + (2.0 ** -8 if out == "bf16" else 0.0)
    tiny = 2.0 ** -149 * (4 + gu[:, :I].double().abs()) * (1 + gu[:, I:2 * I].double().abs())
    if out == "bf16":
        tiny = tiny + 2.0 ** -134
    off = (got[:, :I].double() - want).abs()
    assert bool((off <= 1.01 * half * want.abs() + tiny).all()), float((off / want.abs()).nan_to_num().max())
    assert bool((got[:, I:] == 7).all())


@pytest.mark.parametrize("x", ["bf16", "f32"])
def test_swiglu_over_the_whole_range(sm, x):
    """Gates whose exp under- and overflows, zeros, infinities and NaN."""
    import torch
    g = torch.tensor([0.0, -0.0, 1e-30, -1e-30, 20, -20, 80, -80, 88.8, -88.8, -100, 100, -103, -120, 1e4, -1e4,
                      3e38, -3e38, math.inf, math.nan], device="cuda").to(dt(x))
    for u in (1.0, -2.5, 1e-3, 1e5):
        gu = torch.stack([g, torch.full_like(g, u)]).t().contiguous()
        got = sm.swiglu(gu, out_dtype=torch.float32)[0][:, 0].double()
        want = swiglu64(gu)[:, 0]
        over = want.abs() > 3.5e38
        fin = torch.isfinite(want) & ~over & (want.abs() < 3.3e38)
        tiny = 2.0 ** -149 * (4 + g.double().abs()) * (1 + abs(u))
        assert bool(((got - want).abs() <= 1.01 * 8 * 2.0 ** -24 * want.abs() + tiny)[fin].all())
        assert bool(got[over].isinf().all())
        assert bool(got[-1].isnan()) and bool(got[-2].isinf())
    gu = torch.tensor([[-math.inf, 1.0], [math.inf, 0.0]], device="cuda").to(dt(x))
    assert bool(sm.swiglu(gu, out_dtype=torch.float32)[0].isnan().all())    # inf / inf, inf * 0


@pytest.mark.parametrize("N,I", [(1, 1), (7, 5), (64, 1024), (30, 513), (9, 2049), (5, 4096), (3, 8191), (2, 9000)])
@pytest.mark.parametrize("x", ["bf16", "f32"])
def test_swiglu_codes(sm, N, I, x):
    """A code is off by at most half a step and what fp32 adds: the value's 8 half steps and the
    scale's, its reciprocal's and the product's half steps, each times a code of up to 127."""
    import torch
    say("swiglu codes", N, I, x)
    g = gen(N * I)
    gu = (torch.randn(N, 2 * I, generator=g, device="cuda") * 3).to(dt(x))
    o, sc = sm.swiglu(gu, out_dtype=torch.int8)
    want = swiglu64(gu)
    top = want.abs().amax(dim=1)
    assert bool(((sc.double() - top / 127).abs() <= 10 * 2.0 ** -24 * top / 127 + 2.0 ** -149).all())
    v = want / sc.double()[:, None]
    assert bool(((o.double() - v).abs() <= 0.5 + 127 * 12 * 2.0 ** -24).all())
    assert int(o.min()) >= -127


def test_swiglu_rows_without_value_and_of_zeros(sm):
    import torch
    for I in (40, 700, 9000):
        gu = torch.randn(6, 2 * I, device="cuda")
        gu[1, 3], gu[2, I + 5], gu[3] = math.nan, math.inf, 0
        gu[4] *= 1e-30
        o, sc = sm.swiglu(gu, out_dtype=torch.int8)
        assert bool(sc[1].isnan()) and bool(sc[2].isnan()) and bool((o[1:5] == 0).all())
        assert float(sc[3]) == 2.0 ** -126 and float(sc[4]) == 2.0 ** -126
        assert int(o[0].abs().max()) == 127 and int(o[5].abs().max()) == 127


@pytest.mark.parametrize("I", [64, 1000, 9000])
@pytest.mark.parametrize("out", ["bf16", "i8", "f32"])
def test_swiglu_of_the_rows_that_exist(sm, I, out):
    import torch
    gu = torch.randn(50, 2 * I, device="cuda")
    whole, wsc = sm.swiglu(gu, out_dtype=dt(out))
    for n in (0, 1, 33, 50, 1000, -3):
        o = torch.full_like(whole, 7)
        sc = torch.full((50,), 7.0, device="cuda") if out == "i8" else None
        gu2 = gu.clone()
        live = min(max(n, 0), 50)
        gu2[live:] = math.nan
        sm.swiglu(gu2, out=o, scale=sc, count=torch.tensor([n], dtype=torch.int32, device="cuda"))
        same(o[:live], whole[:live])
        assert bool((o[live:] == 7).all())
        if sc is not None:
            same(sc[:live], wsc[:live])
            assert bool((sc[live:] == 7).all())


# ---- the layer ---------------------------------------------------------------------------

def layer_inputs(T, k, E, H, I, dropped=0.0, seed=0, s="f32"):
    import torch
    g = gen(seed)
    gu = {"weight": codes(g, E, 2 * I, H), "scales": (scales(g, E, 2 * I) * 0.05).to(dt(s))}
    dn = {"weight": codes(g, E, H, I), "scales": (scales(g, E, H) * 0.05).to(dt(s))}
    x, xs = codes(g, T, H), scales(g, T)
    ids = routing(seed, T, k, E, dropped)
    w = torch.rand(T, k, generator=g, device="cuda")
    return ids, w, x, xs, gu, dn


def layer_by_calls(sm, ids, w, x, xs, E, H, I, gu, dn):
    import torch
    rows, rs, off, inv = sm.moe_sort(x, ids, E, x_scale=xs)
    a = sm.i8_gemv(gu, rows, rs, 2 * I, H, y_dtype=torch.bfloat16, offsets=off)
    h, hs = sm.swiglu(a, out_dtype=torch.int8, count=off[E:])
    d = sm.i8_gemv(dn, h, hs, H, I, y_dtype=torch.bfloat16, offsets=off)
    return sm.moe_unsort(d, inv, w)


LAYERS = [(1, 8, 100, 2048, 1024, 0.0), (1, 1, 1, 1, 1, 0.0), (5, 2, 4, 64, 32, 0.0), (64, 8, 100, 256, 128, 0.1),
          (33, 3, 7, 100, 50, 0.3), (300, 4, 16, 512, 300, 0.2), (600, 6, 10, 333, 111, 0.0), (40, 2, 5, 128, 64, 1.0)]


@pytest.mark.parametrize("T,k,E,H,I,dropped", LAYERS)
@pytest.mark.parametrize("s", ["f32", "bf16"])
def test_layer_is_its_calls(sm, T, k, E, H, I, dropped, s):
    import torch
    say("layer", T, k, E, H, I, dropped, s)
    ids, w, x, xs, gu, dn = layer_inputs(T, k, E, H, I, dropped, T + H, s)
    ws = torch.full((sm.moe_i8_workspace_bytes(T, k, E, H, I),), 255, dtype=torch.uint8, device="cuda")
    y = sm.moe_i8(ids, w, x, xs, E, H, I, gu, dn, workspace=ws)
    same(y, layer_by_calls(sm, ids, w, x, xs, E, H, I, gu, dn))
    same(sm.moe_i8(ids, w, x, xs, E, H, I, gu, dn), y)
    gone = ((ids < 0) | (ids >= E)).all(dim=1)
    assert bool((y[gone] == 0).all())
    # a token alone
    t = T // 2
    same(sm.moe_i8(ids[t:t + 1], w[t:t + 1], x[t:t + 1], xs[t:t + 1], E, H, I, gu, dn), y[t:t + 1])


@pytest.mark.parametrize("T,k,E,H,I", [(9, 2, 5, 200, 60), (70, 4, 8, 256, 128)])
def test_layer_against_64_bits(sm, T, k, E, H, I):
    """Bounds by propagation: gate and up carry 2^-8 + 2^-22 of their sizes (bf16, fp32 scales), and
    |d silu| <= 1.1 |dg|; h's codes add half a scale; the down product carries those through |W|,
    its rows 2^-8 again, and the weighted sum k 2^-24."""
    import torch
    ids, w, x, xs, gu, dn = layer_inputs(T, k, E, H, I, 0.2, 3)
    y = sm.moe_i8(ids, w, x, xs, E, H, I, gu, dn)
    half = 2.0 ** -8 + 2.0 ** -22
    for t in range(T):
        want = torch.zeros(H, dtype=torch.float64, device="cuda")
        bound = torch.zeros_like(want)
        for s in range(k):
            e = int(ids[t, s])
            if not 0 <= e < E:
                continue
            xv = x[t].double() * xs[t].double()
            a = (gu["weight"][e].double() * gu["scales"][e].double()[:, None]) @ xv
            g, u = a[:I], a[I:]
            h = g * torch.sigmoid(g) * u
            eh = 1.1 * half * g.abs() * u.abs() * (1 + half) + (g * torch.sigmoid(g)).abs() * half * u.abs() \
                + 2.0 ** -20 * h.abs()
            eh = eh + 0.501 * ((h.abs() + eh).max() / 127)
            wd = dn["weight"][e].double() * dn["scales"][e].double()[:, None]
            d, ed = wd @ h, wd.abs() @ eh
            ed = ed + half * (d.abs() + ed)
            f = float(w[t, s])
            want += f * d
            bound += f * (ed + 1.01 * k * 2.0 ** -24 * (d.abs() + ed))
        assert bool(((y[t].double() - want).abs() <= bound).all())


def test_norm_router_and_layer_in_a_row(sm):
    """A layer on the residual stream: norm to 8 bits, router product, choice, experts, and the
    addition to the stream by the next norm."""
    import torch
    g = gen(31)
    T, E, k, H, I = 50, 16, 4, 256, 96
    _, _, _, _, gu, dn = layer_inputs(1, 1, E, H, I, 0, 7)
    r = torch.randn(T, H, generator=g, device="cuda")
    router = {"weight": torch.randint(-2 ** 31, 2 ** 31, (E, H // 8), generator=g, device="cuda",
                                      dtype=torch.int64).to(torch.int32).view(torch.uint32),
              "scales": torch.rand(E, H // 64, generator=g, device="cuda") * 0.01,
              "biases": -torch.rand(E, H // 64, generator=g, device="cuda") * 0.08}
    x, xs, _ = sm.add_norm(r, out_dtype=torch.int8)
    ids, w = sm.route(sm.q4_gemv(router, x, E, H, x_scale=xs), k)
    y = sm.moe_i8(ids, w, x, xs, E, H, I, gu, dn)
    same(y, layer_by_calls(sm, ids, w, x, xs, E, H, I, gu, dn))
    _, _, r2 = sm.add_norm(r, delta=y, out_dtype=torch.int8)
    same(r2, r + y)


# ---- streams, graphs, threads -------------------------------------------------------------

def everything(sm, T=70, k=4, E=9, H=200, I=72, seed=1, stream=None):
    """One call of each operator; its outputs."""
    import torch
    ids, w, x, xs, gu, dn = layer_inputs(T, k, E, H, I, 0.2, seed)
    rows8 = torch.zeros(T * k, H, dtype=torch.int8, device="cuda")
    rs = torch.zeros(T * k, device="cuda")
    yb = torch.zeros(T * k, 2 * I, device="cuda", dtype=torch.bfloat16)
    h, hs = torch.zeros(T * k, I, dtype=torch.int8, device="cuda"), torch.zeros(T * k, device="cuda")
    d, dr = torch.zeros(T * k, H, device="cuda"), torch.zeros(T * k, H, device="cuda")

    def run():
        rows, sc, off, inv = sm.moe_sort(x, ids, E, x_scale=xs, rows=rows8, row_scale=rs, stream=stream)
        sm.i8_gemv(gu, rows, sc, 2 * I, H, y=yb, offsets=off, stream=stream)
        sm.swiglu(yb, out=h, scale=hs, count=off[E:], stream=stream)
        sm.i8_gemv(dn, h, hs, H, I, y=d, offsets=off, stream=stream)
        y = sm.moe_unsort(d, inv, w, stream=stream)
        _, dw = sm.moe_unsort_grad(y, d, inv, w, drows=dr, stream=stream)
        whole = sm.moe_i8(ids, w, x, xs, E, H, I, gu, dn, stream=stream)
        return [rows, sc, off, inv, yb, h, hs, d, y, dr, dw, whole]
    return run, (x, xs, w)


@pytest.mark.parametrize("T", [3, 70, 900])
def test_captured_and_replayed(sm, T):
    """Replays read new inputs and give the eager call's bits, between the program's own work."""
    import torch
    run, (x, xs, w) = everything(sm, T=T)
    run()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        run()
        s.synchronize()
        with torch.cuda.graph(graph, stream=s):
            outs = run()
    for i in range(4):
        g = gen(100 + i)
        x.copy_(codes(g, *x.shape))
        xs.copy_(scales(g, *xs.shape))
        w.copy_(torch.rand(*w.shape, generator=g, device="cuda"))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got = [o.clone() for o in outs]
        want = [o.clone() for o in run()]
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            same(a, b)


def test_on_another_stream(sm):
    import torch
    run, _ = everything(sm)
    want = [o.clone() for o in run()]
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    other, _ = everything(sm, stream=st)
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        got = [o.clone() for o in other()]
    st.synchronize()
    for a, b in zip(got, want):
        same(a, b)
    with torch.cuda.stream(st):                # as the current stream
        run, _ = everything(sm)
        got = [o.clone() for o in run()]
    st.synchronize()
    for a, b in zip(got, want):
        same(a, b)


def test_two_calls_at_once(sm):
    import torch
    runs, wants = [], []
    streams = [torch.cuda.Stream() for _ in range(2)]
    for i, st in enumerate(streams):
        run, _ = everything(sm, T=600 + 300 * i, seed=40 + i, stream=st)
        torch.cuda.synchronize()
        outs = run()
        torch.cuda.synchronize()       # the calls are on st, the copies on the current stream
        wants.append([o.clone() for o in outs])
        runs.append(run)
    torch.cuda.synchronize()
    for _ in range(5):
        gots = []
        for st, run in zip(streams, runs):
            with torch.cuda.stream(st):
                gots.append([o.clone() for o in run()])
        torch.cuda.synchronize()
        for got, want in zip(gots, wants):
            for a, b in zip(got, want):
                same(a, b)


# ---- refusals of the Python entries --------------------------------------------------------

def test_refusals_on_gpu_tensors(sm):
    import torch
    z = lambda *s, d=torch.float32: torch.zeros(*s, dtype=d, device="cuda")  # noqa: E731
    i8, i32 = torch.int8, torch.int32
    mat = {"weight": z(16, 64, d=i8), "scales": z(16)}
    x, xs = z(3, 64, d=i8), z(3)
    bad = [
        lambda: sm.i8_gemv(mat, z(3, 64), xs, 16, 64), lambda: sm.i8_gemv(mat, x, None, 16, 64),
        lambda: sm.i8_gemv(mat, x, z(2), 16, 64), lambda: sm.i8_gemv(mat, x, xs, 17, 64),
        lambda: sm.i8_gemv(mat, x, xs, 16, 65), lambda: sm.i8_gemv(mat, x, xs, 16, 64, y=z(3, 15)),
        lambda: sm.i8_gemv(mat, x, xs, 16, 64, y=z(2, 16)), lambda: sm.i8_gemv(mat, x, xs, 16, 64, y=z(3, 16, d=i8)),
        lambda: sm.i8_gemv(mat, x, xs, 16, 64, offsets=z(1, d=i32)),
        lambda: sm.i8_gemv(mat, x, xs, 16, 64, offsets=z(3, d=i32)),
        lambda: sm.i8_gemv(mat, x, xs, 16, 64, offsets=z(2)),
        lambda: sm.i8_gemv(mat, x.t().contiguous().t(), xs, 16, 64),
        lambda: sm.i8_gemv(dict(mat, scales=z(16, d=i32)), x, xs, 16, 64),
        lambda: sm.i8_gemv(dict(mat, weight=z(16, 128, d=i8)[:, :64]), x, xs, 16, 64),
        lambda: sm.i8_gemv(mat, x, xs, 16, 131072), lambda: sm.i8_gemv(mat, x, xs, -1, 64),
        lambda: sm.i8_gemv(mat, x, xs.cpu(), 16, 64),
        lambda: sm.moe_sort(z(3, 8), z(4, 2, d=i32), 5), lambda: sm.moe_sort(z(3, 8), z(3, 2), 5),
        lambda: sm.moe_sort(z(3, 8), z(6, d=i32), 5), lambda: sm.moe_sort(z(3, 8), z(3, 65, d=i32), 5),
        lambda: sm.moe_sort(z(3, 8), z(3, 0, d=i32), 5), lambda: sm.moe_sort(z(3, 8), z(3, 2, d=i32), 4097),
        lambda: sm.moe_sort(z(3, 8), z(3, 2, d=i32), 5, rows=z(5, 8)),
        lambda: sm.moe_sort(z(3, 8), z(3, 2, d=i32), 5, rows=z(6, 7)),
        lambda: sm.moe_sort(z(3, 8), z(3, 2, d=i32), 5, rows=z(6, 8, d=torch.bfloat16)),
        lambda: sm.moe_sort(z(3, 8), z(3, 2, d=i32), 5, row_scale=z(6)),
        lambda: sm.moe_sort(z(3, 8), z(3, 2, d=i32), 5, x_scale=z(2)),
        lambda: sm.moe_sort(z(3, 8), z(3, 2, d=i32), 5, offsets=z(5, d=i32)),
        lambda: sm.moe_sort(z(3, 8), z(3, 2, d=i32), 5, inverse=z(3, 1, d=i32)),
        lambda: sm.moe_sort(z(3, 8), z(3, 2, d=i32), 5, workspace=3),
        lambda: sm.moe_sort(z(2000, 8), z(2000, 2, d=i32), 5, workspace=z(1)),
        lambda: sm.moe_sort(z(2000, 8), z(2000, 2, d=i32), 5, workspace=z(100000).t()[::2]),
        lambda: sm.moe_unsort(z(6, 8), z(3, 2, d=i32), z(3, 3)), lambda: sm.moe_unsort(z(6, 8), z(3, 2)),
        lambda: sm.moe_unsort(z(6, 8, d=i8), z(3, 2, d=i32)), lambda: sm.moe_unsort(z(6, 8), z(3, 2, d=i32), y=z(3, 9)),
        lambda: sm.moe_unsort(z(6, 8), z(3, 2, d=i32), y=z(4, 8)), lambda: sm.moe_unsort(z(6, 8), z(6, d=i32), y=z(3, 8)),
        lambda: sm.moe_unsort_grad(z(3, 9), z(6, 8), z(3, 2, d=i32), z(3, 2)),
        lambda: sm.moe_unsort_grad(z(4, 8), z(6, 8), z(3, 2, d=i32), z(3, 2)),
        lambda: sm.moe_unsort_grad(z(3, 8), z(6, 8), z(3, 2, d=i32), None),
        lambda: sm.moe_unsort_grad(z(3, 8), z(6, 8), z(3, 2, d=i32), z(3, 2), drows=z(5, 8)),
        lambda: sm.moe_unsort_grad(z(3, 8), z(6, 8), z(3, 2, d=i32), z(3, 2), drows=z(6, 8, d=torch.bfloat16)),
        lambda: sm.moe_unsort_grad(z(3, 8), z(6, 8), z(3, 2, d=i32), z(3, 2), dw=z(3, 1)),
        lambda: sm.swiglu(z(3, 7)), lambda: sm.swiglu(z(3, 8, d=i8)), lambda: sm.swiglu(z(3, 8), out=z(3, 8)),
        lambda: sm.swiglu(z(3, 8), out=z(2, 4)), lambda: sm.swiglu(z(3, 8), scale=z(3)),
        lambda: sm.swiglu(z(3, 8), out_dtype=i8, scale=z(2)), lambda: sm.swiglu(z(3, 8), count=z(0, d=i32)),
        lambda: sm.swiglu(z(3, 8), count=z(1)),
    ]
    gu, dn = {"weight": z(2, 8, 6, d=i8), "scales": z(2, 8)}, {"weight": z(2, 6, 4, d=i8), "scales": z(2, 6)}
    ok = dict(topk_ids=z(3, 2, d=i32), topk_w=z(3, 2), x=z(3, 6, d=i8), x_scale=z(3), E=2, H=6, I=4, gate_up=gu, down=dn)
    sm.moe_i8(**ok)
    for change in (dict(x=z(3, 7, d=i8)), dict(x=z(4, 6, d=i8)), dict(x=z(3, 12, d=i8)[:, :6]), dict(x_scale=z(2)),
                   dict(topk_w=z(3, 1)), dict(topk_ids=z(3, 2)), dict(E=3), dict(I=5), dict(H=7), dict(I=0),
                   dict(gate_up=dn), dict(down=gu | {"weight": z(2, 6, 3, d=i8)}), dict(y=z(3, 7)),
                   dict(y=z(3, 6, d=torch.bfloat16)), dict(workspace=z(4)), dict(workspace=5)):
        bad.append(lambda c=change: sm.moe_i8(**{**ok, **c}))
    for i, call in enumerate(bad):
        with pytest.raises((TypeError, ValueError, sm.SeedmmError)):
            call()
            raise AssertionError(f"call {i} was taken")
    torch.cuda.synchronize()
