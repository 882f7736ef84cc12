"""GPU tests of the operators of 8-bit experts at the borders of what their documentation
promises: rounding, what is read and written, many experts, and replays with other routings."""
import math
import sys

import pytest

from test_gpu_experts8 import codes, dt, gen, product, same, scales, sizes_to_offsets, swiglu64

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
