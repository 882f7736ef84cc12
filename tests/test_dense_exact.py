"""Inputs of the 4-bit product on which fp32 arithmetic makes no rounding, whatever the order of
its sums, and a CPU check that they tell exact arithmetic from less.

Everything is a whole number and the terms of an output add up to less than 2^24 in magnitude,
so every partial sum is an fp32 number and the result has to be equal, not near.
- kind "x": one large activation a row next to small ones.  In fp32 it is odd and has 18 bits,
  so its three bf16 parts (8 bits each) are all needed; in bf16 it is 2^17, so the group's sum
  has 18 bits and is odd or even by the small ones; 8-bit rows take the type's whole range.
- kind "b": activations of -1, 0 and 1 and large biases, so a weight s q + b has more bits than
  bf16 (9 with bf16 biases, 17 with fp32 ones).
"""
import pytest
import torch


def exact_case(N, M, K, group, x, s, kind, seed):
    """CPU tensors: codes uint8 [M][K], scales, biases [M][G], rows, their 8-bit scales."""
    g = torch.Generator()
    g.manual_seed(seed)
    G = K // group
    st = torch.float32 if s == "f32" else torch.bfloat16
    pick = lambda lo, hi, *shape: torch.randint(lo, hi, shape, generator=g)  # noqa: E731
    codes = pick(0, 16, M, K).to(torch.uint8)
    sc = torch.tensor([-2.0, -1.0, 1.0, 2.0])[pick(0, 4, M, G)]
    xs = None
    if kind == "x":
        bi = pick(-3, 4, M, G).float()
        if x == "i8":
            xv = pick(-128, 128, N, K).float()
            if K > 2048:
                xv[:, 2048:] = pick(-3, 4, N, K - 2048).float()
        else:
            xv = pick(-3, 4, N, K).float() * (torch.rand(N, K, generator=g) < 0.5)
            large = 2 ** 17 + (2 * pick(0, 2 ** 16, N) + 1 if x == "f32" else torch.zeros(N))
            xv[torch.arange(N), pick(0, K, N)] = large.float() * (2 * pick(0, 2, N) - 1).float()
    else:
        xv = pick(-1, 2, N, K).float()
        bi = ((256 + 2 * pick(0, 127, M, G)) * (2 * pick(0, 2, M, G) - 1)).float()
        if s == "f32":
            bi = pick(-3, 4, M, G).float()
            bi[torch.arange(M), pick(0, G, M)] = (2 ** 16 + 2 * pick(0, 2 ** 15, M) + 1).float()
    if x == "i8":
        xs = 2.0 ** pick(-4, 5, N).float()
    return codes, sc.to(st), bi.to(st), xv.to({"f32": torch.float32, "bf16": torch.bfloat16,
                                               "i8": torch.int8}[x]), xs


def exact_words(codes):
    M, K = codes.shape
    q = codes.view(M, K // 8, 8).to(torch.int64)
    w = sum(q[:, :, i] << (4 * i) for i in range(8))
    return torch.where(w >= 2 ** 31, w - 2 ** 32, w).to(torch.int32)


def exact_result(codes, sc, bi, xv, xs, group, rows=None, sums=None, weight=None):
    """The output in 64 bits (whole numbers below 2^24, times the rows' powers of two).  rows,
    sums, weight: roundings planted in the activations, the groups' sums, the weights."""
    N, K = xv.shape
    f = lambda t: t.double()  # noqa: E731
    x = f(xv) if rows is None else f(rows(xv))
    X = f(xv).view(N, K // group, group).sum(dim=2)
    if weight is None:
        w = f(codes) * f(sc).repeat_interleave(group, dim=1)
        y = x @ w.t() + (X if sums is None else f(sums(X))) @ f(bi).t()
        most = x.abs() @ w.abs().t() + X.abs() @ f(bi).abs().t()
        assert float(most.max()) < 2 ** 24
    else:
        w = f(weight(f(codes) * f(sc).repeat_interleave(group, dim=1) + f(bi).repeat_interleave(group, dim=1)))
        y = x @ w.t()
    return y if xs is None else y * f(xs)[:, None]


def parts(n):
    """The first n of the bf16 parts (truncated) of an fp32 number."""
    def cut(t):
        left, got = t.float(), torch.zeros_like(t, dtype=torch.float32)
        for _ in range(n):
            p = (left.view(torch.int32) & -65536).view(torch.float32)
            got, left = got + p, left - p
        return got
    return cut


SIZES = [(3, 40, 256, 64), (5, 33, 2048, 32), (20, 70, 1152, 128), (9, 50, 4224, 128)]


@pytest.mark.parametrize("N,M,K,group", SIZES)
def test_the_cases_tell_exact_arithmetic_from_less(N, M, K, group):
    for x in ("f32", "bf16", "i8"):
        for s in ("f32", "bf16"):
            for kind in ("x", "b"):
                c = exact_case(N, M, K, group, x, s, kind, 1)
                y = exact_result(*c, group)
                assert bool((y.float().double() == y).all())
                off = lambda **kw: float((exact_result(*c, group, **kw) != y).double().mean())  # noqa: E731
                assert off(rows=parts(3), sums=parts(3)) == 0
                # one output that differs tells; a tenth of them leaves no doubt
                if kind == "x" and x == "f32":
                    assert off(rows=parts(2)) > 0.1 and off(sums=parts(2)) > 0.1
                if kind == "x" and x == "bf16":
                    assert off(sums=parts(2)) > 0.1
                if kind == "b":
                    assert off(weight=lambda w: w.to(torch.bfloat16)) > 0.1


def test_the_words_hold_the_codes():
    codes = exact_case(1, 7, 128, 64, "bf16", "bf16", "x", 2)[0]
    w = exact_words(codes).to(torch.int64)
    for k in range(128):
        assert bool(((w[:, k // 8] >> (4 * (k % 8)) & 15) == codes[:, k]).all())
