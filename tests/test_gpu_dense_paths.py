"""GPU tests of every kernel of the 4-bit product: which one a call takes is read from the
workspace it asks for, the results are exact where the inputs allow it (test_dense_exact), and
near the 64-bit result elsewhere.

Tolerance of the random cases, u = 2^-24: an output is a sum of products of which each passes
through at most PL group + 2 K / group + 24 additions (the group's sum over PL parts of the
activation, one fma a group and term, 8 elements' and 16 splits' sums), each off by at most 2 u
of the terms' sum S = sum (|s| q + |b|) |x| (u if it rounds, 2 u if it truncates)."""
import threading

import pytest

from test_dense_exact import exact_case, exact_result, exact_words
from test_gpu_dense import DT, U, q4_case, say, sm, to_mat  # noqa: F401

pytestmark = pytest.mark.gpu

# tokens, weight rows, columns; the kernel they take with bf16 or int8 rows
FEW = [(1, 100, 2048), (4, 17, 384), (16, 130, 2304), (9, 5000, 1152)]
RAW = [(20, 130, 1152), (64, 190, 2304), (61, 700, 4224)]           # rows ordered in the product
LAID_SPLIT = [(70, 8200, 4224)]                                      # 32-token tiles, K split
LAID_ONE = [(200, 10000, 1152)]                                      # 32-token tiles, one split
TWO = [(1100, 4000, 384), (1024, 4096, 128), (1090, 4100, 256)]      # 64-token tiles
FP32 = [(1, 100, 2048), (5, 130, 1152), (6, 100, 2304), (200, 300, 384), (1100, 4000, 256)]


def plan(sm, x, group, M, K, N):
    """(rows laid out in the workspace, splits of K), from the workspace's size."""
    up = lambda v: (v + 255) // 256 * 256  # noqa: E731
    planes = 3 if x == "f32" else 1
    got = sm.q4_workspace_bytes(DT[x], group, M, K, N)
    if got == 0:
        return False, 1
    Kp, Gp = up(K), (K // group + 15) // 16 * 16
    laid = up(planes * N * Kp * 2) + up(3 * N * Gp * 2)
    fits = [(at > 0, S) for at in (laid, 0) for S in range(1, 17)
            if got == at + (up(4 * S * N * M) if S > 1 else 0)]
    assert len(fits) == 1, (got, fits)
    return fits[0]


def wide_tiles(N, M):
    """64-token tiles are taken where there are 512 of them."""
    return -(-N // 64) * -(-M // 128) >= 512


@pytest.mark.parametrize("x", ["bf16", "i8"])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_the_sizes_take_the_kernels_they_are_meant_for(sm, x, group):
    for N, M, K in FEW:
        assert N <= 16 and plan(sm, x, group, M, K, N) == (False, 1)
    for N, M, K in RAW:
        laid, S = plan(sm, x, group, M, K, N)
        assert N > 16 and not laid and S > 1 and not wide_tiles(N, M)
    for N, M, K in LAID_SPLIT:
        laid, S = plan(sm, x, group, M, K, N)
        assert laid and S > 1 and not wide_tiles(N, M)
    for N, M, K in LAID_ONE:
        assert plan(sm, x, group, M, K, N) == (True, 1) and not wide_tiles(N, M)
    for N, M, K in TWO:
        assert plan(sm, x, group, M, K, N) == (True, 1) and wide_tiles(N, M)
    # tiles in multiples of 8 (renumbered over the XCDs) and not, more than one band of 512 tokens
    assert {-(-N // 64) * -(-M // 128) % 8 == 0 for N, M, K in TWO} == {True, False}
    assert {plan(sm, "f32", group, M, K, N) == (False, 1) for N, M, K in FP32} == {True, False}


def put(codes, sc, bi):
    return to_mat(exact_words(codes), sc, bi)


def check_exact(sm, N, M, K, group, x, s, kind):
    import torch
    say("exact", N, M, K, group, x, s, kind)
    case = exact_case(N, M, K, group, x, s, kind, 7)
    codes, sc, bi, xv, xs = case
    ref = exact_result(*(None if t is None else t.cuda() for t in case), group).cpu()
    mat, xd, xsd = put(codes, sc, bi), xv.cuda(), None if xs is None else xs.cuda()
    for y in (torch.float32, torch.bfloat16):
        got = sm.q4_gemv(mat, xd, M, K, group, x_scale=xsd, y_dtype=y)
        torch.cuda.synchronize()
        assert bool((got.cpu() == ref.float().to(y)).all())


@pytest.mark.parametrize("kind", ["x", "b"])
@pytest.mark.parametrize("s", ["bf16", "f32"])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("x,N,M,K", [(x, *n) for x in ("bf16", "i8") for n in FEW + RAW + LAID_SPLIT + LAID_ONE + TWO]
                         + [("f32", *n) for n in FP32])
def test_exact_products(sm, x, N, M, K, group, s, kind):
    check_exact(sm, N, M, K, group, x, s, kind)


@pytest.mark.parametrize("s,group", [("bf16", 64), ("f32", 32)])
@pytest.mark.parametrize("x,N,M,K", [(x, *n) for x in ("bf16", "i8") for n in RAW[-1:] + LAID_SPLIT + LAID_ONE + TWO]
                         + [("f32", *n) for n in FP32])
def test_random_products(sm, x, N, M, K, s, group):
    import torch
    say("random", N, M, K, group, x, s)
    w, sc, bi, xv, xs = (None if t is None else t.cuda() for t in q4_case(N, M, K, group, x, s, 8))
    got = sm.q4_gemv({"weight": w.view(torch.uint32), "scales": sc, "biases": bi}, xv, M, K, group, x_scale=xs)
    q = torch.stack([(w.to(torch.int64) >> (4 * i)) & 15 for i in range(8)], dim=2).view(M, K).double()
    sd, bd = sc.double().repeat_interleave(group, dim=1), bi.double().repeat_interleave(group, dim=1)
    xd = xv.double() if xs is None else xv.double() * xs.double()[:, None]
    ref = torch.mm(xd, (q * sd + bd).t().contiguous())
    S = torch.mm(xd.abs(), (q * sd.abs() + bd.abs()).t().contiguous())
    steps = group * (3 if x == "f32" else 1) + 2 * K // group + 24
    assert bool(((got.double() - ref).abs() <= 2 * steps * U * S + 2 * U * ref.abs() + 1e-37).all())


def large_cases(sm):
    """One call of each kernel for many tokens, with its result."""
    import torch
    out = []
    for x, (N, M, K) in [("bf16", TWO[0]), ("i8", TWO[2]), ("bf16", LAID_SPLIT[0]), ("i8", LAID_ONE[0]),
                         ("f32", FP32[4])]:
        case = exact_case(N, M, K, 64, x, "bf16", "x", 9)
        mat, xs = put(*case[:3]), None if case[4] is None else case[4].cuda()
        ref = exact_result(*(None if t is None else t.cuda() for t in case), 64).float()
        ws = torch.empty(sm.q4_workspace_bytes(DT[x], 64, M, K, N), dtype=torch.uint8, device="cuda")
        out.append((mat, case[3].cuda(), M, K, xs, ref, ws, torch.empty(N, M, device="cuda")))
    return out


def test_large_products_replay_like_eager(sm):
    """Captured with a workspace of the caller's that is overwritten between the replays, on
    inputs that change: every replay's rows are the eager call's."""
    import torch
    for mat, x, M, K, xs, ref, ws, y in large_cases(sm):
        say("captured", x.shape, M, K, x.dtype)
        first = x.clone()
        sm.q4_gemv(mat, x, M, K, 64, x_scale=xs, y=y, workspace=ws)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            sm.q4_gemv(mat, x, M, K, 64, x_scale=xs, y=y, workspace=ws)
        for r in range(4):
            x.copy_(first.roll(r, 0))
            want = sm.q4_gemv(mat, x, M, K, 64, x_scale=xs)      # its own workspace
            ws.fill_(255)
            y.fill_(7)
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            assert bool((y == want).all())
            if r == 0:
                assert bool((y == ref).all())


def test_large_products_at_once(sm):
    """Threads with a stream and a workspace each: the exact results, every time."""
    import torch
    cases = large_cases(sm)
    torch.cuda.synchronize()
    bad = []

    def work(i):
        mat, x, M, K, xs, ref, ws, y = cases[i]
        st = torch.cuda.Stream()
        try:
            for _ in range(6):
                with torch.cuda.stream(st):
                    y.fill_(7)
                sm.q4_gemv(mat, x, M, K, 64, x_scale=xs, y=y, workspace=ws, stream=st)
                st.synchronize()
                if not bool((y == ref).all()):
                    bad.append(i)
        except Exception as e:    # reported by the assertion below
            bad.append((i, repr(e)))
    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(cases))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad, bad


@pytest.mark.parametrize("x,N,M,K", [("f32", 3, 100, 256), ("f32", 40, 100, 256), ("bf16", 3, 100, 256),
                                     ("bf16", 40, 100, 256), ("bf16", 70, 8200, 4224)])
def test_activations_of_few_bits_stay_exact_down_to_2_to_the_minus_133(sm, x, N, M, K):
    """The exact inputs times 2^-90 .. 2^-130 (subnormal ones among them), scales times 2^60."""
    import torch
    case = exact_case(N, M, K, 64, x, "f32", "x", 5)
    ref = exact_result(*(None if t is None else t.cuda() for t in case), 64)
    mat = put(case[0], case[1] * 2.0 ** 60, case[2] * 2.0 ** 60)
    for e in (-90, -110, -126, -130):
        xv = (case[3].double() * 2.0 ** e).to(case[3].dtype)
        assert bool((xv.double() == case[3].double() * 2.0 ** e).all())
        got = sm.q4_gemv(mat, xv.cuda(), M, K, 64)
        torch.cuda.synchronize()
        assert bool((got.double() == ref * 2.0 ** (60 + e)).all()), e
