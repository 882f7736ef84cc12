"""GPU tests of the dense operators at the limits of what their calls accept: the longest
rows, values at the ends of the types' ranges, and what the Python entries refuse.
Tolerances are those of test_gpu_dense."""
import math

import pytest

from test_gpu_dense import (DT, U, block_case, check_norm, check_route, gen, norm_tol, q4_bound,  # noqa: F401
                            q4_ref, route_ref, say, sm)

pytestmark = pytest.mark.gpu


def test_norm_of_the_longest_row(sm):
    """H = 2^31 - 1: a thread's index passes 31 bits in the step that ends its loop."""
    import torch
    H = 2 ** 31 - 1
    say("norm", 1, H)
    g = torch.Generator(device="cuda")
    g.manual_seed(61)
    x = torch.empty(H + 64, dtype=torch.bfloat16, device="cuda")
    x.normal_(generator=g)
    out = torch.full((H + 64,), 9.0, dtype=torch.bfloat16, device="cuda")
    kept = x[H:].clone()
    sm.add_norm(x[:H], out=out[:H])
    torch.cuda.synchronize()
    step = 2 ** 26
    ss = sum(float((x[i:min(i + step, H)].double() ** 2).sum()) for i in range(0, H, step))
    f = 1 / math.sqrt(ss / H + 1e-6)
    tol = norm_tol(H)
    for i in range(0, H, step):
        v = x[i:min(i + step, H)].double() * f
        err = (out[i:min(i + step, H)].double() - v).abs()
        assert bool((err <= (tol + 2.0 ** -8 * (1 + tol)) * v.abs() + 1e-37).all()), i
    assert bool((out[H:] == 9).all()) and bool((x[H:] == kept).all())


def test_block_refuses_a_workspace_that_is_not_its_size(sm):
    """A workspace whose elements share memory, or lie apart, holds fewer bytes than it has
    elements: the layer would write past it."""
    import torch
    blk = block_case(sm, 8, 128, 64, 4, 2, "softmax", 1)[0]
    r = torch.zeros(3, 128, device="cuda")
    n = blk.workspace_bytes(3)
    one = torch.zeros(256, dtype=torch.uint8, device="cuda")
    for bad in (one[:1].expand(n), torch.zeros(2 * n, dtype=torch.uint8, device="cuda")[::2],
                torch.zeros(n, dtype=torch.uint8)):
        with pytest.raises(ValueError, match="workspace"):
            blk.moe(r, workspace=bad)
    with pytest.raises(TypeError, match="workspace"):
        blk.moe(r, workspace=one.data_ptr())
    with pytest.raises(sm.SeedmmError) as e:
        blk.moe(r, workspace=one)
    assert e.value.status == sm.EWORKSPACE
    torch.cuda.synchronize()
    assert bool((one == 0).all()) and bool((r == 0).all())


@pytest.mark.parametrize("E,k", [(3, 3), (40, 8), (100, 8), (512, 10), (512, 64), (4096, 64)])
def test_route_weights_of_tiny_sigmoids(sm, E, k):
    """Sigmoids below what fp32 holds: the weights are still their share of the sum, to 16 u
    (two roundings of the quotients, at most 6 of the sum, one of the division)."""
    import torch
    g = gen(62)
    noise = torch.randn(E, generator=g)
    rows = [noise - c for c in (60.0, 69.0, 88.0, 95.0, 104.0, 120.0, 400.0, 700.0)]
    rows += [torch.full((E,), -120.0), torch.linspace(-100, -102, E), torch.linspace(-40, -110, E)]
    for i in range(3):                 # masked among them, fewer than top_k left, one large
        r = noise - 130
        r[i::3 - i] = -math.inf
        rows.append(r)
    r = torch.full((E,), -math.inf)
    r[E - 1], r[E // 2] = -100.0, -101.0
    rows.append(r)
    r = noise - 100
    r[E // 3] = 0.5
    rows.append(r)
    lg = torch.stack(rows)
    bias = 0.1 * torch.randn(E, generator=g)
    for dt in (torch.float32, torch.bfloat16):
        check_route(sm, lg.to(dt), k, "sigmoid")
        check_route(sm, lg.to(dt), k, "sigmoid", bias)


@pytest.mark.parametrize("H", [1, 40, 2048, 7167, 16384, 30001, 40000])
@pytest.mark.parametrize("x", ["bf16", "f32"])
def test_add_norm_of_rows_whose_squares_leave_fp32(sm, x, H):
    """Rows so small or so large that their squares are no fp32 numbers, with eps of 0, of
    1e-6 and of their squares' size; next to ordinary rows, zeros, an infinity and a NaN."""
    import torch
    g = gen(63)
    base = 1 + torch.rand(H, generator=g)
    sign = torch.where(torch.rand(H, generator=g) < 0.5, -1.0, 1.0)
    sizes = (1e-37, 1e-30, 1e-25, 1e-21, 1e-19, 1e-15, 1.0, 1e15, 1e18, 1e19, 1e25, 1e37)
    rows = torch.stack([base * sign * c for c in sizes] + [torch.zeros(H), base, base]).to(DT[x])
    rows[3, H // 2] = 1e-30            # far apart in one row
    if H > 1:
        rows[9, H // 3] = 1e-15
    rows[-2, H - 1], rows[-1, 0] = math.inf, math.nan
    N, good = len(rows), range(len(sizes))
    w = (1 + 0.3 * torch.rand(H, generator=g)).to(torch.bfloat16)
    d = (rows.float().nan_to_num(0, 0, 0) * 0.25).to(DT[x])
    xd, wd, dd = rows.cuda(), w.cuda(), d.cuda()
    for eps in (0.0, 1e-6, 1e-38, 1e30):
        for delta, dc in ((None, None), (dd, d)):
            for out in ("f32", "bf16", "i8"):
                o, sc, res = sm.add_norm(xd, wd, delta=delta, eps=eps, out_dtype=DT[out])
                torch.cuda.synchronize()
                e32 = float(torch.tensor(eps, dtype=torch.float32))
                for n in good:
                    s = slice(n, n + 1)
                    say(H, x, eps, out, n)
                    check_norm(o[s], None if sc is None else sc[s], None if delta is None else res[s],
                               rows[s], None if dc is None else dc[s], w, e32, out, x)
                if out == "i8":
                    assert math.isnan(float(sc[N - 1])) and math.isnan(float(sc[N - 2]))
                    assert bool((o[N - 2:] == 0).all())
                    if eps:
                        assert bool((o[N - 3] == 0).all()) and float(sc[N - 3]) == 2.0 ** -126
                elif eps:
                    assert bool((o[N - 3] == 0).all())


# ---- more threads than HIP takes in one grid (2^32 in one dimension) --------------------

def around(n, part):
    """Indices at the start, the end and every multiple of `part`."""
    import torch
    at = set(range(min(4, n))) | set(range(max(0, n - 4), n))
    for b in range(part, n, part):
        at |= set(range(b - 2, min(b + 2, n)))
    return torch.tensor(sorted(at))


@pytest.mark.parametrize("N,H,threads", [(2 ** 26 + 9, 3, 64), (2 ** 24 + 7, 520, 256), (2 ** 20 + 3, 8193, 1024)])
def test_norm_of_more_rows_than_a_grid(sm, N, H, threads):
    import torch
    say("norm", N, H)
    g = torch.Generator(device="cuda")
    g.manual_seed(64)
    x = torch.empty(N, H, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    w = torch.rand(H, generator=g, device="cuda") + 0.5
    d = torch.empty(N, H, dtype=torch.bfloat16, device="cuda").normal_(generator=g) if H == 3 else None
    o = torch.empty(N, H, dtype=torch.int8, device="cuda")
    sc = torch.full((N,), -1.0, device="cuda")
    at = around(N, 2 ** 30 // threads)
    xv, dv = x[at.cuda()].cpu(), None if d is None else d[at.cuda()].cpu()
    sm.add_norm(x, w, delta=d, out=o, scale=sc, residual=None if d is None else x)
    torch.cuda.synchronize()
    assert bool((sc > 0).all())
    for i, n in enumerate(at.tolist()):
        s = slice(i, i + 1)
        check_norm(o[n:n + 1], sc[n:n + 1], None if d is None else x[n:n + 1], xv[s],
                   None if d is None else dv[s], w.cpu(), 1e-6, "i8", "bf16")
    if H == 3:
        assert bool((o.abs().amax(dim=1) == 127).all())


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_of_more_tokens_than_a_grid(sm, score):
    import torch
    T, E, k = 2 ** 26 + 5, 8, 2
    say("route", T, E, k, score)
    g = torch.Generator(device="cuda")
    g.manual_seed(65)
    lg = torch.empty(T, E, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    ids = torch.full((T, k), -1, dtype=torch.int32, device="cuda")
    w = torch.full((T, k), -1.0, device="cuda")
    sm.route(lg, k, score=score, ids=ids, w=w)
    torch.cuda.synchronize()
    assert bool((ids >= 0).all()) and bool(((w.sum(dim=1) - 1).abs() < 1e-6).all())
    at = around(T, 2 ** 24)
    ri, rw = route_ref(lg[at.cuda()].float().cpu().numpy(), k, score, None)
    assert (ids[at.cuda()].cpu().numpy() == ri).all()
    assert (abs(w[at.cuda()].cpu().numpy() - rw) <= 64 * U * rw).all()      # (2 span + 16) u, span < 24


@pytest.mark.parametrize("N,M,part", [(1, 2 ** 29 + 40, 2 ** 25), (65, 2 ** 28 + 200, 2 ** 28)])
def test_q4_of_more_weight_rows_than_a_grid(sm, N, M, part):
    """One token: in parts of 2^25 rows; 65 tokens (two tiles): of 2^21 tiles of 128 rows."""
    import torch
    K, group = 32, 32
    say("q4", N, M, K)
    g = torch.Generator(device="cuda")
    g.manual_seed(66)
    w = torch.empty(M, K // 8, dtype=torch.int32, device="cuda").random_(-2 ** 31, 2 ** 31 - 1, generator=g)
    sc = torch.empty(M, 1, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    bi = torch.empty(M, 1, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    x = torch.empty(N, K, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    y = torch.full((N, M), math.nan, dtype=torch.bfloat16, device="cuda")
    sm.q4_gemv({"weight": w.view(torch.uint32), "scales": sc, "biases": bi}, x, M, K, group, y=y)
    torch.cuda.synchronize()
    assert all(bool(torch.isfinite(r).all()) for r in y)
    at = around(M, part).cuda()
    ref, S = q4_ref(w[at].cpu(), sc[at].cpu(), bi[at].cpu(), x.cpu(), None, group)
    assert bool(((y[:, at].cpu().double() - ref).abs() <= q4_bound(ref, S, K, "bf16")).all())


def test_calls_let_other_python_threads_run(sm, tmp_path):
    """A call that waits (a launch can, for room in its queue) does not hold the interpreter:
    the library's functions are replaced by one that waits, two seconds at most, for a flag
    that another Python thread sets."""
    import ctypes
    import subprocess
    import threading
    import time

    import torch
    src, so = tmp_path / "wait.c", str(tmp_path / "wait.so")
    src.write_text("#include <unistd.h>\nvolatile int flag;\nint wait_flag(void) {\n"
                   "  for (int i = 0; i < 2000; ++i) { if (flag) return 0; usleep(1000); }\n"
                   "  return -1;\n}\n")
    subprocess.run(["gcc", "-shared", "-fPIC", "-o", so, str(src)], check=True)
    lib = ctypes.CDLL(so)
    flag = ctypes.c_int.in_dll(lib, "flag")
    address = lambda f: ctypes.cast(f, ctypes.c_void_p).value  # noqa: E731
    names = ("seedmm_q4_gemv", "seedmm_q4_workspace_bytes", "seedmm_add_norm", "seedmm_route")
    real = [address(getattr(sm.lib(), n)) for n in names]
    wait = address(lib.wait_flag)
    x = torch.zeros(2, 64, device="cuda")
    mat = {"weight": torch.zeros(16 * 8, dtype=torch.int32, device="cuda").view(torch.uint32),
           "scales": torch.zeros(16, device="cuda"), "biases": torch.zeros(16, device="cuda")}
    calls = (lambda: sm.q4_gemv(mat, x, 16, 64), lambda: sm.add_norm(x), lambda: sm.route(x, 2))
    for c in calls:
        c()
    torch.cuda.synchronize()

    def later():
        time.sleep(0.05)
        flag.value = 1
    sm._binding.init(wait, real[1], wait, wait, sm.SeedmmError)
    try:
        for c in calls:
            flag.value = 0
            t = threading.Thread(target=later)
            t.start()
            c()         # -1 of the wait would raise
            t.join()
    finally:
        sm._binding.init(*real, sm.SeedmmError)


def test_a_refused_scratch_allocation_is_torch_s_out_of_memory(sm):
    """As where the caller's own allocations fail; the next call works."""
    import torch
    N, M, K = 2 ** 20, 1, 32            # 1.6 GB of laid-out fp32 rows
    torch.cuda.empty_cache()
    x = torch.ones(N, K, device="cuda")
    mat = {"weight": torch.full((4,), 0x11111111, dtype=torch.int32, device="cuda").view(torch.uint32),
           "scales": torch.ones(1, device="cuda"), "biases": torch.zeros(1, device="cuda")}
    y = torch.empty(N, M, device="cuda")
    assert sm.q4_workspace_bytes(torch.float32, 32, M, K, N) > 2 ** 30
    total = torch.cuda.get_device_properties(0).total_memory
    torch.cuda.set_per_process_memory_fraction((torch.cuda.memory_reserved() + 2 ** 29) / total)
    try:
        with pytest.raises(torch.OutOfMemoryError):
            sm.q4_gemv(mat, x, M, K, 32, y=y)
    finally:
        torch.cuda.set_per_process_memory_fraction(1.0)
    sm.q4_gemv(mat, x, M, K, 32, y=y)
    torch.cuda.synchronize()
    assert bool((y == 32).all())
