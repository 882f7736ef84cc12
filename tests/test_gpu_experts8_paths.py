"""GPU tests of the operators of 8-bit experts at the sizes where their kernels change, past 32-bit
offsets, where a launch is made in parts, and from several host threads, against their definitions
in 64 bits or whole numbers (the products' sums are whole, so every path gives the same bits)."""
import sys
import threading

import numpy as np
import pytest

from test_gpu_experts8 import codes, dt, everything, gen, layer_by_calls, layer_inputs, order, product, routing, same, \
    scales, sizes_to_offsets

pytestmark = pytest.mark.gpu


def say(*a):
    print("[case]", *a, file=sys.stderr, flush=True)


@pytest.fixture(scope="module")
def sm():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    from pseudo_random_weight_amd import seedmm
    return seedmm


# ---- the product: every kernel, its tails, its types -----------------------------------------

# rows, channels, columns.  Few rows: 16, 32 and 64 a workgroup, K over 2, 4 or 8 waves; tiles of 128
# channels by 64 and by 128 rows; 256 by 256, one tile, several a workgroup, and tiles in the last
# round for some of the workgroups only.  Columns 16 n, 16 n + 4 and odd for each.
FEW = [(1, 33000, 80), (16, 9000, 2064), (3, 9000, 8208), (17, 70000, 144), (32, 20000, 1040), (30, 3000, 8224),
       (33, 66000, 80), (48, 17000, 272), (64, 2000, 4112), (300, 200, 5008), (61, 5125, 4144), (64, 4096, 2064)]
MID = [(49, 8200, 2064), (100, 4100, 1040), (64, 4096, 4096), (256, 8190, 528), (257, 4097, 272), (1000, 1000, 4112),
       (512, 8200, 16), (513, 6400, 96)]
WIDE = [(2000, 7200, 144), (2049, 8190, 272), (4100, 8190, 80), (3600, 4608, 16), (3585, 4100, 1040), (5000, 7000, 112)]


@pytest.mark.parametrize("more", [0, 4, 8, 3])
@pytest.mark.parametrize("N,M,K", FEW + MID + WIDE)
def test_every_kernel_of_the_product(sm, N, M, K, more):
    K += more
    # types in turn
    s, y = ("f32", "bf16")[(N + more // 4) % 2], ("bf16", "f32")[(N + M + more // 4) % 2]
    say("product", N, M, K, s, y)
    g = gen(N + M + K)
    w, x = codes(g, M, K), codes(g, N, K)
    ws, xs = scales(g, M, kind=s), scales(g, N)
    got = sm.i8_gemv({"weight": w, "scales": ws}, x, xs, M, K, y_dtype=dt(y))
    same(got, product(x, xs, w, ws, y))


@pytest.mark.parametrize("s", ["f32", "bf16"])
@pytest.mark.parametrize("y", ["f32", "bf16"])
@pytest.mark.parametrize("N,M,K", [(300, 2050, 272), (300, 5000, 271), (2100, 7000, 148), (2100, 7000, 160)])
@pytest.mark.parametrize("offset", [0, 4, 20])
def test_tiles_of_each_type_on_4_bytes(sm, N, M, K, s, y, offset):
    """Rows of x and y with a stride, x and w on 4 but not on 16 bytes, y on an element."""
    import torch
    say("tiles", N, M, K, s, y, offset)
    g = gen(N + M + K + offset)
    ldx, ldy = K + 12 + (-K) % 4, M + 5
    x = codes(g, N * ldx + 64)[offset:offset + N * ldx].view(N, ldx)[:, :K]
    w = codes(g, M * K + 64)[offset:offset + M * K].view(M, K)
    yb = torch.full((N * ldy + 64,), 7.0, device="cuda", dtype=dt(y))
    out = yb[offset // 4:offset // 4 + N * ldy].view(N, ldy)
    xs, ws = scales(g, N + 1)[1:], scales(g, M + 1, kind=s)[1:]
    sm.i8_gemv({"weight": w, "scales": ws}, x, xs, M, K, y=out[:, :M])
    want = torch.full_like(yb, 7.0)
    want[offset // 4:offset // 4 + N * ldy].view(N, ldy)[:, :M] = product(x, xs, w, ws, y)
    same(yb, want)


# rows of each expert, rows behind the last, channels, columns
GROUPED = [
    ([1] * 300, 0, 2000, 272), ([3, 0, 8, 5] * 30, 2, 700, 1040), ([9, 10] * 40, 0, 400, 528),
    ([40, 0, 70, 64, 65, 1] * 6, 0, 520, 272), ([200] * 12, 7, 1100, 144), ([0, 1000, 1, 255, 600, 0], 3, 520, 1040),
    ([257] * 30, 0, 1030, 80), ([5000, 0, 0, 1], 0, 3000, 144), ([0] * 500 + [2100], 600, 4100, 48), ([0] * 64, 20000, 512, 64), ([16, 20, 11] * 20, 0, 300, 528),
]


@pytest.mark.parametrize("case", range(len(GROUPED)))
@pytest.mark.parametrize("more", [0, 4, 1])
def test_every_kernel_of_the_grouped_product(sm, case, more):
    import torch
    counts, behind, M, K = GROUPED[case]
    K += more
    E, N = len(counts), sum(counts) + behind
    s, y = ("f32", "bf16")[case % 2], ("bf16", "f32")[(case // 2 + more) % 2]
    say("grouped", case, E, N, M, K, s, y)
    g = gen(case + 50)
    w, x, ws, xs = codes(g, E, M, K), codes(g, N, K), scales(g, E, M, kind=s), scales(g, N)
    out = torch.full((N, M + 2), 3.0, device="cuda", dtype=dt(y))
    sm.i8_gemv({"weight": w, "scales": ws}, x, xs, M, K, y=out[:, :M], offsets=sizes_to_offsets(counts))
    want = torch.full_like(out, 3.0)
    at = 0
    for e, n in enumerate(counts):
        want[at:at + n, :M] = product(x[at:at + n], xs[at:at + n], w[e], ws[e], y)
        at += n
    same(out, want)


@pytest.mark.parametrize("N", [1500, 9000])
def test_tiles_keep_to_their_rows_with_wrong_offsets(sm, N):
    """Offsets that fall, overlap or leave [0, N]: nothing around y is written."""
    import torch
    g = gen(60)
    M, K, E = 640, 144, 5
    w, x, ws, xs = codes(g, E, M, K), codes(g, N, K), scales(g, E, M), scales(g, N)
    for off in ([0, 700, 2 ** 31 - 1, 5, 900, N], [-2 ** 31, 400, 200, 1000, 1000, 3], [N - 1, N + 1, 3 * N, 50, 0, N],
                [0, N, 0, N, 0, N], [-5, -4, -3, -2, -1, -1]):
        yb = torch.full((N + 600, M), 5.0, device="cuda")
        sm.i8_gemv({"weight": w, "scales": ws}, x, xs, M, K, y=yb[300:300 + N],
                   offsets=torch.tensor(off, dtype=torch.int32, device="cuda"))
        torch.cuda.synchronize()
        assert bool((yb[:300] == 5).all()) and bool((yb[300 + N:] == 5).all())


# ---- past 32 bits ------------------------------------------------------------------------------

@pytest.mark.parametrize("rows", [2, 70, 300])
def test_weights_past_32_bits(sm, rows):
    import torch
    E, M, K = 36, 8192, 8192                                     # 2.4 GB
    say("weights past 32 bits", rows)
    g = gen(rows)
    w = torch.empty(E, M, K, dtype=torch.int8, device="cuda")
    for e in (0, 17, E - 1):
        w[e] = codes(g, M, K)
    counts = [rows if e in (0, 17, E - 1) else 0 for e in range(E)]
    x, ws, xs = codes(g, 3 * rows, K), scales(g, E, M), scales(g, 3 * rows)
    y = sm.i8_gemv({"weight": w, "scales": ws}, x, xs, M, K, offsets=sizes_to_offsets(counts))
    for i, e in enumerate((0, 17, E - 1)):
        at = slice(i * rows, (i + 1) * rows)
        same(y[at], product(x[at], xs[at], w[e], ws[e], "f32"))


@pytest.mark.parametrize("N,ldx,K", [(600, 1 << 22, 272), (600, (1 << 22) + 16, 272), (600, (1 << 22) - 1, 272),
                                     (20, 1 << 27, 100), (2300, 1 << 20, 144)])
def test_x_past_32_bits(sm, N, ldx, K):
    import torch
    M = 7000
    say("x past 32 bits", N, ldx, K)
    g = gen(N)
    x = torch.empty(N, ldx, dtype=torch.int8, device="cuda")[:, :K]
    x.copy_(codes(g, N, K))
    w, ws, xs = codes(g, M, K), scales(g, M), scales(g, N)
    same(sm.i8_gemv({"weight": w, "scales": ws}, x, xs, M, K), product(x, xs, w, ws, "f32"))


@pytest.mark.parametrize("N,M,ldy,y", [(2200, 7000, 1 << 20, "f32"), (2200, 7000, (1 << 20) + 1, "bf16"), (300, 600, 1 << 23, "f32"),
                                       (2500, 300, (1 << 20) - 3, "bf16")])
def test_y_past_32_bits(sm, N, M, ldy, y):
    import torch
    K = 144
    say("y past 32 bits", N, M, ldy, y)
    g = gen(N)
    w, x, ws, xs = codes(g, M, K), codes(g, N, K), scales(g, M), scales(g, N)
    yb = torch.empty(N, ldy, dtype=dt(y), device="cuda")
    yb[:, M] = 7
    sm.i8_gemv({"weight": w, "scales": ws}, x, xs, M, K, y=yb[:, :M])
    same(yb[:, :M], product(x, xs, w, ws, y))
    assert bool((yb[:, M] == 7).all())


def test_rows_past_32_bits(sm):
    """Sorted rows, a sum's rows and gradients, and gate_up at offsets past 2^31 elements."""
    import torch
    T, k, E, H, ld = 700, 3, 9, 100, 1 << 21                     # 2100 rows of 2^21
    say("rows past 32 bits")
    g = gen(77)
    ids = routing(5, T, k, E, 0.1)
    inv = torch.from_numpy(order(ids, E)[0].astype(np.int32)).cuda()
    live = inv >= 0
    xb = torch.empty(T * k, ld, dtype=torch.bfloat16, device="cuda")
    x, rows = xb[:T, :H], torch.empty(T * k, ld, dtype=torch.bfloat16, device="cuda")[:, :H]
    x.copy_(torch.randn(T, H, generator=g, device="cuda"))
    sm.moe_sort(x, ids, E, rows=rows)
    want = x[:, None].expand(T, k, H)[live]
    assert torch.equal(rows[inv[live].long()], want)
    # the rows with numbers that are whole, so that every sum is exact
    small = torch.randint(-8, 9, (T * k, H), generator=g, device="cuda").to(torch.bfloat16)
    rows.copy_(small)
    w = torch.randint(-4, 5, (T, k), generator=g, device="cuda").float()
    near = small.float()[inv.clamp(min=0).long()] * (w * live)[..., None]
    y = sm.moe_unsort(rows, inv, w, y=torch.empty(T, 1 << 22, device="cuda")[:, :H])
    assert torch.equal(y, near.sum(1))
    dy = torch.randint(-8, 9, (T, H), generator=g, device="cuda").float()
    dr, dw = sm.moe_unsort_grad(dy, rows, inv, w, drows=xb[:, :H])
    assert torch.equal(dr[inv[live].long()].float(), (dy[:, None] * w[..., None])[live])
    assert torch.equal(dw, (small.float()[inv.clamp(min=0).long()] * dy[:, None]).sum(-1) * live)
    gu = xb[:, :2 * H]
    gu.copy_(torch.randn(T * k, 2 * H, generator=g, device="cuda"))
    same(sm.swiglu(gu)[0], sm.swiglu(gu.contiguous())[0])


# ---- launches in parts: more workgroups than one grid has ----------------------------------------

@pytest.mark.parametrize("K,M", [(1, (1 << 28) + 1000), (16, (1 << 27) + 3000)])
def test_product_in_parts(sm, K, M):
    import torch
    say("product in parts", K, M)
    g = gen(K)
    w = torch.empty(M, K, dtype=torch.int8, device="cuda")
    part = 1 << 24
    for m in range(0, M, part):
        w[m:m + part] = codes(g, min(part, M - m), K)
    x, one = codes(g, 1, K), torch.ones(1, device="cuda")
    y = sm.i8_gemv({"weight": w, "scales": torch.ones(M, device="cuda")}, x, one, M, K, y_dtype=torch.float32)
    for m in range(0, M, part):
        assert torch.equal(y[0, m:m + part], (w[m:m + part].float() * x[0].float()).sum(1))      # whole and small: exact


def test_rows_in_parts(sm):
    import torch
    T = (1 << 24) + 12345                                           # four tokens a workgroup, 2^22 workgroups
    say("rows in parts", T)
    g = gen(1)
    ids = torch.randint(-1, 3, (T, 1), generator=g, device="cuda", dtype=torch.int32)
    x = codes(g, T, 3)
    rows, _, off, inv = sm.moe_sort(x, ids, 3)
    live = ids[:, 0] >= 0
    where = torch.sort(torch.where(live, ids[:, 0], 3), stable=True)[1]
    n = int(live.sum())
    assert off.tolist() == [0] + [int((ids <= e).sum()) - (T - n) for e in range(3)]
    want = torch.full((T,), -1, dtype=torch.int32, device="cuda")
    want[where[:n]] = torch.arange(n, device="cuda", dtype=torch.int32)
    assert torch.equal(inv[:, 0], want) and torch.equal(rows[:n], x[where[:n]])
    r = rows[:n].to(torch.bfloat16)
    w = torch.ones(T, 1, device="cuda")
    y = sm.moe_unsort(r, inv, w)
    assert torch.equal(y, torch.where(live[:, None], x, 0).float())
    dr, dw = sm.moe_unsort_grad(y, r, inv, w)
    assert torch.equal(dr[:n], r) and torch.equal(dw[:, 0], (y * y).sum(1))


@pytest.mark.parametrize("out", ["bf16", "i8"])
def test_swiglu_in_parts(sm, out):
    import torch
    N = (1 << 24) + 777
    say("swiglu in parts", out)
    g = gen(2)
    gu = torch.randn(N, 2, generator=g, device="cuda").to(torch.bfloat16)
    got = sm.swiglu(gu, out_dtype=dt(out))
    few = sm.swiglu(gu[-5000:].contiguous(), out_dtype=dt(out))
    if out == "i8":
        same(got[1][-5000:], few[1])
    same(got[0][-5000:], few[0])


# ---- sorting: where its forms change --------------------------------------------------------------

@pytest.mark.parametrize("T,k,E", [(128, 8, 4096), (129, 8, 4096), (256, 8, 4096), (257, 8, 4096), (1024, 8, 1024), (1025, 8, 1024),
                                   (16384, 8, 64), (16385, 8, 64), (20000, 3, 700), (16, 64, 8), (17, 64, 4000), (512, 2, 4096)])
@pytest.mark.parametrize("H", [16, 1700])
def test_sort_where_its_form_changes(sm, T, k, E, H):
    import torch
    say("sort forms", T, k, E, H)
    g = gen(T + E)
    ids = routing(T + E, T, k, E, 0.05, distinct=False)            # one expert twice in a token, too
    inv, off = order(ids, E)
    x, xs = codes(g, T, H), scales(g, T)
    ws = torch.full((sm.moe_sort_workspace_bytes(T, k, E),), 255, dtype=torch.uint8, device="cuda")
    rows = torch.zeros(T * k, H, dtype=torch.int8, device="cuda")
    rs = torch.zeros(T * k, device="cuda")
    sm.moe_sort(x, ids, E, x_scale=xs, rows=rows, row_scale=rs, workspace=ws)
    _, _, o, i = sm.moe_sort(x, ids, E, x_scale=xs, rows=rows, row_scale=rs)
    assert np.array_equal(o.cpu().numpy(), off) and np.array_equal(i.cpu().numpy(), inv)
    t, s = np.nonzero(inv >= 0)
    place, t = torch.from_numpy(inv[t, s]).cuda(), torch.from_numpy(t).cuda()
    assert torch.equal(rows[place], x[t]) and torch.equal(rs[place], xs[t])
    assert bool((rows[int(off[-1]):] == 0).all()) and bool((rs[int(off[-1]):] == 0).all())


# ---- a padded batch, graphs, host threads -----------------------------------------------------------

@pytest.mark.parametrize("T,pad", [(5, 59), (64, 448), (300, 1748)])
def test_layer_of_a_padded_batch(sm, T, pad):
    """Rows of padding (no expert, codes and scales of any value) change no bit of the others, and
    give zeros."""
    import math
    import torch
    say("padded layer", T, pad)
    k, E, H, I = 4, 12, 300, 200
    ids, w, x, xs, gu, dn = layer_inputs(T + pad, k, E, H, I, 0.0, T)
    ids[T:], w[T:], xs[T:] = -1, math.nan, math.nan
    y = sm.moe_i8(ids, w, x, xs, E, H, I, gu, dn)
    same(y[:T], sm.moe_i8(ids[:T], w[:T], x[:T], xs[:T], E, H, I, gu, dn))
    assert bool((y[T:] == 0).all())


def test_two_graphs_share_a_workspace(sm):
    """Two captured layers with one workspace, replayed in turn on one stream."""
    import torch
    k, E, H, I = 4, 12, 256, 128
    args = [layer_inputs(T, k, E, H, I, 0.1, T) for T in (40, 700)]
    ws = torch.empty(sm.moe_i8_workspace_bytes(700, k, E, H, I), dtype=torch.uint8, device="cuda")
    ys = [torch.empty(a[2].shape[0], H, device="cuda") for a in args]
    st, graphs = torch.cuda.Stream(), []
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        for (ids, w, x, xs, gu, dn), y in zip(args, ys):
            sm.moe_i8(ids, w, x, xs, E, H, I, gu, dn, y=y, workspace=ws)
            st.synchronize()
            graphs.append(torch.cuda.CUDAGraph())
            with torch.cuda.graph(graphs[-1], stream=st):
                sm.moe_i8(ids, w, x, xs, E, H, I, gu, dn, y=y, workspace=ws)
    want = [layer_by_calls(sm, *a[:4], E, H, I, *a[4:]) for a in args]
    for i in range(6):
        for y in ys:
            y.fill_(7)
        torch.cuda.synchronize()
        with torch.cuda.stream(st):
            for g in graphs if i % 2 else graphs[::-1]:
                g.replay()
        torch.cuda.synchronize()
        for y, z in zip(ys, want):
            same(y, z)


def test_host_threads_at_once(sm):
    """Four host threads, each on a stream of its own, get the bits of calls alone."""
    import torch
    streams = [torch.cuda.Stream() for _ in range(4)]
    runs, wants = [], []
    for i, st in enumerate(streams):
        run, _ = everything(sm, T=(3, 64, 300, 1500)[i], seed=70 + i, stream=st)
        torch.cuda.synchronize()
        with torch.cuda.stream(st):
            wants.append([o.cpu() for o in run()])
        runs.append(run)
    errors, done = [], []

    def worker(i):
        try:
            for _ in range(8):
                with torch.cuda.stream(streams[i]):
                    outs = runs[i]()
                    streams[i].synchronize()
                    for a, b in zip(outs, wants[i]):
                        a = a.cpu()
                        if not bool(((a == b) | ((a != a) & (b != b))).all()):
                            errors.append(i)
            done.append(i)
        except Exception as e:      # reported by the main thread
            errors.append((i, repr(e)))

    threads = [threading.Thread(target=worker, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join(timeout=60)
    assert sorted(done) == [0, 1, 2, 3] and not errors, (done, errors)
