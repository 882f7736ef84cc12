"""GPU tests of the product's kernels by name: cases that a call takes to a certain kernel (which
one is checked on the CPU, test_experts8_choice), for each pair of types, and with more experts than
a wave searches at once (64) and than its loads hold (256).  Sums are whole, so every kernel gives
the same bits."""
import sys

import numpy as np
import pytest

from test_gpu_experts8 import codes, dt, gen, product, same, scales, sizes_to_offsets

pytestmark = pytest.mark.gpu


def say(*a):
    print("[case]", *a, file=sys.stderr, flush=True)


@pytest.fixture(scope="module")
def sm():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    from pseudo_random_weight_amd import seedmm
    return seedmm


TYPES = [(s, y) for s in ("f32", "bf16") for y in ("f32", "bf16")]

# kernel (tiles of 64 times these), rows, channels, columns; every pair of types
ONE = [
    ("k_i8_mid<2, 1", 300, 4100, 80), ("k_i8_mid<2, 1", 257, 4500, 132),
    ("k_i8_mid<2, 2", 1000, 3200, 80), ("k_i8_mid<2, 2", 1001, 3300, 156),
    ("k_i8_odd<2, 1", 300, 6600, 65), ("k_i8_odd<2, 1", 257, 6800, 130),
    ("k_i8_odd<2, 2", 1000, 3200, 71), ("k_i8_odd<2, 2", 1001, 3300, 257),
    ("k_i8_wide", 3500, 4608, 1024), ("k_i8_wide", 2000, 7200, 148), ("k_i8_wide", 1536, 8190, 1536),
    # several tiles a workgroup, and a last round for some of the workgroups only
    ("k_i8_wide", 5000, 7600, 272), ("k_i8_wide", 4100, 8190, 324), ("k_i8_wide", 9000, 5003, 1024),
]


def uneven(seed, E, most, empty=()):
    """Rows of E experts, 0 .. most, none for some of them."""
    n = np.random.default_rng(seed).integers(0, most + 1, E)
    n[list(empty)] = 0
    return n.tolist()


# kernel, rows of each expert, rows behind the last, channels, columns.  Several tiles of channels, and
# of rows for one expert; no rows at the borders of what is searched at once; all of the rows with few
# experts in front or behind.
MANY = [
    ("k_i8_wide", [300] * 62 + [0, 0, 700], 3, 300, 80),
    ("k_i8_wide", uneven(1, 100, 800, (63, 64)), 0, 300, 84),
    ("k_i8_wide", [200] * 254 + [0, 0, 1500], 0, 520, 48),
    ("k_i8_wide", [0] * 300 + [60000] + [0] * 5 + [257] * 294, 0, 300, 80),
    ("k_i8_wide", uneven(2, 513, 500, (0, 255, 256, 511, 512)), 9, 130, 84),
    ("k_i8_wide", uneven(3, 1100, 400, range(200, 500)) + [70000], 0, 250, 32),
    ("k_i8_wide", [0] * 700 + [150000], 0, 260, 36),
    ("k_i8_mid<2, 2", uneven(4, 300, 60, (63, 64, 255, 256)), 5, 300, 80),
    ("k_i8_mid<2, 2", [0] * 257 + [9000] + [0] * 200 + [1, 2, 3], 0, 400, 84),
    ("k_i8_mid<2, 2", uneven(5, 1000, 250, range(0, 600)), 0, 130, 48),
    ("k_i8_odd<2, 2", uneven(6, 300, 100, (63, 64, 255, 256)), 5, 300, 81),
    ("k_i8_odd<2, 2", [0] * 257 + [19000] + [0] * 200 + [1, 2, 3], 0, 400, 67),
    ("k_i8_tile", uneven(7, 300, 100, (63, 64, 255, 256)), 5, 130, 15),
    ("k_i8_rows<2, 2", uneven(8, 300, 60, (63, 64, 255, 256)), 5, 130, 81),
    ("k_i8_rows<1, 1", uneven(9, 600, 16, range(100, 300)), 5, 130, 80),
]


def many_types(case):
    return TYPES[case % 4]


@pytest.mark.parametrize("case", range(len(ONE)))
@pytest.mark.parametrize("s,y", TYPES)
def test_kernel_of_one_matrix(sm, case, s, y):
    kernel, N, M, K = ONE[case]
    say(kernel, N, M, K, s, y)
    g = gen(case)
    w, x, ws, xs = codes(g, M, K), codes(g, N, K), scales(g, M, kind=s), scales(g, N)
    same(sm.i8_gemv({"weight": w, "scales": ws}, x, xs, M, K, y_dtype=dt(y)), product(x, xs, w, ws, y))


@pytest.mark.parametrize("case", range(len(MANY)))
def test_kernel_of_many_experts(sm, case):
    import torch
    kernel, counts, behind, M, K = MANY[case]
    s, y = many_types(case)
    E, N = len(counts), sum(counts) + behind
    say(kernel, E, N, M, K, s, y)
    g = gen(case)
    w, x, ws, xs = codes(g, E, M, K), codes(g, N, K), scales(g, E, M, kind=s), scales(g, N)
    out = torch.full((N, M), 3.0, device="cuda", dtype=dt(y))
    sm.i8_gemv({"weight": w, "scales": ws}, x, xs, M, K, y=out, offsets=sizes_to_offsets(counts))
    want = torch.full_like(out, 3.0)
    at = 0
    for e, n in enumerate(counts):
        if n:
            want[at:at + n] = product(x[at:at + n], xs[at:at + n], w[e], ws[e], y)
        at += n
    same(out, want)
