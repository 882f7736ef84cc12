"""GPU tests of the dense operators at the limits of what their calls accept: the longest
rows, values at the ends of the types' ranges, and what the Python entries refuse.
Tolerances are those of test_gpu_dense."""
import math

import pytest

from test_gpu_dense import block_case, check_route, gen, norm_tol, say, sm  # noqa: F401

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
