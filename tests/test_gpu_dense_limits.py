"""GPU tests of the dense operators at the limits of what their calls accept: the longest
rows, values at the ends of the types' ranges, and what the Python entries refuse.
Tolerances are those of test_gpu_dense."""
import math

import pytest

from test_gpu_dense import block_case, norm_tol, say, sm  # noqa: F401

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
