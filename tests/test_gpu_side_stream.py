"""GPU test of layer calls with a second stream (SideStream) on every stream that torch hands out:
its pool holds 32, dealt in turn, so that a program's own stream can be the second stream's."""
import sys

import numpy as np
import pytest

import synth

pytestmark = pytest.mark.gpu


def say(*a):
    print("[case]", *a, file=sys.stderr, flush=True)


def _dev(mat):
    import torch
    return {
        "seeds": torch.from_numpy(mat["seeds"].view(np.int16).copy()).view(torch.uint16).cuda(),
        "coefs": torch.from_numpy(mat["coefs"].view(np.int16).copy()).view(torch.uint16).cuda(),
        "codes": torch.from_numpy(mat["codes"].copy()).cuda(),
        "exp_bias": torch.from_numpy(mat["exp_bias"].copy()).cuda(),
    }


def test_layers_with_a_second_stream_on_any_stream():
    """One second stream for each place of the pool, with a call on one stream of the pool: eager, on the
    stream as the call's, and captured there.  Each gives the bits of a call without it."""
    import torch
    from pseudo_random_weight_amd import seedmm as sm
    E, H, I, P, k, T = 8, 256, 128, 4, 2, 16
    base = synth.config_seed(52)
    mats = [_dev(synth.seed_matrix(base, f"side.{n}", *((I, H) if n != "down" else (H, I)), P, E, exp_bias=eb))
            for n, eb in (("gate", -20), ("up", -19), ("down", -18))]
    ids, w = synth.route_topk(base, "side.r", T, E, k)
    x = synth.bf16_bits(synth.normal_f32(base, "side.x", (T, H)))
    ids, w = torch.from_numpy(ids).cuda(), torch.from_numpy(w).cuda()
    x = torch.from_numpy(x.view(np.int16).copy()).view(torch.bfloat16).cuda()
    want = sm.moe(ids, w, x, E, H, I, P, *mats)
    ws = torch.empty(sm.moe_workspace_bytes(T, k, E, H, I), dtype=torch.uint8, device="cuda")
    y = torch.empty_like(want)
    main = torch.cuda.Stream()
    torch.cuda.synchronize()
    handles = set()
    for i in range(40):
        if i == 20:
            torch.cuda.Stream()      # each takes two of the pool: now the others of each pair
        side = sm.SideStream()
        handles.add(side.stream.cuda_stream)
        say("second stream", i, side.stream.cuda_stream == main.cuda_stream)
        graph = torch.cuda.CUDAGraph()
        for how in ("current", "given", "captured"):
            y.fill_(7)
            torch.cuda.synchronize()
            if how == "current":
                with torch.cuda.stream(main):
                    sm.moe(ids, w, x, E, H, I, P, *mats, y=y, workspace=ws, side=side)
            elif how == "given":
                sm.moe(ids, w, x, E, H, I, P, *mats, y=y, workspace=ws, side=side, stream=main)
            else:
                with torch.cuda.graph(graph, stream=main):
                    sm.moe(ids, w, x, E, H, I, P, *mats, y=y, workspace=ws, side=side)
                graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(y, want), (i, how)
    assert main.cuda_stream in handles
