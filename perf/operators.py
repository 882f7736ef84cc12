"""Cases of the dense operators that stand around a seed-coded routed layer, for measuring.

Three operators of `pseudo_random_weight_amd.seedmm`:

* `q4_gemv`  -- y = x W^T with W in 4-bit codes and a scale and a bias a group of columns
  (the projections, the router and the head that a seed pack keeps in affine 4 bits);
* `add_norm` -- the residual's addition and the root-mean-square norm of the sum, in the
  output's type or in 8 bits with a scale a row;
* `route`    -- the router's choice: the top_k experts of each token and their weights.

`run` computes a case with elementary torch operations, or with `own` through the library.
`exact` computes it in 64 bits from the definition.
"""
import math

import numpy as np
import torch

own = False
_seedmm = None


def _lib():
    global _seedmm
    if _seedmm is None:
        from pseudo_random_weight_amd import seedmm
        _seedmm = seedmm
    return _seedmm


DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "i8": torch.int8}
BYTES = {"f32": 4, "bf16": 2, "i8": 1}


def _q4(name, N, M, K, group, x, y, s="bf16"):
    return {"name": name, "op": "q4", "N": N, "M": M, "K": K, "group": group, "x": x, "y": y, "s": s}


def _norm(name, N, H, x, delta, out):
    return {"name": name, "op": "norm", "N": N, "H": H, "x": x, "delta": delta, "out": out}


def _route(name, T, E, k, score, logits, masked):
    return {"name": name, "op": "route", "T": T, "E": E, "k": k, "score": score, "logits": logits,
            "masked": masked}


def listed():
    return [
        # the router of a 100-expert layer of hidden size 2048 at one token: pure latency
        _q4("q4 router, one token", 1, 100, 2048, 64, "bf16", "f32"),
        # a square projection at one token, fp32 activations and scales, small groups
        _q4("q4 square, one token, fp32", 1, 2048, 2048, 32, "f32", "f32", "f32"),
        # the output head over a large vocabulary at one token: the longest weight stream
        _q4("q4 head, one token", 1, 131072, 2048, 64, "bf16", "f32"),
        # a decode batch on activations in 8 bits
        _q4("q4 decode 16, 8 bits", 16, 8192, 2048, 64, "i8", "bf16"),
        # a decode batch of odd sizes: ragged row tiles, ragged token tiles, 65 groups a row
        _q4("q4 decode 61, odd", 61, 5125, 4160, 64, "bf16", "bf16"),
        # a prompt through a wide projection: matrix-core work
        _q4("q4 prompt 4096", 4096, 8192, 2048, 64, "bf16", "bf16"),
        # the norm before the routed layer at one token (its previous output is fp32)
        _norm("norm, one token", 1, 2048, "bf16", "f32", "bf16"),
        # the norm of a prompt, in 8 bits for the products
        _norm("norm 4096, 8 bits", 4096, 2048, "bf16", "f32", "i8"),
        # an odd width (no row starts on 16 bytes), fp32 residual stream
        _norm("norm 1021, odd", 1021, 7167, "f32", "bf16", "f32"),
        # the router's choice in the 100-expert top-8 layer, one token
        _route("route, one token", 1, 100, 8, "softmax", "f32", 0.0),
        # the same for a prompt
        _route("route 4096", 4096, 100, 8, "softmax", "f32", 0.0),
        # a wide sigmoid router with a selection bias, bf16 logits (many ties), some masked
        _route("route 16384, sigmoid", 16384, 512, 10, "sigmoid", "bf16", 0.1),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["q4", "q4", "norm", "route"])
    if op == "q4":
        group = rng.choice([32, 64, 64, 128])
        x = rng.choice(["bf16", "bf16", "i8", "f32"])
        N = rng.choice([1, _log_int(rng, 1, 4096)])
        K = group * max(1, _log_int(rng, 128, 16384) // group)
        most = min(131072, (131072 * 2048) // K, (4096 * 8192) // N,
                   (4096 * 8192 * 2048) // (N * K * (3 if x == "f32" else 1)))
        M = _log_int(rng, 16, max(17, most))
        return {"op": "q4", "N": N, "M": M, "K": K, "group": group, "x": x,
                "y": rng.choice(["f32", "bf16"]), "s": rng.choice(["bf16", "bf16", "f32"])}
    if op == "norm":
        N = rng.choice([1, _log_int(rng, 1, 8192)])
        H = _log_int(rng, 64, min(16384, (8192 * 2048) // N))
        H = rng.choice([H, max(64, H // 64 * 64)])
        return {"op": "norm", "N": N, "H": H, "x": rng.choice(["bf16", "f32"]),
                "delta": rng.choice(["none", "bf16", "f32"]),
                "out": rng.choice(["bf16", "i8", "f32"])}
    T = rng.choice([1, _log_int(rng, 1, 16384)])
    E = _log_int(rng, 8, 512)
    return {"op": "route", "T": T, "E": E, "k": rng.randint(1, min(16, E)),
            "score": rng.choice(["softmax", "sigmoid"]), "logits": rng.choice(["f32", "bf16"]),
            "masked": rng.choice([0.0, 0.3])}


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    st = dict(case)
    if case["op"] == "q4":
        N, M, K, G = case["N"], case["M"], case["K"], case["K"] // case["group"]
        # codes of rounded normal weights: scale = range / 15, bias = the lower edge
        w = torch.randint(-2 ** 31, 2 ** 31, (M, K // 8), generator=g, device="cuda",
                          dtype=torch.int64).to(torch.int32)
        s = 0.004 * (0.5 + torch.rand(M, G, generator=g, device="cuda"))
        b = -s * (6.5 + 2 * torch.rand(M, G, generator=g, device="cuda"))
        sd = DTYPES[case["s"]]
        st["mat"] = {"weight": w.view(torch.uint32), "scales": s.to(sd), "biases": b.to(sd)}
        # normed activations: unit rows, channels of unequal size
        x = _normal(g, N, K) * torch.exp(0.5 * _normal(g, K))
        st["x_scale"] = None
        if case["x"] == "i8":
            sc = x.abs().amax(dim=1) / 127
            st["x_scale"] = sc
            st["x_rows"] = torch.round(x / sc[:, None]).clamp(-127, 127).to(torch.int8)
        else:
            st["x_rows"] = x.to(DTYPES[case["x"]])
        st["out"] = torch.empty(N, M, dtype=DTYPES[case["y"]], device="cuda")
        return st
    if case["op"] == "norm":
        N, H = case["N"], case["H"]
        gain = torch.exp(0.7 * _normal(g, H))
        st["x_rows"] = (3 * _normal(g, N, H) * gain).to(DTYPES[case["x"]])
        st["d"] = None if case["delta"] == "none" else _normal(g, N, H).to(DTYPES[case["delta"]])
        st["w"] = (1 + 0.2 * _normal(g, H)).to(torch.bfloat16)
        st["eps"] = 1e-6
        st["o"] = torch.empty(N, H, dtype=DTYPES[case["out"]], device="cuda")
        st["sc"] = torch.empty(N, device="cuda") if case["out"] == "i8" else None
        st["r"] = torch.empty(N, H, dtype=DTYPES[case["x"]], device="cuda") if st["d"] is not None else None
        st["values"] = torch.empty(N, H, dtype=torch.bfloat16, device="cuda") if case["out"] == "i8" else None
        return st
    T, E, k = case["T"], case["E"], case["k"]
    lg = _normal(g, T, E)
    if case["masked"]:
        lg = torch.where(torch.rand(T, E, generator=g, device="cuda") < case["masked"],
                         torch.full_like(lg, -math.inf), lg)
    st["lg"] = lg.to(DTYPES[case["logits"]])
    st["bias"] = 0.1 * _normal(g, E) if case["score"] == "sigmoid" else None
    st["ids"] = torch.empty(T, k, dtype=torch.int32, device="cuda")
    st["wt"] = torch.empty(T, k, device="cuda")
    return st


def _plain_q4(st):
    m, group = st["mat"], st["group"]
    M, K = st["M"], st["K"]
    shifts = torch.arange(0, 32, 4, device="cuda", dtype=torch.int32)
    q = (m["weight"].view(torch.int32)[:, :, None] >> shifts) & 15
    w = q.view(M, K // group, group).to(torch.float32) * m["scales"].float()[:, :, None] \
        + m["biases"].float()[:, :, None]
    y = st["x_rows"].float() @ w.view(M, K).t()
    if st["x_scale"] is not None:
        y = y * st["x_scale"][:, None]
    return {"y": y.to(st["out"].dtype)}


def _plain_norm(st):
    # an 8-bit code next to a rounding border needs the 64 bits
    f = torch.float64 if st["sc"] is not None else torch.float32
    r = st["x_rows"].to(f)
    if st["d"] is not None:
        r = r + st["d"].to(f)
    v = r * st["w"].to(f) * torch.rsqrt((r * r).mean(dim=1, keepdim=True) + st["eps"])
    got = {}
    if st["sc"] is not None:
        sc = torch.clamp(v.abs().amax(dim=1, keepdim=True) / 127, min=2.0 ** -126)
        got["out"] = (torch.round(v / sc) * sc).to(torch.bfloat16)
        got["scale"] = sc[:, 0].to(torch.float32)
    else:
        got["out"] = v.to(st["o"].dtype)
    if st["d"] is not None:
        got["residual"] = r.to(st["x_rows"].dtype)
    return got


def _plain_route(st):
    lg, k = st["lg"].float(), st["k"]
    if st["score"] == "sigmoid":
        # scores next to each other need the 64 bits to be ordered
        p = 1 / (1 + torch.exp(-lg.double()))
        key = torch.where(lg == -math.inf, torch.full_like(p, -math.inf), p + st["bias"].double())
    else:
        key = lg
    order = torch.sort(key, dim=1, descending=True, stable=True).indices[:, :k]
    if st["score"] == "sigmoid":
        w = p.gather(1, order).float()
    else:
        sel = lg.gather(1, order)
        w = torch.exp(sel - sel[:, :1])
    w = torch.where(lg.gather(1, order) == -math.inf, torch.zeros_like(w), w)
    total = w.sum(dim=1, keepdim=True)
    w = torch.where(total > 0, w / total, torch.zeros_like(w))
    return {"ids": order.to(torch.int32), "w": w}


def run(st):
    if st["op"] == "q4":
        if own:
            return {"y": _lib().q4_gemv(st["mat"], st["x_rows"], st["M"], st["K"], st["group"],
                                        x_scale=st["x_scale"], y=st["out"])}
        return _plain_q4(st)
    if st["op"] == "norm":
        if own:
            o, sc, r = _lib().add_norm(st["x_rows"], st["w"], delta=st["d"], eps=st["eps"],
                                       out=st["o"], scale=st["sc"], residual=st["r"])
            # 8-bit codes go back as the values that they stand for
            got = {"out": o if sc is None else torch.mul(o, sc[:, None], out=st["values"])}
            if sc is not None:
                got["scale"] = sc
            if st["d"] is not None:
                got["residual"] = r
            return got
        return _plain_norm(st)
    if own:
        ids, w = _lib().route(st["lg"], st["k"], bias=st["bias"], score=st["score"], ids=st["ids"],
                              w=st["wt"])
        return {"ids": ids, "w": w}
    return _plain_route(st)


def work(case):
    if case["op"] == "q4":
        N, M, K = case["N"], case["M"], case["K"]
        b = M * K / 2 + 2 * M * (K // case["group"]) * BYTES[case["s"]]
        b += N * K * BYTES[case["x"]] + N * M * BYTES[case["y"]]
        return {"bytes": b, "flops": 2 * N * M * K}
    if case["op"] == "norm":
        N, H = case["N"], case["H"]
        b = BYTES[case["x"]] + BYTES[case["out"]]
        if case["delta"] != "none":
            b += BYTES[case["delta"]] + BYTES[case["x"]]
        return {"bytes": N * H * b + 2 * H, "flops": 6 * N * H}
    T, E, k = case["T"], case["E"], case["k"]
    return {"bytes": T * E * BYTES[case["logits"]] + 8 * T * k, "flops": 4 * T * E}


def exact(case, seed):
    """The operators' definitions in 64 bits."""
    st = prepare(case, seed)
    if case["op"] == "q4":
        group, M, K = case["group"], case["M"], case["K"]
        x = st["x_rows"].double()
        if st["x_scale"] is not None:
            x = x * st["x_scale"].double()[:, None]
        words = st["mat"]["weight"].view(torch.int32).to(torch.int64)
        y = torch.zeros(case["N"], M, dtype=torch.float64, device="cuda")
        step = max(1, (1 << 26) // K)
        for m0 in range(0, M, step):           # rows of W at a time, to bound the memory
            rows = words[m0:m0 + step]
            w = torch.empty(rows.shape[0], K, dtype=torch.float64, device="cuda")
            for i in range(8):
                w[:, i::8] = (torch.div(rows, 16 ** i, rounding_mode="floor") % 16).double()
            sc = st["mat"]["scales"][m0:m0 + step].double().repeat_interleave(group, dim=1)
            bi = st["mat"]["biases"][m0:m0 + step].double().repeat_interleave(group, dim=1)
            y[:, m0:m0 + step] = torch.mm(x, (w * sc + bi).t().contiguous())
        return {"y": y}
    if case["op"] == "norm":
        r = st["x_rows"].double()
        if st["d"] is not None:
            r = r + st["d"].double()
        rms = torch.sqrt(torch.linalg.vector_norm(r, dim=1) ** 2 / case["H"] + st["eps"])
        v = r / rms[:, None] * st["w"].double()
        got = {"out": v}
        if case["out"] == "i8":
            top = torch.maximum(v.max(dim=1).values, -v.min(dim=1).values)
            sc = torch.clamp(top / 127, min=2.0 ** -126)
            got = {"out": torch.round(v / sc[:, None]) * sc[:, None], "scale": sc}
        if st["d"] is not None:
            got["residual"] = r
        return got
    lg = st["lg"].double().cpu().numpy()
    key = lg
    if case["score"] == "sigmoid":
        with np.errstate(over="ignore"):
            p = np.exp(-np.logaddexp(0.0, -lg))
        key = np.where(np.isneginf(lg), -np.inf, p + st["bias"].double().cpu().numpy())
    order = np.argsort(-key, axis=1, kind="stable")[:, :case["k"]]
    sel = np.take_along_axis(lg, order, axis=1)
    if case["score"] == "sigmoid":
        w = np.where(np.isneginf(sel), 0.0, np.take_along_axis(p, order, axis=1))
    else:
        top = np.where(np.isneginf(sel[:, :1]), 0.0, sel[:, :1])
        w = np.where(np.isneginf(sel), 0.0, np.exp(sel - top))
    total = w.sum(axis=1, keepdims=True)
    w = np.divide(w, total, out=np.zeros_like(w), where=total > 0)
    return {"ids": order.astype(np.int32), "w": w}
