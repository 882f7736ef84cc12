"""Cases of the operators of routed experts in 8-bit integers, for measuring.

Operators of `pseudo_random_weight_amd.seedmm`:

* `i8_gemv`    -- y = x W^T of 8-bit integers with a scale a token and a channel, one matrix
  or a matrix an expert for rows sorted by expert;
* `moe_sort`   -- the tokens of a routed batch as rows in the order of their experts;
* `moe_unsort` -- the rows back, weighted and summed for each token, and `moe_unsort_grad`,
  the gradients of the rows and of the weights;
* `swiglu`     -- silu(gate) * up of a product's rows, in bf16 or fp32, or in 8 bits with a
  scale a row for the next product.

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


def _product(name, N, M, K, y, s="f32"):
    return {"name": name, "op": "product", "N": N, "M": M, "K": K, "y": y, "s": s}


def _grouped(name, T, k, E, M, K, y, dropped=0.0, s="f32"):
    return {"name": name, "op": "grouped", "T": T, "k": k, "E": E, "M": M, "K": K, "y": y, "s": s,
            "dropped": dropped}


def _sort(name, T, k, E, H, x, dropped):
    return {"name": name, "op": "sort", "T": T, "k": k, "E": E, "H": H, "x": x, "dropped": dropped}


def _unsort(name, T, k, E, H, rows, y, weighted, dropped):
    return {"name": name, "op": "unsort", "T": T, "k": k, "E": E, "H": H, "rows": rows, "y": y,
            "weighted": weighted, "dropped": dropped}


def _grad(name, T, k, E, H, rows, dy, dropped):
    return {"name": name, "op": "grad", "T": T, "k": k, "E": E, "H": H, "rows": rows, "dy": dy,
            "dropped": dropped}


def _swiglu(name, N, I, x, out, live):
    return {"name": name, "op": "swiglu", "N": N, "I": I, "x": x, "out": out, "live": live}


def listed():
    return [
        # the output head over a large vocabulary at one token: the longest weight stream
        _product("head, one token", 1, 131072, 2048, "f32", "bf16"),
        # a decode batch of odd sizes: ragged row and token tiles, rows that start on 2 bytes
        _product("decode 61, odd", 61, 5125, 4150, "bf16"),
        # a prompt through a wide projection: matrix-core work
        _product("prompt 4096", 4096, 8192, 2048, "bf16"),
        # gate and up of the 100-expert top-8 layer (2048 -> 1024) at one token: 8 experts, a row each
        _grouped("experts, one token", 1, 8, 100, 2048, 2048, "bf16"),
        # the same for a prompt: some 330 rows an expert
        _grouped("experts, prompt 4096", 4096, 8, 100, 2048, 2048, "bf16"),
        # one token of that layer in its experts' order: pure latency
        _sort("sort, one token", 1, 8, 100, 2048, "bf16", 0.0),
        # the prompt, with some slots dropped (experts of another device, padding tokens)
        _sort("sort, prompt 4096", 4096, 8, 100, 2048, "bf16", 0.1),
        # a decode batch back
        _unsort("unsort, 64 tokens", 64, 8, 100, 2048, "bf16", "f32", True, 0.0),
        # the prompt back
        _unsort("unsort, prompt 4096", 4096, 8, 100, 2048, "bf16", "f32", True, 0.1),
        # its gradients, an odd width (no row starts on 16 bytes), fp32 rows
        _grad("gradient, 1021 odd", 1021, 6, 64, 7167, "f32", "bf16", 0.0),
        # between the products of a 64-token decode step, in 8 bits for the second one
        _swiglu("swiglu, 512 rows, 8 bits", 512, 1024, "bf16", "i8", 1.0),
        # the same for the prompt's rows, kept in bf16, those of dropped slots left out
        _swiglu("swiglu, 32768 rows", 32768, 1024, "bf16", "bf16", 0.9),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))


def _width(rng, lo, hi):
    n = _log_int(rng, lo, hi)
    return rng.choice([n, max(lo, n // 8 * 8), max(lo, n // 64 * 64)])


def draw(rng):
    op = rng.choice(["product", "product", "grouped", "grouped", "sort", "unsort", "grad", "swiglu"])
    if op == "product":
        N = rng.choice([1, _log_int(rng, 1, 4096)])
        K = _width(rng, 128, 16384)
        M = _log_int(rng, 16, min(131072, 131072 * 2048 // K, 4096 * 8192 // N, 4096 * 8192 * 2048 // (N * K)))
        return {"op": op, "N": N, "M": M, "K": K, "y": rng.choice(["f32", "bf16"]),
                "s": rng.choice(["f32", "bf16"])}
    if op == "swiglu":
        N = rng.choice([1, _log_int(rng, 1, 65536)])
        I = _width(rng, 64, min(16384, 32768 * 1024 // N))
        return {"op": op, "N": N, "I": I, "x": rng.choice(["bf16", "f32"]),
                "out": rng.choice(["bf16", "i8", "f32"]), "live": rng.choice([1.0, 0.8])}
    E = _log_int(rng, 8, 128 if op == "grouped" else 512)
    k = rng.randint(1, min(8 if op == "grouped" else 16, E))
    dropped = rng.choice([0.0, 0.3])
    if op == "grouped":
        K = _width(rng, 64, 4096)
        M = _log_int(rng, 64, min(4096, 100 * 2048 * 2048 // (E * K)))
        T = rng.choice([1, _log_int(rng, 1, min(4096, 32768 * 2048 * 2048 // (k * M * K)))])
        return {"op": op, "T": T, "k": k, "E": E, "M": M, "K": K, "y": rng.choice(["f32", "bf16"]),
                "s": rng.choice(["f32", "bf16"]), "dropped": dropped}
    T = rng.choice([1, _log_int(rng, 1, 16384)])
    H = _width(rng, 64, min(8192, 4096 * 8 * 2048 // (T * k)))
    case = {"op": op, "T": T, "k": k, "E": E, "H": H, "dropped": dropped}
    if op == "sort":
        return {**case, "x": rng.choice(["bf16", "f32", "i8"])}
    if op == "unsort":
        return {**case, "rows": rng.choice(["bf16", "f32"]), "y": rng.choice(["f32", "bf16"]),
                "weighted": rng.random() < 0.7}
    return {**case, "rows": rng.choice(["bf16", "f32"]), "dy": rng.choice(["f32", "bf16"])}


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _codes(v):
    """Rows in 8 bits and their scales."""
    s = v.abs().amax(dim=-1) / 127
    return torch.round(v / s[..., None]).clamp(-127, 127).to(torch.int8), s


def _routing(case, g):
    """ids [T][k] of a router that likes some experts better, -1 in dropped slots."""
    T, k, E = case["T"], case["k"], case["E"]
    ids = torch.topk(_normal(g, T, E) + 0.5 * _normal(g, E), k, dim=1).indices.to(torch.int32)
    if case["dropped"]:
        ids[torch.rand(T, k, generator=g, device="cuda") < case["dropped"]] = -1
    return ids


def _places(ids, E):
    """The sorted order of the pairs: place of each (or -1), and the experts' offsets."""
    flat = ids.flatten().cpu().numpy().astype(np.int64)
    counts = np.bincount(flat[flat >= 0], minlength=E)
    offsets = np.concatenate([[0], np.cumsum(counts)])
    live = np.nonzero(flat >= 0)[0]
    place = np.full(flat.size, -1)
    place[live[np.argsort(flat[live], kind="stable")]] = np.arange(live.size)
    dev = ids.device
    return (torch.from_numpy(place.astype(np.int32)).to(dev).view(ids.shape),
            torch.from_numpy(offsets.astype(np.int32)).to(dev))


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    st = dict(case)
    op = case["op"]
    if op in ("product", "grouped"):
        M, K = case["M"], case["K"]
        E = case["E"] if op == "grouped" else 1
        N = case["T"] * case["k"] if op == "grouped" else case["N"]
        w = torch.empty(E, M, K, dtype=torch.int8, device="cuda")
        s = torch.empty(E, M, device="cuda")
        for e in range(E):
            w[e], s[e] = _codes(0.02 * _normal(g, M, K))
        st["mat"] = {"weight": w, "scales": s.to(DTYPES[case["s"]])}
        # normed activations: unit rows, channels of unequal size
        st["x"], st["x_scale"] = _codes(_normal(g, N, K) * torch.exp(0.5 * _normal(g, K)))
        st["offsets"] = _places(_routing(case, g), E)[1] if op == "grouped" else None
        st["y_rows"] = torch.zeros(N, M, dtype=DTYPES[case["y"]], device="cuda")
        return st
    if op == "swiglu":
        N, I = case["N"], case["I"]
        st["gate_up"] = (1.5 * _normal(g, N, 2 * I)).to(DTYPES[case["x"]])
        live = N if case["live"] == 1.0 else int(round(N * case["live"]))
        st["count"] = None if live == N else torch.tensor([live], dtype=torch.int32, device="cuda")
        st["o"] = torch.zeros(N, I, dtype=DTYPES[case["out"]], device="cuda")
        st["sc"] = torch.zeros(N, device="cuda") if case["out"] == "i8" else None
        st["values"] = torch.empty(N, I, dtype=torch.bfloat16, device="cuda") if case["out"] == "i8" else None
        return st
    T, k, E, H = case["T"], case["k"], case["E"], case["H"]
    ids = _routing(case, g)
    if op == "sort":
        st["ids"] = ids
        x = _normal(g, T, H) * torch.exp(0.5 * _normal(g, H))
        st["x_scale"] = None
        if case["x"] == "i8":
            st["x_rows"], st["x_scale"] = _codes(x)
            st["values"] = torch.empty(T * k, H, dtype=torch.bfloat16, device="cuda")
        else:
            st["x_rows"] = x.to(DTYPES[case["x"]])
        st["rows_out"] = torch.zeros(T * k, H, dtype=DTYPES[case["x"]], device="cuda")
        st["scale_out"] = torch.zeros(T * k, device="cuda") if case["x"] == "i8" else None
        st["off"] = torch.empty(E + 1, dtype=torch.int32, device="cuda")
        st["inv"] = torch.empty(T, k, dtype=torch.int32, device="cuda")
        return st
    st["inv"] = _places(ids, E)[0]
    st["y_rows"] = _normal(g, T * k, H).to(DTYPES[case["rows"]])
    st["w"] = torch.softmax(_normal(g, T, k), dim=1)
    if op == "unsort":
        if not case["weighted"]:      # the gradient of moe_sort: the slots' rows are added
            st["w"] = None
        st["y_out"] = torch.empty(T, H, dtype=DTYPES[case["y"]], device="cuda")
        return st
    st["dy_rows"] = _normal(g, T, H).to(DTYPES[case["dy"]])
    st["drows"] = torch.zeros(T * k, H, dtype=DTYPES[case["rows"]], device="cuda")
    st["dw"] = torch.empty(T, k, device="cuda")
    return st


def _plain_product(st):
    w, s = st["mat"]["weight"][0], st["mat"]["scales"][0].float()
    y = (st["x"].float() @ w.float().t()) * st["x_scale"][:, None] * s
    return {"y": y.to(st["y_rows"].dtype)}


def _plain_grouped(st):
    # an expert after the other: one batched product over experts padded to the longest takes
    # twice as long for a prompt
    off = st["offsets"].tolist()
    w, s = st["mat"]["weight"], st["mat"]["scales"].float()
    y = st["y_rows"].clone()
    for e, (a, b) in enumerate(zip(off, off[1:])):
        if a < b:
            v = (st["x"][a:b].float() @ w[e].float().t()) * st["x_scale"][a:b, None] * s[e]
            y[a:b] = v.to(y.dtype)
    return {"y": y}


def _plain_sort(st):
    E, k = st["E"], st["k"]
    flat = st["ids"].flatten().long()
    key = torch.where((flat >= 0) & (flat < E), flat, torch.full_like(flat, E))
    by, order = torch.sort(key, stable=True)
    off = torch.searchsorted(by, torch.arange(E + 1, device="cuda"))
    place = torch.empty_like(order)
    place[order] = torch.arange(order.numel(), device="cuda")
    kept = by < E
    rows = st["x_rows"][order // k]
    got = {"offsets": off.to(torch.int32),
           "inverse": torch.where(key < E, place, torch.full_like(place, -1)).to(torch.int32).view(-1, k)}
    if st["x_scale"] is not None:
        sc = torch.where(kept, st["x_scale"][order // k], st["scale_out"])
        got["scale"] = sc
        rows = torch.where(kept[:, None], rows, st["rows_out"])
        got["rows"] = (rows.float() * sc[:, None]).to(torch.bfloat16)
    else:
        got["rows"] = torch.where(kept[:, None], rows, st["rows_out"])
    return got


def _plain_unsort(st):
    inv = st["inv"].long()
    rows = st["y_rows"][inv.clamp(min=0)].float()
    if st["w"] is not None:
        rows = rows * st["w"][:, :, None]
    rows = torch.where((inv >= 0)[:, :, None], rows, torch.zeros((), device="cuda"))
    return {"y": rows.sum(dim=1).to(st["y_out"].dtype)}


def _plain_grad(st):
    inv, dy = st["inv"].long(), st["dy_rows"].float()
    kept = inv >= 0
    rows = st["y_rows"][inv.clamp(min=0)].float()
    dw = torch.where(kept, (rows * dy[:, None, :]).sum(dim=2), torch.zeros((), device="cuda"))
    drows = st["drows"].clone()
    drows[inv[kept]] = (st["w"][:, :, None] * dy[:, None, :])[kept].to(drows.dtype)
    return {"drows": drows, "dw": dw}


def _plain_swiglu(st):
    # an 8-bit code next to a rounding border needs the 64 bits
    f = torch.float64 if st["sc"] is not None else torch.float32
    g, u = st["gate_up"].to(f).chunk(2, dim=1)
    h = g / (1 + torch.exp(-g)) * u
    got = {}
    if st["sc"] is not None:
        sc = torch.clamp(h.abs().amax(dim=1, keepdim=True) / 127, min=2.0 ** -126)
        got["out"] = (torch.round(h / sc) * sc).to(torch.bfloat16)
        got["scale"] = sc[:, 0].to(torch.float32)
    else:
        got["out"] = h.to(st["o"].dtype)
    if st["count"] is not None:
        kept = torch.arange(st["N"], device="cuda") < st["count"]
        got["out"] = torch.where(kept[:, None], got["out"], torch.zeros((), dtype=got["out"].dtype, device="cuda"))
        if st["sc"] is not None:
            got["scale"] = torch.where(kept, got["scale"], st["sc"])
    return got


def run(st):
    op = st["op"]
    if not own:
        return {"product": _plain_product, "grouped": _plain_grouped, "sort": _plain_sort,
                "unsort": _plain_unsort, "grad": _plain_grad, "swiglu": _plain_swiglu}[op](st)
    lib = _lib()
    if op in ("product", "grouped"):
        return {"y": lib.i8_gemv(st["mat"], st["x"], st["x_scale"], st["M"], st["K"], y=st["y_rows"],
                                 offsets=st["offsets"])}
    if op == "sort":
        rows, sc, off, inv = lib.moe_sort(st["x_rows"], st["ids"], st["E"], x_scale=st["x_scale"],
                                          rows=st["rows_out"], row_scale=st["scale_out"],
                                          offsets=st["off"], inverse=st["inv"])
        got = {"offsets": off, "inverse": inv, "rows": rows}
        if sc is not None:
            # 8-bit codes go back as the values that they stand for
            got["scale"], got["rows"] = sc, torch.mul(rows, sc[:, None], out=st["values"])
        return got
    if op == "unsort":
        return {"y": lib.moe_unsort(st["y_rows"], st["inv"], st["w"], y=st["y_out"])}
    if op == "grad":
        drows, dw = lib.moe_unsort_grad(st["dy_rows"], st["y_rows"], st["inv"], st["w"],
                                        drows=st["drows"], dw=st["dw"])
        return {"drows": drows, "dw": dw}
    o, sc = lib.swiglu(st["gate_up"], out=st["o"], scale=st["sc"], count=st["count"])
    if sc is None:
        return {"out": o}
    return {"out": torch.mul(o, sc[:, None], out=st["values"]), "scale": sc}


def work(case):
    op = case["op"]
    if op == "product":
        N, M, K = case["N"], case["M"], case["K"]
        b = M * K + M * BYTES[case["s"]] + N * (K + 4) + N * M * BYTES[case["y"]]
        return {"bytes": b, "flops": 2 * N * M * K}
    if op == "swiglu":
        n = int(round(case["N"] * case["live"])) * case["I"]
        return {"bytes": n * (2 * BYTES[case["x"]] + BYTES[case["out"]]), "flops": 6 * n}
    T, k, E = case["T"], case["k"], case["E"]
    live = T * k * (1 - case["dropped"])
    if op == "grouped":
        M, K = case["M"], case["K"]
        used = E * (1 - (1 - k * (1 - case["dropped"]) / E) ** T)      # experts that have rows
        b = used * M * (K + BYTES[case["s"]]) + live * (K + 4 + M * BYTES[case["y"]]) + 4 * E
        return {"bytes": b, "flops": 2 * live * M * K}
    H = case["H"]
    if op == "sort":
        return {"bytes": (T + live) * H * BYTES[case["x"]] + 8 * T * k + 4 * E, "flops": T * k}
    if op == "unsort":
        b = live * H * BYTES[case["rows"]] + T * H * BYTES[case["y"]] + 8 * T * k
        return {"bytes": b, "flops": 2 * live * H}
    b = 2 * live * H * BYTES[case["rows"]] + T * H * BYTES[case["dy"]] + 12 * T * k
    return {"bytes": b, "flops": 3 * live * H}


def exact(case, seed):
    """The operators' definitions in 64 bits."""
    st = prepare(case, seed)
    op = case["op"]
    if op in ("product", "grouped"):
        E = case.get("E", 1)
        N, M = st["x"].shape[0], case["M"]
        off = [0, N] if op == "product" else st["offsets"].tolist()
        y = torch.zeros(N, M, dtype=torch.float64, device="cuda")
        for e in range(E):
            a, b = off[e], off[e + 1]
            if a == b:
                continue
            x = st["x"][a:b].double() * st["x_scale"][a:b].double()[:, None]
            for m0 in range(0, M, 16384):          # rows of W at a time, to bound the memory
                w = st["mat"]["weight"][e, m0:m0 + 16384].double()
                w = w * st["mat"]["scales"][e, m0:m0 + 16384].double()[:, None]
                y[a:b, m0:m0 + 16384] = torch.mm(x, w.t().contiguous())
        return {"y": y}
    if op == "swiglu":
        N, I = case["N"], case["I"]
        n = N if st["count"] is None else int(st["count"])
        v = st["gate_up"][:n].double()
        h = v[:, :I] * torch.sigmoid(v[:, :I]) * v[:, I:]
        out = torch.zeros(N, I, dtype=torch.float64, device="cuda")
        if case["out"] != "i8":
            out[:n] = h
            return {"out": out}
        sc = torch.zeros(N, dtype=torch.float64, device="cuda")
        sc[:n] = torch.clamp(torch.maximum(h.max(dim=1).values, -h.min(dim=1).values) / 127, min=2.0 ** -126)
        out[:n] = torch.round(h / sc[:n, None]) * sc[:n, None]
        return {"out": out, "scale": sc}
    T, k, E, H = case["T"], case["k"], case["E"], case["H"]
    if op == "sort":
        inv, off = _places(st["ids"], E)
        x = st["x_rows"].double()
        if st["x_scale"] is not None:
            x = x * st["x_scale"].double()[:, None]
        rows = torch.zeros(T * k, H, dtype=torch.float64, device="cuda")
        sc = torch.zeros(T * k, dtype=torch.float64, device="cuda")
        for s in range(k):
            kept = inv[:, s] >= 0
            rows[inv[:, s][kept].long()] = x[kept]
            if st["x_scale"] is not None:
                sc[inv[:, s][kept].long()] = st["x_scale"].double()[kept]
        got = {"offsets": off, "inverse": inv, "rows": rows}
        if st["x_scale"] is not None:
            got["scale"] = sc
        return got
    inv = st["inv"]
    if op == "unsort":
        y = torch.zeros(T, H, dtype=torch.float64, device="cuda")
        for s in range(k):
            kept = inv[:, s] >= 0
            r = st["y_rows"][inv[:, s][kept].long()].double()
            y[kept] += r if st["w"] is None else r * st["w"][kept, s].double()[:, None]
        return {"y": y}
    dy = st["dy_rows"].double()
    drows = torch.zeros(T * k, H, dtype=torch.float64, device="cuda")
    dw = torch.zeros(T, k, dtype=torch.float64, device="cuda")
    for s in range(k):
        kept = inv[:, s] >= 0
        at = inv[:, s][kept].long()
        drows[at] = dy[kept] * st["w"][kept, s].double()[:, None]
        dw[kept, s] = torch.linalg.vecdot(st["y_rows"][at].double(), dy[kept])
    return {"drows": drows, "dw": dw}
