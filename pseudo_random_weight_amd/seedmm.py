"""Thin Python binding of the seedmm C ABI (include/seedmm.h).

Argument marshalling only: tensors are passed to the HIP library as device pointers
plus sizes, on torch's current HIP stream or the one passed in (outputs and scratch the
binding allocates belong to that stream).  Every step of the computation runs in
the library's kernels; there is no Python or CPU fallback, and a missing library
raises at import.

No call records a gradient: a result carries no graph, whatever its inputs require.
Where gradients are offered they are calls of their own (moe_unsort for moe_sort's
rows, moe_unsort_grad for moe_unsort), for a torch.autograd.Function of the caller's;
the products, swiglu and the layers have none.
"""
from __future__ import annotations

import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libseedmm.so")

OK, EINVAL, EALIGN, EWORKSPACE, EHIP, ECAPACITY, ESCRATCH = 0, -1, -2, -3, -4, -5, -6
F32, BF16, I8 = 0, 1, 2
SOFTMAX, SIGMOID = 0, 1
NOALLOC_SCRATCH_BYTES = 8 << 20      # SEEDMM_NOALLOC_SCRATCH_BYTES of include/seedmm.h


class SeedmmError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: {_lib.seedmm_strerror(status).decode()} (status {status})")
        self.status = status


class SeedMat(ctypes.Structure):
    _fields_ = [("seeds", ctypes.c_void_p), ("coefs", ctypes.c_void_p),
                ("codes", ctypes.c_void_p), ("exp_bias", ctypes.c_void_p)]


class SeedBlock(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_void_p) for n in ("norm_weight", "router_weight", "router_scales",
                                                "router_biases", "router_bias", "p4mask")]
                + [(n, SeedMat) for n in ("gate", "up", "down")] + [("eps", ctypes.c_float)]
                + [(n, ctypes.c_int) for n in ("norm_dtype", "router_dtype", "group", "score",
                                               "top_k", "E", "H", "I", "P")])


class I8Mat(ctypes.Structure):
    _fields_ = [("weight", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("s_dtype", ctypes.c_int)]


class SeedSide(ctypes.Structure):
    _fields_ = [("stream", ctypes.c_void_p), ("fork", ctypes.c_void_p),
                ("join", ctypes.c_void_p)]


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"{LIB_PATH} is missing: build it with `python -m pseudo_random_weight_amd.build` "
            "(there is no fallback path)")
    L = ctypes.CDLL(LIB_PATH)
    p, i32 = ctypes.c_void_p, ctypes.c_int
    L.seedmm_gemv.argtypes = [p, p, p, ctypes.c_int32, p, p, i32, i32, i32]
    L.seedmm_gemv_ex.argtypes = [p, p, p, ctypes.c_int32, p, i32, i32, p, i32, i32, i32, i32, i32, p]
    L.seedmm_reconstruct.argtypes = [p, p, p, ctypes.c_int32, p, i32, i32, i32, i32, p]
    L.seedmm_moe_dispatch.argtypes = [p, i32, i32, i32, p, p, p]
    L.seedmm_moe_workspace_bytes.restype = ctypes.c_size_t
    L.seedmm_moe_workspace_bytes.argtypes = [i32, i32, i32, i32, i32]
    L.seedmm_moe.argtypes = [p, p, i32, i32, p, p, i32, i32, i32, i32, SeedMat, SeedMat, SeedMat,
                             p, ctypes.c_size_t, p]
    L.seedmm_moe_timed.argtypes = L.seedmm_moe.argtypes + [p]
    L.seedmm_moe_noalloc.argtypes = [p, p, i32, i32, p, p, i32, i32, i32, i32, SeedMat, SeedMat,
                                     SeedMat, p]
    L.seedmm_moe_ex.argtypes = [p, p, i32, i32, p, p, i32, i32, i32, i32, p, SeedMat, SeedMat,
                                SeedMat, p, ctypes.c_size_t, p, ctypes.POINTER(SeedSide)]
    L.seedmm_search.argtypes = [p, i32, p, i32, i32, i32, ctypes.c_int32, p, p, p, p, p, p]
    L.seedmm_search_table_bytes.restype = ctypes.c_size_t
    L.seedmm_search_table_bytes.argtypes = [i32]
    L.seedmm_search_prepare.argtypes = [i32, p, ctypes.c_size_t, p]
    L.seedmm_moe_mixed.argtypes = [p, p, i32, i32, p, p, i32, i32, i32, p, SeedMat, SeedMat,
                                   SeedMat, p, ctypes.c_size_t, p]
    sz = ctypes.c_size_t
    L.seedmm_cache_state_bytes.restype = sz
    L.seedmm_cache_state_bytes.argtypes = [i32, i32]
    L.seedmm_cache_device_bytes.restype = sz
    L.seedmm_cache_device_bytes.argtypes = [i32, i32, i32, i32, i32]
    L.seedmm_cache_record_layout.restype = sz
    L.seedmm_cache_record_layout.argtypes = [i32, i32, i32, p]
    L.seedmm_cache_init.argtypes = [p, sz, i32, i32, i32, i32, i32, p, p, p, sz]
    L.seedmm_cache_reset.argtypes = [p]
    L.seedmm_cache_plan.argtypes = [p, p, i32, i32, p, p]
    L.seedmm_cache_moe.argtypes = [p, p, p, p, i32, i32, p, p, p, sz, p]
    L.seedmm_cache_stats.argtypes = [p, p]
    i64 = ctypes.c_int64
    L.seedmm_q4_gemv.argtypes = [p, p, p, i32, i32, p, i32, i32, p, p, i32, i32, i32, i32, i32, p,
                                 sz, p]
    L.seedmm_q4_workspace_bytes.restype = sz
    L.seedmm_q4_workspace_bytes.argtypes = [i32, i32, i32, i32, i32]
    L.seedmm_add_norm.argtypes = [p, i32, i64, p, i32, i64, p, i32, ctypes.c_float, p, i64, p, i32,
                                  i64, p, i32, i32, p]
    L.seedmm_route.argtypes = [p, i32, i64, p, i32, i32, i32, i32, p, p, p]
    blk = ctypes.POINTER(SeedBlock)
    L.seedmm_moe_block_workspace_bytes.restype = sz
    L.seedmm_moe_block_workspace_bytes.argtypes = [blk, i32]
    L.seedmm_moe_block.argtypes = [blk, p, i32, p, i32, p, p, p, i32, p, sz, p,
                                   ctypes.POINTER(SeedSide)]
    L.seedmm_i8_gemv.argtypes = [p, p, i32, i32, p, p, i64, p, p, i32, i64, i32, i32, i32, p]
    L.seedmm_moe_sort.argtypes = [p, i32, i32, i32, p, i32, i64, p, p, i64, p, i32, p, p, p, sz, p]
    L.seedmm_moe_sort_workspace_bytes.restype = sz
    L.seedmm_moe_sort_workspace_bytes.argtypes = [i32, i32, i32]
    L.seedmm_moe_unsort.argtypes = [p, i32, i64, i32, p, p, p, i32, i64, i32, i32, i32, p]
    L.seedmm_moe_unsort_grad.argtypes = [p, i32, i64, p, i32, i64, i32, p, p, p, i64, p, i32, i32, i32, p]
    L.seedmm_swiglu.argtypes = [p, i32, i64, p, i32, i64, p, p, i32, i32, p]
    L.seedmm_moe_i8_workspace_bytes.restype = sz
    L.seedmm_moe_i8_workspace_bytes.argtypes = [i32, i32, i32, i32, i32]
    L.seedmm_moe_i8.argtypes = [p, p, i32, i32, p, p, p, i32, i32, i32, I8Mat, I8Mat, p, sz, p]
    L.seedmm_strerror.restype = ctypes.c_char_p
    L.seedmm_strerror.argtypes = [i32]
    L.seedmm_version.restype = i32
    for name in ("seedmm_gemv", "seedmm_gemv_ex", "seedmm_reconstruct", "seedmm_moe_dispatch",
                 "seedmm_moe", "seedmm_moe_timed", "seedmm_moe_ex", "seedmm_moe_noalloc",
                 "seedmm_search",
                 "seedmm_search_prepare", "seedmm_moe_mixed",
                 "seedmm_cache_init", "seedmm_cache_reset", "seedmm_cache_plan",
                 "seedmm_cache_moe", "seedmm_cache_stats", "seedmm_q4_gemv", "seedmm_add_norm",
                 "seedmm_route", "seedmm_moe_block", "seedmm_i8_gemv", "seedmm_moe_sort",
                 "seedmm_moe_unsort", "seedmm_moe_unsort_grad", "seedmm_swiglu", "seedmm_moe_i8"):
        getattr(L, name).restype = i32
    return L


_lib = _load()

EXPORTS = ("seedmm_gemv", "seedmm_gemv_ex", "seedmm_reconstruct", "seedmm_moe_dispatch",
           "seedmm_moe_workspace_bytes", "seedmm_moe", "seedmm_moe_timed", "seedmm_moe_ex",
           "seedmm_moe_noalloc",
           "seedmm_moe_mixed", "seedmm_search", "seedmm_search_table_bytes",
           "seedmm_search_prepare", "seedmm_cache_record_layout", "seedmm_cache_state_bytes",
           "seedmm_cache_device_bytes",
           "seedmm_cache_init", "seedmm_cache_reset", "seedmm_cache_plan", "seedmm_cache_moe",
           "seedmm_cache_stats", "seedmm_q4_gemv", "seedmm_q4_workspace_bytes",
           "seedmm_add_norm", "seedmm_route",
           "seedmm_moe_block_workspace_bytes", "seedmm_moe_block", "seedmm_i8_gemv",
           "seedmm_moe_sort", "seedmm_moe_sort_workspace_bytes", "seedmm_moe_unsort",
           "seedmm_moe_unsort_grad", "seedmm_swiglu", "seedmm_moe_i8_workspace_bytes",
           "seedmm_moe_i8", "seedmm_strerror",
           "seedmm_version")


def lib():
    return _lib


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return ctypes.c_void_p(t)
    return ctypes.c_void_p(t.data_ptr())


# raw handle of a device's current stream without building a torch Stream object
_raw_current = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _current_stream_handle(index=None) -> int:
    if index is None:
        index = torch.cuda.current_device()
    if _raw_current is not None:
        return _raw_current(index)
    return torch.cuda.current_stream(index).cuda_stream


def _stream(stream=None):
    if stream is None:
        return ctypes.c_void_p(_current_stream_handle())
    return ctypes.c_void_p(stream.cuda_stream)


def _on(stream):
    """Allocation context: new tensors belong to `stream` (None: the current stream), so
    the caching allocator does not hand their memory to other streams while the
    library's kernels on `stream` may still use it."""
    return torch.cuda.stream(stream) if stream is not None else _Nothing()


class _Nothing:
    def __enter__(self):
        return None

    def __exit__(self, *a):
        return False


class SideStream:
    """A second stream of one device and its fork / join events, for moe(side=...) and
    moe_mixed(side=...): the layer runs one half of its expert launches there
    (seedmm_moe_ex).  Owned by the caller; concurrent layer calls need one each."""

    def __init__(self, device=None):
        dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
        self.stream = torch.cuda.Stream(device=dev)          # default priority
        # torch deals its streams out of a pool of 32 in turn, so a program's own stream (that of a
        # capture, say) may be this very one; then the calls take another of the pool
        self.spare = torch.cuda.Stream(device=dev)
        while self.spare.cuda_stream == self.stream.cuda_stream:
            self.spare = torch.cuda.Stream(device=dev)
        self.fork = torch.cuda.Event()
        self.join = torch.cuda.Event()
        # torch creates an event on its first record: record both once so handles exist
        self.fork.record(self.stream)
        self.join.record(self.stream)
        self.stream.synchronize()

    def c(self, main: int = 0) -> SeedSide:
        """For a call on the stream with handle `main`, which the second stream is not."""
        second = self.stream.cuda_stream
        return SeedSide(second if second != main else self.spare.cuda_stream, self.fork.cuda_event, self.join.cuda_event)


def _check(status: int, what: str):
    if status != OK:
        raise SeedmmError(status, what)


def _dev(t, dtype, name):
    if not (isinstance(t, torch.Tensor) and t.is_cuda):
        raise TypeError(f"{name} must be a CUDA (HIP) tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


def _mat(m: dict):
    _dev(m["seeds"], torch.uint16, "seeds")
    _dev(m["coefs"], torch.uint16, "coefs")
    _dev(m["codes"], torch.uint8, "codes")
    return m


def stream_sizes(E: int, M: int, K: int, Ps) -> dict:
    """Elements of the seeds (u16), coefs (u16) and codes (u8) streams of E stacked [M][K]
    matrices; Ps is one P for all, or a P per matrix (mixed packs)."""
    n = M * (K // 8)
    Ps = [int(Ps)] * E if isinstance(Ps, int) else [int(p) for p in Ps]
    if len(Ps) != E:
        raise ValueError(f"{len(Ps)} values of P for {E} matrices")
    coef_nibbles = sum(n * p for p in Ps)
    return {"seeds": E * n, "coefs": (coef_nibbles + 3) // 4, "codes": (E * n + 1) // 2}


def _check_streams(m: dict, E: int, M: int, K: int, Ps, name: str, exact_coefs=True):
    """The kernels index the streams from (E, M, K, P) alone: a stream shorter than that
    would be read out of bounds, so it is refused here, before anything is launched."""
    need = stream_sizes(E, M, K, Ps)
    for k, n in need.items():
        if not exact_coefs and k == "coefs":
            continue
        if m[k].numel() < n:
            raise ValueError(f"{name}.{k} has {m[k].numel()} elements; {E} stacked {M}x{K} "
                             f"matrices need {n}")
    eb = m.get("exp_bias")
    if isinstance(eb, torch.Tensor) and eb.numel() < E:
        raise ValueError(f"{name}.exp_bias has {eb.numel()} entries for {E} matrices")


def _check_numel(t, n, name):
    if t.numel() < n:
        raise ValueError(f"{name} has {t.numel()} elements, {n} needed")


def gemv(mat: dict, x: torch.Tensor, M: int, K: int, P: int, y: torch.Tensor = None):
    """y = W x for fp32 x[K] (seedmm_gemv).  The C call has no stream argument and runs on
    the null stream; under another current stream the binding orders it after that
    stream's earlier work and that stream's later work after it (events, no host wait)."""
    _mat(mat)
    _check_streams(mat, 1, M, K, P, "W")
    _dev(x, torch.float32, "x")
    _check_numel(x, K, "x")
    if y is None:
        y = torch.empty(M, dtype=torch.float32, device=x.device)
    _dev(y, torch.float32, "y")
    _check_numel(y, M, "y")
    eb = int(mat["exp_bias_host"][0]) if "exp_bias_host" in mat else int(mat["exp_bias"][0])
    args = (_ptr(mat["seeds"]), _ptr(mat["coefs"]), _ptr(mat["codes"]), eb, _ptr(x), _ptr(y),
            M, K, P)
    idx = x.device.index
    if idx == torch.cuda.current_device() and _current_stream_handle(idx) == 0:
        status = _lib.seedmm_gemv(*args)       # torch's default stream is the null stream
    else:
        with torch.cuda.device(x.device):
            cur, null = torch.cuda.current_stream(), torch.cuda.default_stream()
            null.wait_stream(cur)
            status = _lib.seedmm_gemv(*args)
            cur.wait_stream(null)
    _check(status, "seedmm_gemv")
    return y


def gemv_ex(mat: dict, x: torch.Tensor, M: int, K: int, P: int, y: torch.Tensor = None,
            stream=None):
    """Y[n] = W X[n] for X fp32 or bf16 [N][K] (seedmm_gemv_ex)."""
    _mat(mat)
    if x.dtype not in (torch.float32, torch.bfloat16):
        raise TypeError("x must be float32 or bfloat16")
    _dev(x, x.dtype, "x")
    _check_streams(mat, 1, M, K, P, "W")
    N = x.shape[0] if x.dim() == 2 else 1
    ldx = x.shape[-1]
    if ldx < K:
        raise ValueError(f"x rows hold {ldx} elements, K = {K}")
    if y is None:
        with _on(stream):
            y = torch.empty((N, M), dtype=torch.float32, device=x.device)
    _dev(y, torch.float32, "y")
    if y.shape[-1] < M or y.numel() < N * y.shape[-1]:
        raise ValueError(f"y must hold [{N}][{M}]")
    eb = int(mat["exp_bias_host"][0]) if "exp_bias_host" in mat else int(mat["exp_bias"][0])
    _check(_lib.seedmm_gemv_ex(_ptr(mat["seeds"]), _ptr(mat["coefs"]), _ptr(mat["codes"]), eb,
                               _ptr(x), F32 if x.dtype == torch.float32 else BF16, ldx, _ptr(y),
                               y.shape[-1], M, K, P, N, _stream(stream)), "seedmm_gemv_ex")
    return y


def reconstruct(mat: dict, M: int, K: int, P: int, dtype=torch.float32, out=None, stream=None):
    """W[M][K] in fp32 (exact) or bf16 (seedmm_reconstruct)."""
    _mat(mat)
    _check_streams(mat, 1, M, K, P, "W")
    dev = mat["seeds"].device
    if out is None:
        with _on(stream):
            out = torch.empty((M, K), dtype=dtype, device=dev)
    _dev(out, dtype, "W")
    _check_numel(out, M * K, "W")
    eb = int(mat["exp_bias_host"][0]) if "exp_bias_host" in mat else int(mat["exp_bias"][0])
    _check(_lib.seedmm_reconstruct(_ptr(mat["seeds"]), _ptr(mat["coefs"]), _ptr(mat["codes"]), eb,
                                   _ptr(out), F32 if dtype == torch.float32 else BF16, M, K, P,
                                   _stream(stream)), "seedmm_reconstruct")
    return out


def moe_dispatch(topk_ids: torch.Tensor, E: int, stream=None):
    """(counts int32[E], lists int32[E][T]) for topk_ids int32 [T][top_k]."""
    _dev(topk_ids, torch.int32, "topk_ids")
    T, k = topk_ids.shape
    with _on(stream):
        counts = torch.empty(E, dtype=torch.int32, device=topk_ids.device)
        lists = torch.full((E, max(T, 1)), -1, dtype=torch.int32, device=topk_ids.device)
    _check(_lib.seedmm_moe_dispatch(_ptr(topk_ids), T, k, E, _ptr(counts), _ptr(lists),
                                    _stream(stream)), "seedmm_moe_dispatch")
    return counts, lists


def moe_workspace_bytes(T: int, top_k: int, E: int, H: int, I: int) -> int:
    return int(_lib.seedmm_moe_workspace_bytes(T, top_k, E, H, I))


def _seedmat(m: dict) -> SeedMat:
    _mat(m)
    _dev(m["exp_bias"], torch.int32, "exp_bias")
    return SeedMat(m["seeds"].data_ptr(), m["coefs"].data_ptr(), m["codes"].data_ptr(),
                   m["exp_bias"].data_ptr())


def _check_layer(T, k, topk_w, x, E, H, I, Ps, gate, up, down, exact_coefs=True):
    _check_numel(topk_w, T * k, "topk_w")
    _check_numel(x, T * H, "x")
    for name, m, (M, K) in (("gate", gate, (I, H)), ("up", up, (I, H)), ("down", down, (H, I))):
        _check_streams(m, E, M, K, Ps, name, exact_coefs)


def check_topk_ids(topk_ids, E: int):
    """Host check of a routing's expert ids, which the layer calls leave to the caller:
    every id in [0, E) and the top_k ids of each token distinct.  Copies the ids to the
    host (a synchronisation); raises ValueError naming the first token that breaks it."""
    ids = topk_ids.detach().to("cpu").to(torch.int64)
    if ids.dim() != 2:
        raise ValueError("topk_ids must be [T][top_k]")
    bad = ((ids < 0) | (ids >= E)).any(dim=1)
    if bool(bad.any()):
        t = int(bad.nonzero()[0, 0])
        raise ValueError(f"topk_ids[{t}] holds an expert id outside [0, {E})")
    if ids.shape[1] > 1:
        srt = ids.sort(dim=1).values
        dup = (srt[:, 1:] == srt[:, :-1]).any(dim=1)
        if bool(dup.any()):
            t = int(dup.nonzero()[0, 0])
            raise ValueError(f"topk_ids[{t}] names one expert twice")


def moe(topk_ids, topk_w, x, E, H, I, P, gate, up, down, y=None, workspace=None, stream=None,
        events=None, side=None, check_ids=False):
    """Routed SwiGLU MoE layer (seedmm_moe); x bf16 [T][H] -> y fp32 [T][H].
    `events`: optional 5 raw hipEvent_t handles (ints) recorded between the stages
    (seedmm_moe_timed).  `side`: optional SideStream for the second half of the expert
    launches (seedmm_moe_ex).  `check_ids`: validate topk_ids on the host first
    (check_topk_ids)."""
    if check_ids:
        check_topk_ids(topk_ids, E)
    _dev(topk_ids, torch.int32, "topk_ids")
    _dev(topk_w, torch.float32, "topk_w")
    _dev(x, torch.bfloat16, "x")
    T, k = topk_ids.shape
    _check_layer(T, k, topk_w, x, E, H, I, P, gate, up, down)
    if events is not None and side is not None:
        raise ValueError("the timed layer call runs on one stream (no side stream)")
    with _on(stream):
        if y is None:
            y = torch.empty((T, H), dtype=torch.float32, device=x.device)
        need = moe_workspace_bytes(T, k, E, H, I)
        if workspace is None:
            workspace = torch.empty(need, dtype=torch.uint8, device=x.device)
    _dev(y, torch.float32, "y")
    _check_numel(y, T * H, "y")
    args = (_ptr(topk_ids), _ptr(topk_w), T, k, _ptr(x), _ptr(y), E, H, I, P,
            _seedmat(gate), _seedmat(up), _seedmat(down), _ptr(workspace),
            workspace.numel() * workspace.element_size(), _stream(stream))
    if events is not None:
        arr = (ctypes.c_void_p * 5)(*[getattr(ev, "cuda_event", ev) for ev in events])
        _check(_lib.seedmm_moe_timed(*args, arr), "seedmm_moe_timed")
    elif side is not None:
        sd = side.c(args[-1].value or 0)
        _check(_lib.seedmm_moe_ex(*args[:10], None, *args[10:], ctypes.byref(sd)),
               "seedmm_moe_ex")
    else:
        _check(_lib.seedmm_moe(*args), "seedmm_moe")
    return y


def p4_mask(Ps, device) -> torch.Tensor:
    """Device bitmask of the experts with P = 4 (bit e of word e // 32)."""
    E = len(Ps)
    words = [0] * ((E + 31) // 32)
    for e, P in enumerate(Ps):
        if int(P) == 4:
            words[e >> 5] |= 1 << (e & 31)
        elif int(P) != 3:
            raise ValueError("every expert's P must be 3 or 4")
    return torch.tensor([w - (1 << 32) if w >= (1 << 31) else w for w in words],
                        dtype=torch.int32, device=device)


def moe_mixed(topk_ids, topk_w, x, E, H, I, p4mask, gate, up, down, y=None, workspace=None,
              stream=None, Ps=None, side=None, check_ids=False):
    """Routed SwiGLU MoE layer with P chosen per expert (seedmm_moe_mixed); p4mask from
    p4_mask(Ps).  Given Ps, the coefficient streams are checked against it; without, only
    the seed and code streams are (the mask lives on the device).  `side`: optional
    SideStream for the P = 3 launches (seedmm_moe_ex with P = 0).  `check_ids`: validate
    topk_ids on the host first (check_topk_ids)."""
    if check_ids:
        check_topk_ids(topk_ids, E)
    _dev(topk_ids, torch.int32, "topk_ids")
    _dev(topk_w, torch.float32, "topk_w")
    _dev(x, torch.bfloat16, "x")
    _dev(p4mask, torch.int32, "p4mask")
    _check_numel(p4mask, (E + 31) // 32, "p4mask")
    T, k = topk_ids.shape
    _check_layer(T, k, topk_w, x, E, H, I, Ps if Ps is not None else 3, gate, up, down,
                 exact_coefs=Ps is not None)
    with _on(stream):
        if y is None:
            y = torch.empty((T, H), dtype=torch.float32, device=x.device)
        if workspace is None:
            workspace = torch.empty(moe_workspace_bytes(T, k, E, H, I), dtype=torch.uint8,
                                    device=x.device)
    _dev(y, torch.float32, "y")
    _check_numel(y, T * H, "y")
    args = (_ptr(topk_ids), _ptr(topk_w), T, k, _ptr(x), _ptr(y), E, H, I)
    rest = (_seedmat(gate), _seedmat(up), _seedmat(down), _ptr(workspace),
            workspace.numel() * workspace.element_size(), _stream(stream))
    if side is not None:
        sd = side.c(rest[-1].value or 0)
        _check(_lib.seedmm_moe_ex(*args, 0, _ptr(p4mask), *rest, ctypes.byref(sd)),
               "seedmm_moe_ex")
    else:
        _check(_lib.seedmm_moe_mixed(*args, _ptr(p4mask), *rest), "seedmm_moe_mixed")
    return y


_TABLES = {}


def search_table(P: int, device=None, stream=None):
    """The encoder's per-seed table for P on a device (seedmm_search_prepare), filled
    once and kept by this module for later searches on that device."""
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    key = (dev.index, int(P))
    if key not in _TABLES:
        n = int(_lib.seedmm_search_table_bytes(P))
        if n == 0:
            raise SeedmmError(EINVAL, "seedmm_search_table_bytes")
        with torch.cuda.device(dev):   # the fill runs on that device (its current stream if none given)
            with _on(stream):
                buf = torch.empty(n + 256, dtype=torch.uint8, device=dev)
            off = (-buf.data_ptr()) % 256
            tab = buf[off:off + n]
            _check(_lib.seedmm_search_prepare(P, _ptr(tab), n, _stream(stream)),
                   "seedmm_search_prepare")
            # later searches may run on other streams: wait for the fill once, here
            (stream or torch.cuda.current_stream()).synchronize()
        _TABLES[key] = (buf, tab)
    return _TABLES[key][1]


def search(W: torch.Tensor, P: int, exp_bias: int, colw: torch.Tensor = None, err=True,
           stream=None):
    """Encode fp32 W [M][K] by the exhaustive seed search (seedmm_search): a dict with
    seeds, coefs, codes (device tensors, the products' layout), exp_bias and, if asked,
    err (float64 [M*K/8], squared error of every block)."""
    _dev(W, torch.float32, "W")
    M, K = W.shape
    if colw is not None:
        _dev(colw, torch.float32, "colw")
        _check_numel(colw, K, "colw")
    nblk = M * (K // 8)
    dev = W.device
    table = search_table(P, dev, stream) if colw is None else None
    with _on(stream):
        out = {"seeds": torch.empty(nblk, dtype=torch.uint16, device=dev),
               "coefs": torch.empty((nblk * P + 3) // 4, dtype=torch.uint16, device=dev),
               "codes": torch.empty((nblk + 1) // 2, dtype=torch.uint8, device=dev),
               "exp_bias": torch.full((1,), exp_bias, dtype=torch.int32, device=dev),
               "exp_bias_host": [exp_bias]}
        e = torch.empty(nblk, dtype=torch.float64, device=dev) if err else None
    _check(_lib.seedmm_search(_ptr(W), K, _ptr(colw), M, K, P, exp_bias, _ptr(out["seeds"]),
                              _ptr(out["coefs"]), _ptr(out["codes"]), _ptr(e), _ptr(table),
                              _stream(stream)), "seedmm_search")
    if err:
        out["err"] = e
    return out


class ExpertCache:
    """A layer whose routed experts live in pinned host memory, with S device slots for
    the recently used ones (seedmm_cache_*).  Calls must reach the device in call order:
    use one stream for every call on a cache (a call's record copies can overwrite slots
    the previous call still reads).  host: {"gate", "up", "down"} -> dicts of
    numpy streams (seeds, coefs, codes, exp_bias) stacked as for moe(); they are packed
    once into expert records in pinned host memory (offsets from
    seedmm_cache_record_layout), and the exp_bias arrays go to device memory."""

    def __init__(self, host: dict, E: int, H: int, I: int, P: int, S: int, device="cuda"):
        import numpy as np
        self.E, self.H, self.I, self.P, self.S = E, H, I, P, S
        offs = (ctypes.c_size_t * 9)()
        rec = int(_lib.seedmm_cache_record_layout(H, I, P, offs))
        nstate = int(_lib.seedmm_cache_state_bytes(E, S))
        ndev = int(_lib.seedmm_cache_device_bytes(E, H, I, P, S))
        if rec == 0 or nstate == 0 or ndev == 0:
            raise SeedmmError(EINVAL, "seedmm_cache sizes")
        self.record_bytes = rec
        for n, (M, K) in (("gate", (I, H)), ("up", (I, H)), ("down", (H, I))):
            need = stream_sizes(E, M, K, P)
            for part, cnt in need.items():
                if np.asarray(host[n][part]).size < cnt:
                    raise ValueError(f"{n}.{part} has {np.asarray(host[n][part]).size} "
                                     f"elements; {E} stacked {M}x{K} matrices need {cnt}")
            if np.asarray(host[n]["exp_bias"]).size < E:
                raise ValueError(f"{n}.exp_bias has fewer than {E} entries")
        pack = torch.zeros(E * rec, dtype=torch.uint8, pin_memory=True)
        view = pack.numpy().reshape(E, rec)
        for m, n in enumerate(("gate", "up", "down")):
            for k, part in enumerate(("seeds", "coefs", "codes")):
                a = np.ascontiguousarray(host[n][part]).view(np.uint8).reshape(E, -1)
                o = offs[3 * m + k]
                view[:, o:o + a.shape[1]] = a
        self._pack = pack
        eb = np.stack([np.asarray(host[n]["exp_bias"], dtype=np.int32) for n in ("gate", "up", "down")])
        self._exp_bias = torch.from_numpy(np.ascontiguousarray(eb)).to(device)
        self._state = torch.empty((nstate + 7) // 8, dtype=torch.int64)   # host, 8-byte aligned
        self._device = torch.empty(ndev + 256, dtype=torch.uint8, device=device)
        off = (-self._device.data_ptr()) % 256
        _check(_lib.seedmm_cache_init(self.handle, nstate, E, H, I, P, S,
                                      ctypes.c_void_p(pack.data_ptr()),
                                      ctypes.c_void_p(self._exp_bias.data_ptr()),
                                      ctypes.c_void_p(self._device.data_ptr() + off), ndev),
               "seedmm_cache_init")

    @property
    def handle(self):
        return ctypes.c_void_p(self._state.data_ptr())

    @property
    def device_bytes(self) -> int:
        return int(_lib.seedmm_cache_device_bytes(self.E, self.H, self.I, self.P, self.S))

    def reset(self):
        _check(_lib.seedmm_cache_reset(self.handle), "seedmm_cache_reset")

    def plan(self, topk_ids_host):
        """Host-only plan of one call: [(expert, slot), ...] loads (changes the state)."""
        import numpy as np
        ids = np.ascontiguousarray(topk_ids_host, dtype=np.int32)
        T, k = ids.shape
        loads = np.zeros(2 * self.S, dtype=np.int32)
        n = ctypes.c_int(0)
        _check(_lib.seedmm_cache_plan(self.handle, ids.ctypes.data_as(ctypes.c_void_p), T, k,
                                      loads.ctypes.data_as(ctypes.c_void_p), ctypes.byref(n)),
               "seedmm_cache_plan")
        return [(int(loads[2 * i]), int(loads[2 * i + 1])) for i in range(n.value)]

    def moe(self, topk_ids_host, topk_ids, topk_w, x, y=None, workspace=None, stream=None):
        """The routed layer through the cache (seedmm_cache_moe); topk_ids_host is the
        host copy (numpy int32 [T][top_k]) of the device topk_ids."""
        import numpy as np
        ids_h = np.ascontiguousarray(topk_ids_host, dtype=np.int32)
        _dev(topk_ids, torch.int32, "topk_ids")
        _dev(topk_w, torch.float32, "topk_w")
        _dev(x, torch.bfloat16, "x")
        T, k = topk_ids.shape
        if ids_h.shape != (T, k):
            raise ValueError("topk_ids_host and topk_ids differ in shape")
        _check_numel(topk_w, T * k, "topk_w")
        _check_numel(x, T * self.H, "x")
        with _on(stream):
            if y is None:
                y = torch.empty((T, self.H), dtype=torch.float32, device=x.device)
            if workspace is None:
                workspace = torch.empty(moe_workspace_bytes(T, k, self.E, self.H, self.I),
                                        dtype=torch.uint8, device=x.device)
        _dev(y, torch.float32, "y")
        _check_numel(y, T * self.H, "y")
        _check(_lib.seedmm_cache_moe(self.handle, ids_h.ctypes.data_as(ctypes.c_void_p),
                                     _ptr(topk_ids), _ptr(topk_w), T, k, _ptr(x), _ptr(y),
                                     _ptr(workspace),
                                     workspace.numel() * workspace.element_size(),
                                     _stream(stream)), "seedmm_cache_moe")
        return y

    def stats(self) -> dict:
        out = (ctypes.c_uint64 * 5)()
        _check(_lib.seedmm_cache_stats(self.handle, out), "seedmm_cache_stats")
        return dict(zip(("calls", "uses", "hits", "misses", "bytes"), (int(v) for v in out)))


# ---- dense operators around the routed layer -----------------------------------------
# Their arguments are checked and marshalled in the module _binding (csrc/binding.cpp).  It is
# built against the installed torch and loaded by the first call that needs it, so that the
# calls above work without it.

_dense = None      # the module, once loaded


def _load_binding():
    global _dense
    path = os.path.join(_HERE, "_binding.so")
    if not os.path.exists(path):
        raise ImportError(f"{path} is missing: build it with "
                          "`python -m pseudo_random_weight_amd.build`")
    from . import _binding as m
    m.init(*(ctypes.cast(getattr(_lib, n), ctypes.c_void_p).value
             for n in ("seedmm_q4_gemv", "seedmm_q4_workspace_bytes", "seedmm_add_norm",
                       "seedmm_route")), SeedmmError)
    m.init_experts(*(ctypes.cast(getattr(_lib, n), ctypes.c_void_p).value
                     for n in ("seedmm_i8_gemv", "seedmm_moe_sort", "seedmm_moe_sort_workspace_bytes",
                               "seedmm_moe_unsort", "seedmm_moe_unsort_grad", "seedmm_swiglu",
                               "seedmm_moe_i8", "seedmm_moe_i8_workspace_bytes")))
    _dense = m
    return m


def __getattr__(name):
    if name == "_binding":
        return _dense or _load_binding()
    raise AttributeError(f"module {__name__!r} has no attribute {name!r}")


_FLOATS = {torch.float32: F32, torch.bfloat16: BF16}
_ROWS = {torch.float32: F32, torch.bfloat16: BF16, torch.int8: I8}
_INT32 = {torch.int32: 0}
_FP32 = {torch.float32: F32}


def _flat(t, types, n, name, dev):
    """dtype code of a contiguous GPU tensor of at least n elements."""
    if not (isinstance(t, torch.Tensor) and t.is_cuda):
        raise TypeError(f"{name} must be a CUDA (HIP) tensor")
    if t.dtype not in types:
        raise TypeError(f"{name} must be one of {[str(d) for d in types]}, got {t.dtype}")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on another device")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.numel() < n:
        raise ValueError(f"{name} has {t.numel()} elements, {n} needed")
    return types[t.dtype]


def _check_q4(mat, M, K, group, dev):
    if group not in (32, 64, 128) or K % group:
        raise ValueError(f"K = {K} must be a multiple of the group, and the group 32, 64 or 128")
    _flat(mat["weight"], {torch.uint32: 0}, M * (K // 8), "weight", dev)
    sd = _flat(mat["scales"], _FLOATS, M * (K // group), "scales", dev)
    if _flat(mat["biases"], _FLOATS, M * (K // group), "biases", dev) != sd:
        raise TypeError("scales and biases must have one type")
    return sd


def _handle(stream, t):
    """A stream's handle for the call on tensor t's device (None: its current stream)."""
    if stream is None:
        return None
    if stream.device.index != t.get_device():
        raise ValueError("the stream belongs to another device than the tensors")
    return stream.cuda_stream


def _gpu(t, name):
    if not (isinstance(t, torch.Tensor) and t.is_cuda):
        raise TypeError(f"{name} must be a CUDA (HIP) tensor")
    return t


def q4_workspace_bytes(x_dtype, group: int, M: int, K: int, N: int) -> int:
    """Bytes of the workspace that q4_gemv needs for N rows of x_dtype."""
    return int(_lib.seedmm_q4_workspace_bytes(_ROWS[x_dtype], group, M, K, N))


def q4_gemv(mat: dict, x: torch.Tensor, M: int, K: int, group: int = 64, x_scale=None, y=None,
            y_dtype=torch.float32, workspace=None, stream=None):
    """y = x W^T for W in affine 4 bits (seedmm_q4_gemv).  mat: {"weight": uint32 [M*K/8],
    "scales", "biases": fp32 or bf16 [M*K/group]}; x fp32, bf16 or int8 [N][K] (or [K]),
    int8 rows with x_scale fp32 [N]; y [N][M] (or [M]) fp32 or bf16.  workspace: a GPU tensor
    of q4_workspace_bytes(...) bytes, allocated here if it is needed and not given."""
    if y is None:
        with _on(stream):
            y = torch.empty((*_gpu(x, "x").shape[:-1], M), dtype=y_dtype, device=x.device)
    if stream is not None:
        _gpu(x, "x")
        if workspace is None and x.dtype in _ROWS and x.dim() == 2:
            need = q4_workspace_bytes(x.dtype, group, M, K, x.shape[0])
            if need:       # scratch of a call on another stream belongs to that stream
                with _on(stream):
                    workspace = torch.empty(need, dtype=torch.uint8, device=x.device)
        stream = _handle(stream, x)
    (_dense or _load_binding()).q4_gemv(mat["weight"], mat["scales"], mat["biases"], group, x,
                                        x_scale, y, workspace, M, K, stream)
    return y


def add_norm(x: torch.Tensor, weight=None, delta=None, eps: float = 1e-6,
             out_dtype=torch.bfloat16, residual=None, out=None, scale=None, stream=None):
    """(out, scale, residual): r = x + delta and its root-mean-square norm (seedmm_add_norm).
    x fp32 or bf16 [N][H] (or [H]); delta fp32 or bf16 of x's shape or None; weight fp32 or
    bf16 [H] or None; out of out_dtype (float32, bfloat16, or int8 with scale fp32 [N]; scale
    is None otherwise).  residual: r in x's type (pass x itself to update it in place); x if
    there is no delta and none is asked for."""
    if out is None:
        with _on(stream):
            out = torch.empty(_gpu(x, "x").shape, dtype=out_dtype, device=x.device)
    if scale is None and out.dtype is torch.int8:
        with _on(stream):
            scale = torch.empty(_gpu(x, "x").shape[:-1] if x.dim() > 1 else 1, dtype=torch.float32,
                                device=x.device)
    if delta is not None and residual is None:
        with _on(stream):
            residual = torch.empty(_gpu(x, "x").shape, dtype=x.dtype, device=x.device)
    (_dense or _load_binding()).add_norm(x, weight, delta, eps, residual, out, scale,
                                         None if stream is None else _handle(stream, _gpu(x, "x")))
    return out, scale, x if residual is None else residual


_SCORES = {"softmax": SOFTMAX, "sigmoid": SIGMOID}


def route(logits: torch.Tensor, top_k: int, bias=None, score: str = "softmax", ids=None, w=None,
          stream=None):
    """(ids int32 [T][top_k], w fp32 [T][top_k]) of router logits fp32 or bf16 [T][E]
    (seedmm_route): the routing that moe() takes.  score "softmax", or "sigmoid" with an
    optional fp32 selection bias [E]."""
    kind = _SCORES.get(score)
    if kind is None:
        raise ValueError(f"score must be one of {sorted(_SCORES)}")
    if ids is None or w is None:
        if _gpu(logits, "logits").dim() != 2 or top_k < 1:
            raise ValueError("logits must be [T][E] and top_k positive")
        shape = (logits.shape[0], top_k)
        with _on(stream):
            if ids is None:
                ids = torch.empty(shape, dtype=torch.int32, device=logits.device)
            if w is None:
                w = torch.empty(shape, dtype=torch.float32, device=logits.device)
    (_dense or _load_binding()).route(logits, top_k, bias, kind, ids, w,
                                      None if stream is None else _handle(stream, _gpu(logits, "logits")))
    return ids, w


class MoeBlock:
    """One routed layer with its norm and router (seedmm_moe_block): holds the layer's
    tensors.  gate/up/down as for moe(); router: an [E][H] affine 4-bit matrix as for
    q4_gemv(); norm_weight fp32 or bf16 [H] or None.  P = 3 or 4, or Ps (a P per expert)
    for mixed packs."""

    def __init__(self, E, H, I, P, top_k, gate, up, down, router, group=64, norm_weight=None,
                 eps=1e-6, score="softmax", router_bias=None, Ps=None):
        dev = gate["seeds"].get_device()
        for name, m, (M, K) in (("gate", gate, (I, H)), ("up", up, (I, H)), ("down", down, (H, I))):
            _seedmat(m)
            _check_streams(m, E, M, K, Ps if Ps is not None else P, name)
            for part in ("seeds", "coefs", "codes", "exp_bias"):
                if m[part].get_device() != dev:
                    raise ValueError(f"{name}.{part} is on another device")
        if score not in _SCORES:
            raise ValueError(f"score must be one of {sorted(_SCORES)}")
        rd = _check_q4(router, E, H, group, dev)
        nd = F32 if norm_weight is None else _flat(norm_weight, _FLOATS, H, "norm_weight", dev)
        if router_bias is not None:
            _flat(router_bias, _FP32, E, "router_bias", dev)
        self.p4mask = None if Ps is None else p4_mask(Ps, gate["seeds"].device)
        self.E, self.H, self.top_k, self.device = E, H, top_k, gate["seeds"].device
        self._keep = (gate, up, down, router, norm_weight, router_bias)
        ptr = lambda t: None if t is None else t.data_ptr()
        self._c = SeedBlock(ptr(norm_weight), ptr(router["weight"]), ptr(router["scales"]),
                            ptr(router["biases"]), ptr(router_bias), ptr(self.p4mask),
                            _seedmat(gate), _seedmat(up), _seedmat(down), eps, nd, rd, group,
                            _SCORES[score], top_k, E, H, I, 0 if Ps is not None else P)
        if self.workspace_bytes(1) == 0:
            raise SeedmmError(EINVAL, "seedmm_moe_block sizes")

    def workspace_bytes(self, T: int) -> int:
        return int(_lib.seedmm_moe_block_workspace_bytes(ctypes.byref(self._c), T))

    def moe(self, r, delta=None, y=None, ids=None, w=None, workspace=None, stream=None, side=None):
        """y fp32 [T][H] of the residual stream r (fp32 or bf16 [T][H], contiguous), which
        delta (fp32 or bf16 [T][H]) is added to in place first.  ids, w: optional tensors
        that receive the routing."""
        dev = self.device.index
        rd = _flat(r, _FLOATS, 0, "r", dev)
        if r.dim() != 2 or r.shape[1] != self.H:
            raise ValueError(f"r must be [T][{self.H}]")
        T = r.shape[0]
        dd = F32 if delta is None else _flat(delta, _FLOATS, T * self.H, "delta", dev)
        with _on(stream):
            if y is None:
                y = torch.empty((T, self.H), dtype=torch.float32, device=r.device)
            if workspace is None:
                workspace = torch.empty(self.workspace_bytes(T), dtype=torch.uint8, device=r.device)
        _flat(y, _FP32, T * self.H, "y", dev)
        if ids is not None:
            _flat(ids, _INT32, T * self.top_k, "ids", dev)
        if w is not None:
            _flat(w, _FP32, T * self.top_k, "w", dev)
        if not isinstance(workspace, torch.Tensor):
            raise TypeError("the workspace must be a tensor")
        if workspace.get_device() != dev or not workspace.is_contiguous():
            raise ValueError("the workspace must be a contiguous tensor on the layer's device")
        ptr = lambda t: None if t is None else t.data_ptr()
        handle = _handle(stream, r)
        if handle is None:
            handle = _current_stream_handle(dev)
        sd = None if side is None else ctypes.byref(side.c(handle))
        with torch.cuda.device(dev):
            _check(_lib.seedmm_moe_block(
                ctypes.byref(self._c), r.data_ptr(), rd, ptr(delta), dd, y.data_ptr(), ptr(ids),
                ptr(w), T, workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                handle, sd), "seedmm_moe_block")
        return y


# ---- routed experts in 8-bit integers ------------------------------------------------

def i8_gemv(mat: dict, x: torch.Tensor, x_scale: torch.Tensor, M: int, K: int, y=None,
            y_dtype=torch.float32, offsets=None, stream=None):
    """y = x W^T in 8-bit integers with a scale a row and a channel (seedmm_i8_gemv).  mat:
    {"weight": int8 [M*K], "scales": fp32 or bf16 [M]}; x int8 [N][K] (or [K]) with x_scale
    fp32 [N]; y [N][M] (or [M]) fp32 or bf16.  offsets: int32 [E+1] of moe_sort, for rows sorted
    by expert and E stacked matrices; rows of y behind offsets[E] are left as they were (a y
    allocated here holds no values there)."""
    if y is None:
        if M < 0:
            raise ValueError(f"M = {M} is out of range")
        with _on(stream):
            y = torch.empty((*_gpu(x, "x").shape[:-1], M), dtype=y_dtype, device=x.device)
    (_dense or _load_binding()).i8_gemv(mat["weight"], mat["scales"], x, x_scale, y, offsets, M, K,
                                        None if stream is None else _handle(stream, _gpu(x, "x")))
    return y


def moe_sort_workspace_bytes(T: int, top_k: int, E: int) -> int:
    """Bytes of the workspace that moe_sort needs for T tokens."""
    return int(_lib.seedmm_moe_sort_workspace_bytes(T, top_k, E))


def moe_sort(x: torch.Tensor, topk_ids: torch.Tensor, E: int, x_scale=None, rows=None,
             row_scale=None, offsets=None, inverse=None, workspace=None, stream=None):
    """(rows, row_scale, offsets, inverse): the tokens' rows in the order of their experts
    (seedmm_moe_sort).  x fp32, bf16 or int8 [T][H], with x_scale fp32 [T] or None; topk_ids
    int32 [T][top_k], ids outside of [0, E) dropped.  rows [T*top_k][H] and row_scale (None
    without x_scale) hold values up to row offsets[E]; offsets int32 [E+1]; inverse int32
    [T][top_k], the row of each slot or -1."""
    if rows is None or offsets is None or inverse is None or (x_scale is not None and row_scale is None):
        if _gpu(topk_ids, "topk_ids").dim() != 2:
            raise ValueError("topk_ids must be a contiguous [T][top_k] tensor")
        n, dev = topk_ids.numel(), _gpu(x, "x").device
        with _on(stream):
            if rows is None:
                rows = torch.empty((n, x.shape[-1]), dtype=x.dtype, device=dev)
            if row_scale is None and x_scale is not None:
                row_scale = torch.empty(n, dtype=torch.float32, device=dev)
            if offsets is None:
                offsets = torch.empty(E + 1, dtype=torch.int32, device=dev)
            if inverse is None:
                inverse = torch.empty(topk_ids.shape, dtype=torch.int32, device=dev)
    if stream is not None:
        if workspace is None and _gpu(topk_ids, "topk_ids").dim() == 2:
            need = moe_sort_workspace_bytes(*topk_ids.shape, E)
            if need:       # scratch of a call on another stream belongs to that stream
                with _on(stream):
                    workspace = torch.empty(need, dtype=torch.uint8, device=_gpu(x, "x").device)
        stream = _handle(stream, _gpu(x, "x"))
    (_dense or _load_binding()).moe_sort(x, topk_ids, E, x_scale, rows, row_scale, offsets, inverse,
                                         workspace, stream)
    return rows, row_scale, offsets, inverse


def moe_unsort(rows: torch.Tensor, inverse: torch.Tensor, topk_w=None, y=None,
               y_dtype=torch.float32, stream=None):
    """y [T][H] fp32 or bf16: each token's rows, weighted and summed (seedmm_moe_unsort).  rows
    fp32 or bf16 [n][H]; inverse int32 [T][top_k] of moe_sort; topk_w fp32 [T][top_k] or None
    (ones: the gradient of moe_sort's rows with respect to x)."""
    if y is None:
        with _on(stream):
            y = torch.empty((_gpu(inverse, "inverse").shape[0], _gpu(rows, "rows").shape[-1]),
                            dtype=y_dtype, device=rows.device)
    (_dense or _load_binding()).moe_unsort(rows, inverse, topk_w, y,
                                           None if stream is None else _handle(stream, _gpu(rows, "rows")))
    return y


def moe_unsort_grad(dy: torch.Tensor, rows: torch.Tensor, inverse: torch.Tensor,
                    topk_w: torch.Tensor, drows=None, dw=None, stream=None):
    """(drows, dw): moe_unsort's gradients for dy fp32 or bf16 [T][H] (seedmm_moe_unsort_grad), to be
    called by the caller's backward pass: moe_unsort itself records none.
    drows has rows' shape and type (rows that no slot names are left as they were; a drows
    allocated here holds no values there), dw is fp32 [T][top_k]."""
    if drows is None or dw is None:
        with _on(stream):
            if drows is None:
                drows = torch.empty(_gpu(rows, "rows").shape, dtype=rows.dtype, device=rows.device)
            if dw is None:
                dw = torch.empty(_gpu(inverse, "inverse").shape, dtype=torch.float32,
                                 device=inverse.device)
    (_dense or _load_binding()).moe_unsort_grad(
        dy, rows, inverse, topk_w, drows, dw,
        None if stream is None else _handle(stream, _gpu(rows, "rows")))
    return drows, dw


def swiglu(gate_up: torch.Tensor, out_dtype=torch.bfloat16, out=None, scale=None, count=None,
           stream=None):
    """(out, scale): silu(gate) * up of rows [N][2I] fp32 or bf16 that hold gate, then up
    (seedmm_swiglu).  out [N][I] of out_dtype (float32, bfloat16, or int8 with scale fp32 [N];
    scale is None otherwise).  count: int32 [1] on the GPU, the number of rows that exist
    (offsets[E:] of moe_sort), or None for all."""
    if out is None:
        with _on(stream):
            out = torch.empty((*_gpu(gate_up, "gate_up").shape[:-1], gate_up.shape[-1] // 2),
                              dtype=out_dtype, device=gate_up.device)
    if scale is None and out.dtype is torch.int8:
        with _on(stream):
            scale = torch.empty(_gpu(gate_up, "gate_up").shape[:-1] if gate_up.dim() > 1 else 1,
                                dtype=torch.float32, device=gate_up.device)
    (_dense or _load_binding()).swiglu(gate_up, out, scale, count,
                                       None if stream is None else _handle(stream, _gpu(gate_up, "gate_up")))
    return out, scale


def moe_i8_workspace_bytes(T: int, top_k: int, E: int, H: int, I: int) -> int:
    """Bytes of the workspace that moe_i8 needs for T tokens."""
    return int(_lib.seedmm_moe_i8_workspace_bytes(T, top_k, E, H, I))


def moe_i8(topk_ids, topk_w, x, x_scale, E, H, I, gate_up, down, y=None, workspace=None,
           stream=None):
    """y fp32 [T][H]: the routed SwiGLU layer of experts in 8-bit integers (seedmm_moe_i8).  x
    int8 [T][H] with x_scale fp32 [T] (add_norm's); gate_up, down: matrices as for i8_gemv, E
    stacked [2I][H] (gate rows, then up rows) and [H][I]; topk_ids int32 and topk_w fp32
    [T][top_k], an id outside of [0, E) drops its slot.  The rows behind both products are bf16; for
    fp32 ones behind the second, call moe_sort, i8_gemv, swiglu, i8_gemv and moe_unsort."""
    if y is None:
        with _on(stream):
            y = torch.empty(_gpu(x, "x").shape, dtype=torch.float32, device=x.device)
    if stream is not None:
        if workspace is None and _gpu(topk_ids, "topk_ids").dim() == 2:
            with _on(stream):
                workspace = torch.empty(moe_i8_workspace_bytes(*topk_ids.shape, E, H, I),
                                        dtype=torch.uint8, device=_gpu(x, "x").device)
        stream = _handle(stream, _gpu(x, "x"))
    (_dense or _load_binding()).moe_i8(topk_ids, topk_w, x, x_scale, E, H, I, gate_up["weight"],
                                       gate_up["scales"], down["weight"], down["scales"], y, workspace,
                                       stream)
    return y
