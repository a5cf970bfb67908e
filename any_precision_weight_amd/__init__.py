"""Python binding of libapmoe (ctypes), the any-precision MoE expert layer for
MI355X (gfx950).

Argument marshalling only: every step runs in the HIP kernels of
``libapmoe.so``.  Tensors are torch device tensors (PyTorch provides device
memory and streams); they are passed to the C ABI as raw pointers.  There is
no fallback: if the library is missing, importing the functions raises.

Function names and argument order follow ``include/apmoe.h``.
"""
from __future__ import annotations

import ctypes
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libapmoe.so")
# the same library built with every counted vector-memory wait drained to zero
SAFE_LIB_PATH = os.path.join(_HERE, "libapmoe_safe.so")

OK, INVALID_ARG, UNSUPPORTED, NOT_RESIDENT, HIP_ERROR, OUT_OF_MEMORY = range(6)
GATE_UP, DOWN = 0, 1
F16, F32, BF16, E4M3 = 0, 1, 2, 3
MIN_BITS, MAX_BITS, PLANES = 3, 8, 8

EXPORTED = [
    "apmoe_status_string", "apmoe_last_error", "apmoe_version", "apmoe_create", "apmoe_destroy", "apmoe_ctx_faults",
    "apmoe_block_bytes", "apmoe_table_create", "apmoe_table_destroy", "apmoe_table_set_block",
    "apmoe_table_set_bits", "apmoe_table_set_plane", "apmoe_table_validate", "apmoe_table_committed_bits",
    "apmoe_table_commit", "apmoe_lut_build", "apmoe_tiled_plane_words", "apmoe_tile_planes", "apmoe_pack_planes", "apmoe_route", "apmoe_route_workspace", "apmoe_route_stats", "apmoe_gemm",
    "apmoe_gemm_act", "apmoe_act",
    "apmoe_combine", "apmoe_moe_workspace", "apmoe_moe_forward", "apmoe_page_out", "apmoe_page_in",
    "apmoe_moe_forward_noalloc", "apmoe_norm", "apmoe_gemm_fp8", "apmoe_gemm_act_fp8", "apmoe_moe_workspace_fp8",
    "apmoe_moe_forward_fp8", "apmoe_kv_append", "apmoe_attn_workspace", "apmoe_attn_decode", "apmoe_attn_prefill",
]


class ApmoeError(RuntimeError):
    def __init__(self, status: int, fn: str, detail: str):
        self.status = status
        super().__init__(f"{fn}: status {status} ({_status_text(status)}): {detail}")


class BlockDesc(ctypes.Structure):
    _fields_ = [
        ("n", ctypes.c_int32), ("k", ctypes.c_int32), ("q", ctypes.c_int32), ("d", ctypes.c_int32),
        ("resident_mask", ctypes.c_uint32),
        ("plane", ctypes.c_void_p * PLANES),
        ("lut", ctypes.c_void_p * (MAX_BITS + 1)),
    ]


class Fp8Desc(ctypes.Structure):
    _fields_ = [
        ("E", ctypes.c_int32), ("H", ctypes.c_int32), ("F", ctypes.c_int32),
        ("gate_up", ctypes.c_void_p), ("gate_up_scale", ctypes.c_void_p),
        ("down", ctypes.c_void_p), ("down_scale", ctypes.c_void_p),
    ]


class KvCacheDesc(ctypes.Structure):
    _fields_ = [
        ("dtype", ctypes.c_int32), ("n_pages", ctypes.c_int32), ("page", ctypes.c_int32),
        ("kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
        ("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p),
    ]


class KvBatchDesc(ctypes.Structure):
    _fields_ = [
        ("B", ctypes.c_int32), ("T", ctypes.c_int32), ("max_pages", ctypes.c_int32), ("max_len", ctypes.c_int32),
        ("pages", ctypes.c_void_p), ("lens", ctypes.c_void_p), ("q_offsets", ctypes.c_void_p),
    ]


_lib = None


def _status_text(s: int) -> str:
    try:
        return lib().apmoe_status_string(s).decode()
    except Exception:  # pragma: no cover - library missing
        return "?"


_loaded: dict[str, ctypes.CDLL] = {}


def load_library(path: str) -> ctypes.CDLL:
    """Load a libapmoe build (once per path; raises if it has not been built).
    Contexts and tables remember the library that made them, so two builds can be
    used side by side in one process."""
    if path not in _loaded:
        if not os.path.exists(path):
            raise ImportError(f"{path} is missing: build it with `python -m any_precision_weight_amd.build`")
        L = ctypes.CDLL(path)
        _declare(L)
        _loaded[path] = L
    return _loaded[path]


def lib() -> ctypes.CDLL:
    """The default build, libapmoe.so."""
    global _lib
    if _lib is None:
        _lib = load_library(LIB_PATH)
    return _lib


def _declare(L):
    P, I32, I64, SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
    F32_ = ctypes.c_float
    S = ctypes.c_int32
    sig = {
        "apmoe_status_string": (ctypes.c_char_p, [S]),
        "apmoe_last_error": (ctypes.c_char_p, []),
        "apmoe_version": (I32, []),
        "apmoe_create": (S, [ctypes.POINTER(P), ctypes.c_int]),
        "apmoe_destroy": (S, [P]),
        "apmoe_ctx_faults": (S, [P, ctypes.POINTER(I32)]),
        "apmoe_block_bytes": (I64, [I32, I32, I32]),
        "apmoe_table_create": (S, [I32, I32, ctypes.POINTER(P)]),
        "apmoe_table_destroy": (S, [P]),
        "apmoe_table_set_block": (S, [P, I32, I32, I32, ctypes.POINTER(BlockDesc)]),
        "apmoe_table_set_bits": (S, [P, I32, I32, I32, I32]),
        "apmoe_table_set_plane": (S, [P, I32, I32, I32, I32, P, I32]),
        "apmoe_table_validate": (S, [P]),
        "apmoe_table_committed_bits": (S, [P, I32, I32, I32, ctypes.POINTER(I32)]),
        "apmoe_table_commit": (S, [P, P, P]),
        "apmoe_lut_build": (S, [P, P, I32, P, P]),
        "apmoe_tiled_plane_words": (I64, [I32, I32]),
        "apmoe_tile_planes": (S, [P, P, I32, I32, P, P]),
        "apmoe_pack_planes": (S, [P, P, I32, I32, P, P]),
        "apmoe_route": (S, [P, P, P, P, I32, I32, I32, I32, I32, I32, P, P, P, P, P, P, P]),
        "apmoe_route_workspace": (S, [P, I32, I32, I32, I32, ctypes.POINTER(SZ)]),
        "apmoe_route_stats": (S, [P, P, P, P, I32, I32, I32, P, P, P, P]),
        "apmoe_gemm": (S, [P, P, I32, I32, P, I32, P, P, I32, I32, P, I32, P]),
        "apmoe_gemm_act": (S, [P, P, I32, P, I32, P, P, I32, I32, P, P]),
        "apmoe_act": (S, [P, P, I32, I32, P, P]),
        "apmoe_combine": (S, [P, P, I32, P, P, I32, I32, I32, P, P]),
        "apmoe_moe_workspace": (S, [P, I32, I32, I32, I32, ctypes.POINTER(SZ)]),
        "apmoe_moe_forward": (S, [P, P, I32, P, P, P, I32, I32, I32, I32, P, SZ, P, P]),
        "apmoe_moe_forward_noalloc": (S, [P, P, I32, P, P, P, I32, I32, I32, I32, P, P]),
        "apmoe_norm": (S, [P, P, I32, P, P, I32, P, F32_, I32, I32, P, P, P, P]),
        "apmoe_gemm_fp8": (S, [P, P, P, P, P, I32, I32, I32, I32, P, P, I32, I32, P, I32, P]),
        "apmoe_gemm_act_fp8": (S, [P, P, P, P, P, I32, I32, I32, I32, P, P, I32, I32, P, P, P]),
        "apmoe_moe_workspace_fp8": (S, [P, ctypes.POINTER(Fp8Desc), I32, I32, I32, ctypes.POINTER(SZ)]),
        "apmoe_moe_forward_fp8": (S, [P, ctypes.POINTER(Fp8Desc), P, P, P, P, P, I32, I32, I32, I32, P, SZ, P, P]),
        "apmoe_kv_append": (S, [P, ctypes.POINTER(KvCacheDesc), ctypes.POINTER(KvBatchDesc), P, I64, P, I64, P, I64, I32,
                                I32, P, I32, I32, I32, P, P]),
        "apmoe_attn_workspace": (S, [P, ctypes.POINTER(KvCacheDesc), ctypes.POINTER(KvBatchDesc), I32,
                                     ctypes.POINTER(SZ)]),
        "apmoe_attn_decode": (S, [P, ctypes.POINTER(KvCacheDesc), ctypes.POINTER(KvBatchDesc), P, I64, I32, I32, F32_,
                                  I32, I32, P, SZ, P, P, P, P]),
        "apmoe_attn_prefill": (S, [P, ctypes.POINTER(KvCacheDesc), ctypes.POINTER(KvBatchDesc), P, I64, I32, I32, F32_,
                                   I32, I32, P, SZ, P, P, P, P]),
        "apmoe_page_out": (S, [P, P, I32, I32, I32, I32, ctypes.POINTER(P), P, P, P]),
        "apmoe_page_in": (S, [P, P, I32, I32, I32, I32, ctypes.POINTER(P), ctypes.POINTER(P), P, P, P]),
    }
    for name, (res, args) in sig.items():
        f = getattr(L, name)
        f.restype = res
        f.argtypes = args


def _check(status: int, fn: str, L: ctypes.CDLL | None = None) -> None:
    if status != OK:
        raise ApmoeError(status, fn, (L or lib()).apmoe_last_error().decode())


def ptr(t) -> int | None:
    """Raw pointer of a torch tensor / int / None."""
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def stream_handle(stream=None) -> int | None:
    import torch
    s = torch.cuda.current_stream() if stream is None else stream
    return s.cuda_stream or None


# --------------------------------------------------------------------------- API

def version() -> int:
    return lib().apmoe_version()


def block_bytes(n: int, k: int, b: int) -> int:
    return int(lib().apmoe_block_bytes(n, k, b))


class Context:
    """apmoe_create / apmoe_destroy.  A context owns a side stream and the completion
    counters of the fused launches: calls on one context that may run at the same time
    must be ordered by the caller (or use a context each).  APMOE_UNFUSED=1 in the
    environment when the context is created gives one that runs every layer step in
    its own launches; APMOE_LAYER_KERNEL=1 one that runs a small batch's gate_up and
    down in one launch (the one-launch decode layer) instead of two."""

    def __init__(self, device: int = 0, library: ctypes.CDLL | None = None):
        self.L = lib() if library is None else library
        h = ctypes.c_void_p()
        _check(self.L.apmoe_create(ctypes.byref(h), device), "apmoe_create", self.L)
        self.handle = h.value
        self.device = device

    def faults(self) -> int:
        """apmoe_ctx_faults: the context's sticky fault flags (0 = none; synchronises)."""
        v = ctypes.c_int32()
        _check(self.L.apmoe_ctx_faults(self.handle, ctypes.byref(v)), "apmoe_ctx_faults", self.L)
        return v.value

    def close(self):
        if self.handle:
            self.L.apmoe_destroy(self.handle)
            self.handle = None

    def __del__(self):  # pragma: no cover
        try:
            self.close()
        except Exception:
            pass


class Table:
    """apmoe_table_* : staging, validation and stream-ordered commit."""

    def __init__(self, n_layers: int, n_experts: int, library: ctypes.CDLL | None = None):
        self.L = lib() if library is None else library
        h = ctypes.c_void_p()
        _check(self.L.apmoe_table_create(n_layers, n_experts, ctypes.byref(h)), "apmoe_table_create", self.L)
        self.handle = h.value
        self.n_layers, self.n_experts = n_layers, n_experts

    def set_block(self, layer: int, expert: int, kind: int, n: int, k: int, q: int, planes, luts,
                  d: int | None = None, resident_mask: int | None = None) -> None:
        """planes: 8 device pointers/tensors (None = not resident);
        luts: dict {b: tensor/pointer} for b in 3..8."""
        desc = BlockDesc()
        desc.n, desc.k, desc.q = n, k, q
        desc.d = q if d is None else d
        mask = 0
        for p in range(PLANES):
            pp = ptr(planes[p]) if p < len(planes) else None
            desc.plane[p] = pp
            if pp:
                mask |= 1 << p
        desc.resident_mask = mask if resident_mask is None else resident_mask
        for b in range(MAX_BITS + 1):
            desc.lut[b] = ptr(luts.get(b)) if b in luts else None
        _check(self.L.apmoe_table_set_block(self.handle, layer, expert, kind, ctypes.byref(desc)),
               "apmoe_table_set_block", self.L)

    def set_bits(self, layer: int, expert: int, kind: int, q: int) -> None:
        _check(self.L.apmoe_table_set_bits(self.handle, layer, expert, kind, q), "apmoe_table_set_bits", self.L)

    def set_plane(self, layer: int, expert: int, kind: int, p: int, plane, resident: bool) -> None:
        _check(self.L.apmoe_table_set_plane(self.handle, layer, expert, kind, p, ptr(plane), int(resident)),
               "apmoe_table_set_plane", self.L)

    def validate(self) -> int:
        """Status apmoe_table_commit would return (no exception)."""
        return int(self.L.apmoe_table_validate(self.handle))

    def committed_bits(self, layer: int, expert: int, kind: int) -> int:
        q = ctypes.c_int32()
        _check(self.L.apmoe_table_committed_bits(self.handle, layer, expert, kind, ctypes.byref(q)),
               "apmoe_table_committed_bits", self.L)
        return q.value

    def commit(self, ctx: Context, stream=None) -> None:
        _check(self.L.apmoe_table_commit(ctx.handle, self.handle, stream_handle(stream)), "apmoe_table_commit", self.L)

    def close(self):
        if self.handle:
            self.L.apmoe_table_destroy(self.handle)
            self.handle = None

    def __del__(self):  # pragma: no cover
        try:
            self.close()
        except Exception:
            pass


def lut_build(ctx: Context, parent, n: int, levels: dict, stream=None) -> None:
    arr = (ctypes.c_void_p * (MAX_BITS + 1))(*[ptr(levels.get(b)) for b in range(MAX_BITS + 1)])
    _check(ctx.L.apmoe_lut_build(ctx.handle, ptr(parent), n, ctypes.cast(arr, ctypes.c_void_p),
                                 stream_handle(stream)), "apmoe_lut_build", ctx.L)


def tiled_plane_words(n: int, k: int) -> int:
    return int(lib().apmoe_tiled_plane_words(n, k))


def tile_planes(ctx: Context, canonical, n: int, k: int, tiled, stream=None) -> None:
    _check(ctx.L.apmoe_tile_planes(ctx.handle, ptr(canonical), n, k, ptr(tiled), stream_handle(stream)),
           "apmoe_tile_planes", ctx.L)


def pack_planes(ctx: Context, codes, n: int, k: int, planes, stream=None) -> None:
    _check(ctx.L.apmoe_pack_planes(ctx.handle, ptr(codes), n, k, ptr(planes), stream_handle(stream)),
           "apmoe_pack_planes", ctx.L)


def route(ctx: Context, x, w_router, bias, T: int, H: int, E: int, topk: int, renormalize: bool, topk_ids,
          topk_w, counts, offsets, perm, inv_perm, stream=None, n_shared: int = 0) -> None:
    """Top-k routing over E routed experts; with n_shared > 0 each token's row of
    topk_ids / topk_w (stride topk + n_shared) ends with the shared experts
    E .. E + n_shared - 1 at weight 1, and counts / offsets cover E + n_shared experts."""
    _check(ctx.L.apmoe_route(ctx.handle, ptr(x), ptr(w_router), ptr(bias), T, H, E, topk, n_shared, int(renormalize),
                             ptr(topk_ids), ptr(topk_w), ptr(counts), ptr(offsets), ptr(perm), ptr(inv_perm),
                             stream_handle(stream)), "apmoe_route", ctx.L)


def route_workspace(ctx: Context, T: int, E: int, topk: int, n_shared: int = 0) -> int:
    n = ctypes.c_size_t()
    _check(ctx.L.apmoe_route_workspace(ctx.handle, T, E, topk, n_shared, ctypes.byref(n)), "apmoe_route_workspace",
           ctx.L)
    return n.value


def route_stats(ctx: Context, topk_w, perm, offsets, T: int, topk: int, E: int, mass, total, selections,
                stream=None) -> None:
    """Add one routed batch to the routing-statistics accumulators (Eq. 1):
    mass[E] fp64, total[1] fp64, selections[E] int64, all device memory."""
    _check(ctx.L.apmoe_route_stats(ctx.handle, ptr(topk_w), ptr(perm), ptr(offsets), T, topk, E, ptr(mass),
                                   ptr(total), ptr(selections), stream_handle(stream)), "apmoe_route_stats", ctx.L)


def gemm(ctx: Context, table: Table, layer: int, kind: int, inp, gather: bool, perm, offsets, T: int, topk: int,
         out, out_dtype: int, stream=None) -> None:
    _check(ctx.L.apmoe_gemm(ctx.handle, table.handle, layer, kind, ptr(inp), int(gather), ptr(perm), ptr(offsets),
                            T, topk, ptr(out), out_dtype, stream_handle(stream)), "apmoe_gemm", ctx.L)


def gemm_act(ctx: Context, table: Table, layer: int, x, gather: bool, perm, offsets, T: int, topk: int, a,
             stream=None) -> None:
    """gate_up product with SiLU(gate) * up in its epilogue: fp16 a [T*topk][F]."""
    _check(ctx.L.apmoe_gemm_act(ctx.handle, table.handle, layer, ptr(x), int(gather), ptr(perm), ptr(offsets), T,
                                topk, ptr(a), stream_handle(stream)), "apmoe_gemm_act", ctx.L)


def act(ctx: Context, h, R: int, F: int, a, stream=None) -> None:
    _check(ctx.L.apmoe_act(ctx.handle, ptr(h), R, F, ptr(a), stream_handle(stream)), "apmoe_act", ctx.L)


def combine(ctx: Context, y, y_dtype: int, topk_w, inv_perm, T: int, topk: int, H: int, out, stream=None) -> None:
    _check(ctx.L.apmoe_combine(ctx.handle, ptr(y), y_dtype, ptr(topk_w), ptr(inv_perm), T, topk, H, ptr(out),
                               stream_handle(stream)), "apmoe_combine", ctx.L)


def moe_workspace(table: Table, layer: int, T: int, topk: int, n_shared: int = 0) -> int:
    n = ctypes.c_size_t()
    _check(table.L.apmoe_moe_workspace(table.handle, layer, T, topk, n_shared, ctypes.byref(n)), "apmoe_moe_workspace",
           table.L)
    return n.value


def moe_forward(ctx: Context, table: Table, layer: int, x, w_router, bias, T: int, topk: int, renormalize: bool,
                ws, ws_bytes: int, out, stream=None, n_shared: int = 0) -> None:
    """Whole layer; the table's last n_shared experts of the layer are shared ones."""
    _check(ctx.L.apmoe_moe_forward(ctx.handle, table.handle, layer, ptr(x), ptr(w_router), ptr(bias), T, topk,
                                   n_shared,
                                   int(renormalize), ptr(ws), ws_bytes, ptr(out), stream_handle(stream)),
           "apmoe_moe_forward", ctx.L)


NOALLOC_SCRATCH_BYTES = 64 << 20


def moe_forward_noalloc(ctx: Context, table: Table, layer: int, x, w_router, bias, T: int, topk: int,
                        renormalize: bool, out, stream=None, n_shared: int = 0) -> None:
    """The whole layer with the library's static scratch as its workspace (no device
    allocation by the call)."""
    _check(ctx.L.apmoe_moe_forward_noalloc(ctx.handle, table.handle, layer, ptr(x), ptr(w_router), ptr(bias), T,
                                           topk, n_shared, int(renormalize), ptr(out), stream_handle(stream)),
           "apmoe_moe_forward_noalloc", ctx.L)


# --------------------------------------------------------------------------- 8-bit path

_float_ids, _e4m3_types, _f32, _i32 = None, None, None, None


def _load_types() -> None:
    """torch is imported with the first call that takes tensors, not with the package."""
    global _float_ids, _e4m3_types, _f32, _i32
    if _float_ids is None:
        import torch
        _e4m3_types, _f32, _i32 = (torch.float8_e4m3fn, torch.uint8), (torch.float32,), (torch.int32,)
        _float_ids = {torch.float16: F16, torch.bfloat16: BF16, torch.float32: F32}


def _arg(ctx: Context, t, name: str, n: int, types) -> int | None:
    """Pointer of an argument of n elements.  A tensor must have one of the types, be
    contiguous, lie on the context's device and hold at least n elements; None and raw
    pointers (int) are passed on, without these checks."""
    if t is None or isinstance(t, int):
        return t
    if n < 0 or t.dtype not in types or not t.is_contiguous() or t.numel() < n:
        raise ValueError(f"{name}: need {n} contiguous elements of {' / '.join(map(str, types))}, got "
                         f"{tuple(t.shape)} of {t.dtype}{'' if t.is_contiguous() else ', not contiguous'}")
    if t.get_device() != ctx.device:
        raise ValueError(f"{name} is on {t.device}, the context on cuda:{ctx.device}")
    return t.data_ptr()


_raw_stream = None


def _stream_of(ctx: Context, stream) -> int | None:
    global _raw_stream
    if stream is not None:
        return stream.cuda_stream or None
    if _raw_stream is None:
        import torch
        # the handle alone, where torch has it: a Stream object costs as much as the rest of a small call
        _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
            lambda device: torch.cuda.current_stream(device).cuda_stream)
    return _raw_stream(ctx.device) or None


def _types(t, name: str):
    """(number of the type in the C ABI, the type as a tuple) of a floating tensor: the
    arguments whose type a call takes from them must be tensors."""
    _load_types()
    d = _float_ids.get(getattr(t, "dtype", None))
    if d is None:
        raise ValueError(f"{name}: need a tensor of float16, bfloat16 or float32, got {getattr(t, 'dtype', type(t))}")
    return d, (t.dtype,)


def norm(ctx: Context, x, residual, residual_out, gamma, eps: float, T: int, H: int, y, y8=None, y_scale=None,
         stream=None) -> None:
    """Root-mean-square norm of x + residual (residual None: of x).  residual_out gets
    the sum (it may be residual), y the norm in x's type and / or y8, y_scale the norm
    as e4m3 with a scale for each 128 columns.  Types are the tensors' own: float16,
    bfloat16 or float32 (so x and residual must be tensors, no raw pointers)."""
    xt, xtypes = _types(x, "x")
    rt, rtypes = (0, xtypes) if residual is None else _types(residual, "residual")
    n = T * H
    _check(ctx.L.apmoe_norm(ctx.handle, _arg(ctx, x, "x", n, xtypes), xt, _arg(ctx, residual, "residual", n, rtypes),
                            _arg(ctx, residual_out, "residual_out", n, rtypes), rt,
                            _arg(ctx, gamma, "gamma", H, xtypes), eps, T, H, _arg(ctx, y, "y", n, xtypes),
                            _arg(ctx, y8, "y8", n, _e4m3_types), _arg(ctx, y_scale, "y_scale", T * -(-H // 128), _f32),
                            _stream_of(ctx, stream)), "apmoe_norm", ctx.L)


def _fp8_inputs(ctx, x8, x_scale, w8, w_scale, E, rows, n_scale, K, perm, offsets, T, topk, gather):
    _load_types()
    kb, R = -(-K // 128), T * topk
    n = T if gather else R
    f32, i32 = _f32, _i32
    return (_arg(ctx, x8, "x8", n * K, _e4m3_types), _arg(ctx, x_scale, "x_scale", n * kb, f32),
            _arg(ctx, w8, "w8", E * rows * K, _e4m3_types), _arg(ctx, w_scale, "w_scale", E * n_scale * kb, f32),
            _arg(ctx, perm, "perm", R, i32), _arg(ctx, offsets, "offsets", E + 1, i32))


def gemm_fp8(ctx: Context, x8, x_scale, w8, w_scale, E: int, N: int, K: int, gather: bool, perm, offsets, T: int,
             topk: int, out, stream=None) -> None:
    """The experts' product on e4m3 operands with fp32 scales (x_scale by 128 columns,
    w_scale by 128 x 128 block); out is a tensor, whose type is taken.  Dense: E = topk = 1,
    gather False, perm and offsets None."""
    xp, xsp, wp, wsp, pp, op = _fp8_inputs(ctx, x8, x_scale, w8, w_scale, E, N, -(-N // 128), K, perm, offsets, T,
                                           topk, gather)
    dt, types = _types(out, "out")
    _check(ctx.L.apmoe_gemm_fp8(ctx.handle, xp, xsp, wp, wsp, E, N, K, int(gather), pp, op, T, topk,
                                _arg(ctx, out, "out", T * topk * N, types), dt, _stream_of(ctx, stream)),
           "apmoe_gemm_fp8", ctx.L)


def gemm_act_fp8(ctx: Context, x8, x_scale, w8, w_scale, E: int, F: int, K: int, gather: bool, perm, offsets, T: int,
                 topk: int, a8, a_scale, stream=None) -> None:
    """The gate_up product on e4m3 operands with SiLU(gate) * up and the 8-bit output in
    its epilogue: a8 e4m3 [T*topk][F], a_scale fp32 [T*topk][ceil(F/128)]."""
    fb = -(-F // 128)
    xp, xsp, wp, wsp, pp, op = _fp8_inputs(ctx, x8, x_scale, w8, w_scale, E, 2 * F, 2 * fb, K, perm, offsets, T, topk,
                                           gather)
    _check(ctx.L.apmoe_gemm_act_fp8(ctx.handle, xp, xsp, wp, wsp, E, F, K, int(gather), pp, op, T, topk,
                                    _arg(ctx, a8, "a8", T * topk * F, _e4m3_types),
                                    _arg(ctx, a_scale, "a_scale", T * topk * fb, _f32),
                                    _stream_of(ctx, stream)), "apmoe_gemm_act_fp8", ctx.L)


class Fp8Experts:
    """The e4m3 experts of one layer: gate_up [E][2F][H] with scales
    [E][2][ceil(F/128)][ceil(H/128)], down [E][H][F] with scales
    [E][ceil(H/128)][ceil(F/128)] (any shape with that many elements; E, H and F are
    read from gate_up and down).  Holds the tensors, so they live as long as it does."""

    def __init__(self, gate_up, gate_up_scale, down, down_scale):
        _load_types()
        E, H, F = down.shape
        if tuple(gate_up.shape) != (E, 2 * F, H):
            raise ValueError(f"gate_up {tuple(gate_up.shape)} and down {tuple(down.shape)} are not [E][2F][H], [E][H][F]")
        self.E, self.H, self.F = E, H, F
        self.device = down.get_device()
        hb, fb = -(-H // 128), -(-F // 128)
        self.tensors = (gate_up, gate_up_scale, down, down_scale)
        d = Fp8Desc()
        d.E, d.H, d.F = E, H, F
        d.gate_up = _arg(self, gate_up, "gate_up", E * 2 * F * H, _e4m3_types)
        d.gate_up_scale = _arg(self, gate_up_scale, "gate_up_scale", E * 2 * fb * hb, _f32)
        d.down = _arg(self, down, "down", E * H * F, _e4m3_types)
        d.down_scale = _arg(self, down_scale, "down_scale", E * hb * fb, _f32)
        self.desc = d
        self.ref = ctypes.byref(d)


def moe_workspace_fp8(ctx: Context, experts: Fp8Experts, T: int, topk: int, n_shared: int = 0) -> int:
    n = ctypes.c_size_t()
    _check(ctx.L.apmoe_moe_workspace_fp8(ctx.handle, experts.ref, T, topk, n_shared, ctypes.byref(n)),
           "apmoe_moe_workspace_fp8", ctx.L)
    return n.value


def moe_forward_fp8(ctx: Context, experts: Fp8Experts, x, x8, x_scale, w_router, bias, T: int, topk: int,
                    renormalize: bool, ws, out, stream=None, n_shared: int = 0) -> None:
    """Whole layer on e4m3 experts: x fp16 is what the router reads, x8 / x_scale the
    same rows in 8 bits (norm gives both).  ws: a byte tensor of moe_workspace_fp8 bytes."""
    import torch
    if not isinstance(ws, torch.Tensor):
        raise ValueError(f"ws: need a byte tensor, got {type(ws)}")
    if experts.device != ctx.device:
        raise ValueError(f"the experts are on cuda:{experts.device}, the context on cuda:{ctx.device}")
    E, H = experts.E, experts.H
    f16, f32 = (torch.float16,), (torch.float32,)
    _check(ctx.L.apmoe_moe_forward_fp8(ctx.handle, experts.ref, _arg(ctx, x, "x", T * H, f16),
                                       _arg(ctx, x8, "x8", T * H, _e4m3_types),
                                       _arg(ctx, x_scale, "x_scale", T * -(-H // 128), f32),
                                       _arg(ctx, w_router, "w_router", (E - n_shared) * H, f16),
                                       _arg(ctx, bias, "bias", E - n_shared, f32), T, topk, n_shared, int(renormalize),
                                       _arg(ctx, ws, "ws", 0, (torch.uint8,)), ws.numel(),
                                       _arg(ctx, out, "out", T * H, f16), _stream_of(ctx, stream)),
           "apmoe_moe_forward_fp8", ctx.L)


# --------------------------------------------------------------------------- paged key-value cache

_MAX32 = 0x7FFFFFFF


def _int32(**numbers) -> None:
    """ctypes cuts a number to the C ABI's 32 bits, and another one would be taken."""
    for name, n in numbers.items():
        if not -_MAX32 - 1 <= n <= _MAX32:
            raise ValueError(f"{name}={n} does not fit into 32 bits")


class KvCache:
    """A pool of pages of the key-value cache: k and v of n_pages * kv_heads * page *
    head_dim elements (any shape that begins with n_pages), float16, bfloat16, or e4m3
    (float8_e4m3fn or uint8) with float32 scales of n_pages * kv_heads * page elements.
    Holds the tensors, so they live as long as it does."""

    def __init__(self, k, v, page: int, kv_heads: int, head_dim: int, k_scale=None, v_scale=None):
        _load_types()
        e4m3 = k.dtype in _e4m3_types
        if not e4m3 and _float_ids.get(k.dtype) not in (F16, BF16):
            raise ValueError(f"k: need float16, bfloat16 or e4m3, got {k.dtype}")
        if e4m3 and (k_scale is None or v_scale is None):
            raise ValueError("an e4m3 cache needs k_scale and v_scale")
        _int32(n_pages=k.shape[0], page=page, kv_heads=kv_heads, head_dim=head_dim)
        self.n_pages, self.page, self.kv_heads, self.head_dim = k.shape[0], page, kv_heads, head_dim
        self.device = k.get_device()
        self.tensors = (k, v, k_scale, v_scale)
        rows = self.n_pages * kv_heads * page
        types = _e4m3_types if e4m3 else (k.dtype,)
        d = KvCacheDesc()
        d.dtype = E4M3 if e4m3 else _float_ids[k.dtype]
        d.n_pages, d.page, d.kv_heads, d.head_dim = self.n_pages, page, kv_heads, head_dim
        d.k = _arg(self, k, "k", rows * head_dim, types)
        d.v = _arg(self, v, "v", rows * head_dim, types)
        if e4m3:
            d.k_scale = _arg(self, k_scale, "k_scale", rows, _f32)
            d.v_scale = _arg(self, v_scale, "v_scale", rows, _f32)
        self.desc = d
        self.ref = ctypes.byref(d)


class KvBatch:
    """The sequences of a call: pages int32 [B][max_pages], lens int32 [B] (this call's
    tokens included), T rows, q_offsets int32 [B + 1] (None: one row a sequence), max_len
    a bound of the lengths (0: what the pages hold).  Holds the tensors."""

    def __init__(self, pages, lens, T: int, q_offsets=None, max_len: int = 0):
        _load_types()
        if pages.dim() != 2 or pages.shape[0] != lens.numel():
            raise ValueError(f"pages {tuple(pages.shape)} and lens {tuple(lens.shape)} are not [B][max_pages], [B]")
        _int32(B=pages.shape[0], T=T, max_pages=pages.shape[1], max_len=max_len)
        self.B, self.T = pages.shape[0], T
        self.device = pages.get_device()
        self.tensors = (pages, lens, q_offsets)
        d = KvBatchDesc()
        d.B, d.T, d.max_pages, d.max_len = self.B, T, pages.shape[1], max_len
        d.pages = _arg(self, pages, "pages", pages.numel(), _i32)
        d.lens = _arg(self, lens, "lens", self.B, _i32)
        d.q_offsets = _arg(self, q_offsets, "q_offsets", self.B + 1, _i32)
        self.desc = d
        self.ref = ctypes.byref(d)


def _kv_on(ctx: Context, cache: KvCache, batch: KvBatch) -> None:
    if cache.device != ctx.device or batch.device != ctx.device:
        raise ValueError(f"the cache is on cuda:{cache.device}, the batch on cuda:{batch.device}, the context on "
                         f"cuda:{ctx.device}")


def _matrix(ctx: Context, t, name: str, T: int, width: int, types):
    """(pointer, stride) of a 2-dimensional tensor of at least T rows and `width` dense
    columns; rows may be apart."""
    shape, strides = t.shape, t.stride()
    if len(shape) != 2 or shape[0] < T or shape[1] != width or strides[1] != 1 or t.dtype not in types:
        raise ValueError(f"{name}: need [{T}][{width}] of {' / '.join(map(str, types))} with dense rows, got "
                         f"{tuple(shape)} of {t.dtype}, strides {strides}")
    if t.get_device() != ctx.device:
        raise ValueError(f"{name} is on {t.device}, the context on cuda:{ctx.device}")
    return t.data_ptr(), strides[0] if shape[0] > 1 else max(strides[0], width)


def kv_append(ctx: Context, cache: KvCache, batch: KvBatch, q, k, v, q_heads: int, rope, rot: int, interleaved: bool,
              q_out, stream=None) -> None:
    """Position rotation of the new rows' queries and keys (rope float32 [n_pos][rot]: a
    position's cosines, then its sines; None with rot 0), keys and values into the cache.
    q [T][q_heads * D], k, v [T][kv_heads * D], rows may be apart; q_out [T][q_heads * D].
    q and q_out None with q_heads 0."""
    _kv_on(ctx, cache, batch)
    T, D = batch.T, cache.head_dim
    dt, types = _types(k, "k")
    qp, qs = (None, 0) if q is None else _matrix(ctx, q, "q", T, q_heads * D, types)
    kp, ks = _matrix(ctx, k, "k", T, cache.kv_heads * D, types)
    vp, vs = _matrix(ctx, v, "v", T, cache.kv_heads * D, types)
    n_pos = 0
    if rope is not None:
        if rope.dim() != 2 or rope.shape[1] != rot:
            raise ValueError(f"rope: need [positions][{rot}], got {tuple(rope.shape)}")
        n_pos = rope.shape[0]
    if not (0 <= q_heads <= _MAX32 and 0 <= rot <= _MAX32 and n_pos <= _MAX32):
        _int32(q_heads=q_heads, rot=rot, n_pos=n_pos)
    st = ctx.L.apmoe_kv_append(ctx.handle, cache.ref, batch.ref, qp, qs, kp, ks, vp, vs, dt, q_heads,
                               _arg(ctx, rope, "rope", n_pos * rot, _f32), n_pos, rot, 1 if interleaved else 0,
                               _arg(ctx, q_out, "q_out", T * q_heads * D, types), _stream_of(ctx, stream))
    if st:
        _check(st, "apmoe_kv_append", ctx.L)


def attn_workspace(ctx: Context, cache: KvCache, batch: KvBatch, q_heads: int) -> int:
    _int32(q_heads=q_heads)
    n = ctypes.c_size_t()
    _check(ctx.L.apmoe_attn_workspace(ctx.handle, cache.ref, batch.ref, q_heads, ctypes.byref(n)),
           "apmoe_attn_workspace", ctx.L)
    return n.value


_u8 = None


def _attn(fn: str, ctx, cache, batch, q, q_heads, scale, window, sinks, ws, out, out8, out_scale, stream) -> None:
    global _u8
    if _u8 is None:
        import torch
        _u8 = (torch.uint8,)
    if not hasattr(ws, "data_ptr"):
        raise ValueError(f"ws: need a byte tensor, got {type(ws)}")
    _kv_on(ctx, cache, batch)
    if not (0 <= window <= _MAX32 and 0 <= sinks <= _MAX32):
        _int32(window=window, sinks=sinks)
    dt, types = _types(q, "q")
    n = batch.T * q_heads * cache.head_dim
    qp, qs = _matrix(ctx, q, "q", batch.T, q_heads * cache.head_dim, types)
    st = getattr(ctx.L, fn)(ctx.handle, cache.ref, batch.ref, qp, qs, dt, q_heads, scale, window, sinks,
                            _arg(ctx, ws, "ws", 0, _u8), ws.numel(), _arg(ctx, out, "out", n, types),
                            _arg(ctx, out8, "out8", n, _e4m3_types), _arg(ctx, out_scale, "out_scale", n // 128, _f32),
                            _stream_of(ctx, stream))
    if st:
        _check(st, fn, ctx.L)


def attn_decode(ctx: Context, cache: KvCache, batch: KvBatch, q, q_heads: int, scale: float, window: int, sinks: int,
                ws, out, out8=None, out_scale=None, stream=None) -> None:
    """Attention of one new token of each sequence (q [B][q_heads * D]) over its cache;
    window 0: over all of it, else over the last `window` tokens and the first `sinks`.
    out in q's type and / or out8, out_scale (e4m3 rows with a scale for each 128 columns).
    ws: a byte tensor of attn_workspace bytes."""
    _attn("apmoe_attn_decode", ctx, cache, batch, q, q_heads, scale, window, sinks, ws, out, out8, out_scale, stream)


def attn_prefill(ctx: Context, cache: KvCache, batch: KvBatch, q, q_heads: int, scale: float, window: int, sinks: int,
                 ws, out, out8=None, out_scale=None, stream=None) -> None:
    """The same for the new tokens of prompts or of their chunks (q_offsets), each row at its
    own position; their keys and values have been appended before."""
    _attn("apmoe_attn_prefill", ctx, cache, batch, q, q_heads, scale, window, sinks, ws, out, out8, out_scale, stream)


# --------------------------------------------------------------------------- page movement

def _plane_array(planes):
    arr = (ctypes.c_void_p * PLANES)()
    for p, t in enumerate(planes if planes is not None else []):
        if p < PLANES:
            arr[p] = ptr(t)
    return arr


def _event_handle(ev, stream) -> int:
    """Raw hipEvent_t of a torch.cuda.Event (recorded once on `stream` so that the
    handle exists; the library records it again)."""
    ev.record(stream)
    return ev.cuda_event


def page_out(ctx: Context, table: Table, layer: int, expert: int, kind: int, q_new: int, host_planes,
             stream, copy_stream, done_event) -> None:
    """Lower (layer, expert, kind) to q_new and copy planes q_new.. to host_planes[p]
    (8-entry list; pinned tensors).  done_event (torch.cuda.Event) completes once the
    device planes may be freed."""
    _check(ctx.L.apmoe_page_out(ctx.handle, table.handle, layer, expert, kind, q_new, _plane_array(host_planes),
                                stream_handle(stream), stream_handle(copy_stream),
                                _event_handle(done_event, copy_stream)), "apmoe_page_out", ctx.L)


def page_in(ctx: Context, table: Table, layer: int, expert: int, kind: int, q_new: int, host_planes, dev_planes,
            stream, copy_stream, copied_event) -> None:
    """Copy host_planes[p] to dev_planes[p] for the planes above the current bitwidth,
    then raise (layer, expert, kind) to q_new with a commit on `stream` that waits for
    the copies."""
    _check(ctx.L.apmoe_page_in(ctx.handle, table.handle, layer, expert, kind, q_new, _plane_array(host_planes),
                               _plane_array(dev_planes), stream_handle(stream), stream_handle(copy_stream),
                               _event_handle(copied_event, copy_stream)), "apmoe_page_in", ctx.L)
