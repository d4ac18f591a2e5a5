"""ctypes binding of libloraforge.so: the C ABI of include/loraforge.h, same names.

Argument marshalling only: every step of the path runs in the library's CUDA
kernels.  Tensors are torch tensors used as device allocations; their data
pointers are passed through.  There is no fallback: if the shared library is
missing or fails to load, every call raises.
"""
from __future__ import annotations

import ctypes
import os

import numpy as np

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libloraforge.so")

LF_OK = 0
STATUS_NAMES = {0: "LF_OK", 1: "LF_ERR_INVALID_ARG", 2: "LF_ERR_SHAPE", 3: "LF_ERR_BAD_INDEX",
                4: "LF_ERR_WORKSPACE", 5: "LF_ERR_NUMERIC", 6: "LF_ERR_TIMEOUT", 7: "LF_ERR_CUDA",
                8: "LF_ERR_ALIGNMENT"}

# lf_module: int32 d_out, d_in, r, group; int64 B_off, A_off  (32 bytes, natural alignment)
MODULE_DTYPE = np.dtype([("d_out", "<i4"), ("d_in", "<i4"), ("r", "<i4"), ("group", "<i4"),
                         ("B_off", "<i8"), ("A_off", "<i8")], align=True)
assert MODULE_DTYPE.itemsize == 32


# lf_jd_problem: int32 d_out, d_in, rank, first, count; int64 U_off, Vt_off, sigma_off (48 bytes)
JD_PROBLEM_DTYPE = np.dtype([("d_out", "<i4"), ("d_in", "<i4"), ("rank", "<i4"), ("first", "<i4"),
                             ("count", "<i4"), ("U_off", "<i8"), ("Vt_off", "<i8"), ("sigma_off", "<i8")],
                            align=True)
assert JD_PROBLEM_DTYPE.itemsize == 48


class lf_policy(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int32), ("ratio_num", ctypes.c_int32),
                ("ratio_den", ctypes.c_int32), ("floor", ctypes.c_int32)]


def policy_U(num: int, den: int, floor: int = 1) -> lf_policy:
    return lf_policy(0, num, den, floor)


def policy_S(num: int, den: int, floor: int = 1, absolute: bool = False) -> lf_policy:
    """LoRAForge-S (normalised energies), or with absolute=True the variant that ranks
    candidates by sigma^2 (kind 2)."""
    return lf_policy(2 if absolute else 1, num, den, floor)


def policy_E(num: int, den: int, floor: int = 1) -> lf_policy:
    """Energy fraction (kind 3): the smallest rank >= floor keeping num/den of each
    module's spectral energy."""
    return lf_policy(3, num, den, floor)


class lf_phase_time(ctypes.Structure):
    _fields_ = [("name", ctypes.c_char * 32), ("total_ms", ctypes.c_double), ("launches", ctypes.c_int64)]


class lf_slice(ctypes.Structure):
    """One output slice of lf_lora_shrink_expand_slices (mirrors the C struct)."""
    _fields_ = [("d_out", ctypes.c_int32), ("max_rank", ctypes.c_int32), ("y_offset", ctypes.c_int64),
                ("ranks", ctypes.c_void_p), ("off_A", ctypes.c_void_p), ("off_Bt", ctypes.c_void_p),
                ("A_pool", ctypes.c_void_p), ("Bt_pool", ctypes.c_void_p),
                ("pool_elems_A", ctypes.c_int64), ("pool_elems_Bt", ctypes.c_int64)]


class lf_projection(ctypes.Structure):
    """One projection of lf_lora_shrink_expand_projections (mirrors the C struct)."""
    _fields_ = [("x", ctypes.c_void_p), ("y", ctypes.c_void_p), ("d_in", ctypes.c_int32),
                ("reserved", ctypes.c_int32), ("y_ld", ctypes.c_int64), ("slice", lf_slice)]


MAX_PROJECTIONS = 8


class lf_router(ctypes.Structure):
    """Routing of tokens to experts (mirrors the C struct; make_router)."""
    _fields_ = [("n_experts", ctypes.c_int32), ("top_k", ctypes.c_int32), ("score", ctypes.c_int32),
                ("n_groups", ctypes.c_int32), ("top_groups", ctypes.c_int32), ("group_top", ctypes.c_int32),
                ("renorm", ctypes.c_int32), ("weight_scale", ctypes.c_float)]


class lf_mixture_projection(ctypes.Structure):
    """One projection of lf_lora_mixture (mirrors the C struct)."""
    _fields_ = [("x", ctypes.c_void_p), ("base", ctypes.c_void_p), ("y", ctypes.c_void_p), ("d_in", ctypes.c_int32),
                ("reserved", ctypes.c_int32), ("x_ld", ctypes.c_int64), ("y_ld", ctypes.c_int64), ("slice", lf_slice)]


class lf_mixture_grad(ctypes.Structure):
    """One projection of lf_lora_mixture_backward (mirrors the C struct)."""
    _fields_ = [("x", ctypes.c_void_p), ("dy", ctypes.c_void_p), ("dx_base", ctypes.c_void_p), ("dx", ctypes.c_void_p),
                ("d_in", ctypes.c_int32), ("reserved", ctypes.c_int32), ("x_ld", ctypes.c_int64),
                ("dy_ld", ctypes.c_int64), ("dx_ld", ctypes.c_int64), ("slice", lf_slice)]


class lf_w4_projection(ctypes.Structure):
    """One projection of lf_w4_projections (mirrors the C struct)."""
    _fields_ = [("x", ctypes.c_void_p), ("y", ctypes.c_void_p), ("q", ctypes.c_void_p), ("scales", ctypes.c_void_p),
                ("zeros", ctypes.c_void_p), ("bias", ctypes.c_void_p), ("d_in", ctypes.c_int32),
                ("d_out", ctypes.c_int32), ("group", ctypes.c_int32), ("reserved", ctypes.c_int32),
                ("x_ld", ctypes.c_int64), ("y_ld", ctypes.c_int64)]


ROUTER_MAX_EXPERTS = 1024
ROUTER_MAX_K = 16
# element types of logits and weight matrices
LF_F32, LF_BF16, LF_F16 = 0, 1, 2
_TYPE_CODES: dict = {}


def type_code(dtype) -> int:
    """LF_F32 / LF_BF16 / LF_F16 of a torch dtype."""
    if not _TYPE_CODES:
        import torch
        _TYPE_CODES.update({torch.float32: LF_F32, torch.bfloat16: LF_BF16, torch.float16: LF_F16})
    code = _TYPE_CODES.get(dtype)
    if code is None:
        raise ValueError(f"float32, bfloat16 or float16 expected, got {dtype}")
    return code


class LFError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {STATUS_NAMES.get(status, status)}")


_lib = None
_P = ctypes.c_void_p
_I32 = ctypes.c_int32
_I64 = ctypes.c_int64
_SZ = ctypes.c_size_t


def lib() -> ctypes.CDLL:
    """Load libloraforge.so (raises OSError if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise OSError(f"libloraforge.so not built (expected at {LIB_PATH}); "
                          "run python -m post_hoc_rank_b200.build")
        L = ctypes.CDLL(LIB_PATH)
        L.lf_rank_stride.argtypes = [_P, _I32]; L.lf_rank_stride.restype = _I32
        L.lf_tsqr_workspace_size.argtypes = [_P, _I32]; L.lf_tsqr_workspace_size.restype = _SZ
        L.lf_tsqr_batched.argtypes = [_P, _I32, _P, _P, _P, _P, _P, _P, _P, _P, _SZ, _P]
        L.lf_tsqr_batched.restype = ctypes.c_int
        L.lf_select_workspace_size.argtypes = [_P, _I32]; L.lf_select_workspace_size.restype = _SZ
        L.lf_select_ranks.argtypes = [_P, _I32, lf_policy, _P, _P, _P, _P, _P, _SZ, _P]
        L.lf_select_ranks.restype = ctypes.c_int
        L.lf_export_workspace_size.argtypes = [_P, _I32]; L.lf_export_workspace_size.restype = _SZ
        L.lf_export_pool_bound.argtypes = [_P, _I32, lf_policy, _P, _P]; L.lf_export_pool_bound.restype = None
        L.lf_truncate_export.argtypes = [_P, _I32, lf_policy, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P,
                                         _P, _P, _P, _P, _I64, _I64, _P, _SZ, _P]
        L.lf_truncate_export.restype = ctypes.c_int
        L.lf_apply_workspace_size.argtypes = [_I32, _I32]; L.lf_apply_workspace_size.restype = _SZ
        L.lf_lora_shrink_expand.argtypes = [_I32, _I32, _I32, _P, _P, _P, _I32, _P, _P, _P, _P, _P,
                                            _I64, _I64, ctypes.c_float, _P, _P, _SZ, _P]
        L.lf_lora_shrink_expand.restype = ctypes.c_int
        L.lf_apply_slices_workspace_size.argtypes = [_I32, _I32, _I32]
        L.lf_apply_slices_workspace_size.restype = _SZ
        L.lf_lora_shrink_expand_slices.argtypes = [_I32, _I32, _P, _P, _I64, _P, _I32, _P, _I32,
                                                   ctypes.c_float, _P, _P, _P, _SZ, _P]
        L.lf_lora_shrink_expand_slices.restype = ctypes.c_int
        L.lf_lora_sigma_sandwich.argtypes = [_I32, _I32, _I32, _P, _P, _P, _I32, _I32, _P, _P, _P, _I32,
                                             ctypes.c_float, _P, _SZ, _P]
        L.lf_lora_sigma_sandwich.restype = ctypes.c_int
        L.lf_route_tokens.argtypes = [_I32, _P, _I32, _P, _SZ, _P]; L.lf_route_tokens.restype = ctypes.c_int
        L.lf_lora_shrink_expand_slices_routed.argtypes = [_I32, _I32, _P, _P, _I64, _P, _I32, _P, _I32,
                                                          ctypes.c_float, _P, _P, _SZ, _P]
        L.lf_lora_shrink_expand_slices_routed.restype = ctypes.c_int
        L.lf_lora_shrink_expand_projections.argtypes = [_I32, _P, _I32, _P, _I32, ctypes.c_float, _P, _P, _SZ, _P]
        L.lf_lora_shrink_expand_projections.restype = ctypes.c_int
        L.lf_jd_workspace_size.argtypes = [_P, _I32, _P, _I32, _P, _I32]; L.lf_jd_workspace_size.restype = _SZ
        L.lf_jd_full.argtypes = [_P, _I32, _P, _I32, _P, _I32, _P, _P, _P, _I32, _P, _P, _P, _P, _SZ, _P]
        L.lf_jd_full.restype = ctypes.c_int
        L.lf_lora_shrink_expand_noalloc.argtypes = [_I32, _I32, _I32, _P, _P, _P, _I32, _P, _P, _P, _P, _P,
                                                    _I64, _I64, ctypes.c_float, _P, _P]
        L.lf_lora_shrink_expand_noalloc.restype = ctypes.c_int
        L.lf_check_bounded_wait.argtypes = [_I32, _P]; L.lf_check_bounded_wait.restype = ctypes.c_int
        L.lf_pool_workspace_size.argtypes = [_I32, _I32, _P, _P, _I32]; L.lf_pool_workspace_size.restype = _SZ
        L.lf_pool_subspace.argtypes = [_I32, _I32, _P, _P, _I32, _P, _I32, _I32, _P, _P, _P, _P, _P, _P, _SZ, _P]
        L.lf_pool_subspace.restype = ctypes.c_int
        _F = ctypes.c_float
        L.lf_route_experts.argtypes = [_I32, _P, _P, _I32, _I64, _P, _P, _P, _P, _P]
        L.lf_route_experts.restype = ctypes.c_int
        L.lf_route_experts_backward.argtypes = [_I32, _P, _P, _I32, _I64, _P, _P, _P, _I64, _P]
        L.lf_route_experts_backward.restype = ctypes.c_int
        for f in (L.lf_lora_mixture_workspace_size, L.lf_lora_mixture_backward_workspace_size):
            f.argtypes = [_I32, _I32, _I32, _P, _I32]
            f.restype = _SZ
        L.lf_lora_mixture.argtypes = [_I32, _I32, _P, _P, _I32, _P, _I32, _F, _P, _P, _SZ, _P]
        L.lf_lora_mixture.restype = ctypes.c_int
        L.lf_lora_mixture_backward.argtypes = [_I32, _I32, _P, _P, _I32, _P, _I32, _F, _P, _P, _P, _SZ, _P]
        L.lf_lora_mixture_backward.restype = ctypes.c_int
        L.lf_w4_quantize.argtypes = [_P, _I32, _I32, _I32, _I32, _P, _P, _P, _P]; L.lf_w4_quantize.restype = ctypes.c_int
        L.lf_w4_dequantize.argtypes = [_P, _P, _P, _I32, _I32, _I32, _P, _I32, _P]
        L.lf_w4_dequantize.restype = ctypes.c_int
        L.lf_w4_projections.argtypes = [_I32, _P, _I32, _P]; L.lf_w4_projections.restype = ctypes.c_int
        L.lf_status_string.argtypes = [ctypes.c_int]; L.lf_status_string.restype = ctypes.c_char_p
        L.lf_get_device_status.argtypes = [_P]; L.lf_get_device_status.restype = ctypes.c_int
        L.lf_profile_enable.argtypes = [ctypes.c_int]; L.lf_profile_enable.restype = None
        L.lf_profile_reset.argtypes = []; L.lf_profile_reset.restype = None
        L.lf_profile_read.argtypes = [_P, _I32]; L.lf_profile_read.restype = _I32
        L.lf_launch_count.argtypes = []; L.lf_launch_count.restype = _I64
        _lib = L
    return _lib


def exported_symbols() -> list[str]:
    return ["lf_rank_stride", "lf_tsqr_workspace_size", "lf_tsqr_batched", "lf_select_workspace_size",
            "lf_select_ranks", "lf_export_workspace_size", "lf_export_pool_bound", "lf_truncate_export",
            "lf_apply_workspace_size", "lf_lora_shrink_expand", "lf_status_string", "lf_get_device_status",
            "lf_profile_enable", "lf_profile_reset", "lf_profile_read", "lf_launch_count",
            "lf_lora_shrink_expand_noalloc", "lf_apply_slices_workspace_size", "lf_lora_shrink_expand_slices",
            "lf_lora_sigma_sandwich", "lf_jd_workspace_size", "lf_jd_full", "lf_route_tokens",
            "lf_lora_shrink_expand_slices_routed", "lf_check_bounded_wait", "lf_pool_workspace_size",
            "lf_pool_subspace", "lf_lora_shrink_expand_projections", "lf_route_experts", "lf_route_experts_backward",
            "lf_lora_mixture_workspace_size", "lf_lora_mixture_backward_workspace_size", "lf_lora_mixture", "lf_lora_mixture_backward", "lf_w4_quantize",
            "lf_w4_dequantize", "lf_w4_projections"]

# Limits of lf_lora_shrink_expand_noalloc (its scratch is a fixed array in the library).
NOALLOC_MAX_TOKENS = 16384
NOALLOC_MAX_ADAPTERS = 4096


def _ptr(t) -> int | None:
    if t is None:
        return None
    if hasattr(t, "data_ptr"):
        return t.data_ptr()
    if isinstance(t, int):
        return t
    return t.ctypes.data


def _mods_ptr(mods: np.ndarray):
    assert mods.dtype == MODULE_DTYPE and mods.flags["C_CONTIGUOUS"]
    return mods.ctypes.data, int(mods.shape[0])


_CUDA_NOW: list = []


def _cuda_now():
    """[current device, handle of a device's current stream].  torch.cuda.current_stream() builds a
    Stream object to ask for its handle (3 us a call); torch's own calls under it give the handle
    alone, and where a version of torch lacks them the public ones are taken."""
    if not _CUDA_NOW:
        import torch
        device = getattr(torch._C, "_cuda_getDevice", None)
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        _CUDA_NOW.extend((device or torch.cuda.current_device,
                          raw or (lambda index: torch.cuda.current_stream(index).cuda_stream)))
    return _CUDA_NOW


def current_device() -> int:
    return _cuda_now()[0]()


def _stream(stream) -> int | None:
    if stream is None:
        return _cuda_now()[1](current_device())
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(st: int, where: str) -> int:
    if st != LF_OK:
        raise LFError(st, where)
    return st


def lf_rank_stride(mods: np.ndarray) -> int:
    p, n = _mods_ptr(mods)
    return lib().lf_rank_stride(p, n)


def lf_tsqr_workspace_size(mods: np.ndarray) -> int:
    p, n = _mods_ptr(mods)
    return lib().lf_tsqr_workspace_size(p, n)


def lf_tsqr_batched(mods, B_base, A_base, R_B, R_A, sigma, U, V, ws, stream=None, check=True) -> int:
    p, n = _mods_ptr(mods)
    st = lib().lf_tsqr_batched(p, n, _ptr(B_base), _ptr(A_base), _ptr(R_B), _ptr(R_A), _ptr(sigma),
                               _ptr(U), _ptr(V), _ptr(ws), ws.numel() if ws is not None else 0, _stream(stream))
    return _check(st, "lf_tsqr_batched") if check else st


def lf_select_workspace_size(mods: np.ndarray) -> int:
    p, n = _mods_ptr(mods)
    return lib().lf_select_workspace_size(p, n)


def lf_select_ranks(mods, pol: lf_policy, sigma, ranks, off_A, off_Bt, ws, stream=None, check=True) -> int:
    p, n = _mods_ptr(mods)
    st = lib().lf_select_ranks(p, n, pol, _ptr(sigma), _ptr(ranks), _ptr(off_A), _ptr(off_Bt), _ptr(ws),
                               ws.numel() if ws is not None else 0, _stream(stream))
    return _check(st, "lf_select_ranks") if check else st


def lf_export_workspace_size(mods: np.ndarray) -> int:
    p, n = _mods_ptr(mods)
    return lib().lf_export_workspace_size(p, n)


def lf_export_pool_bound(mods: np.ndarray, pol: lf_policy) -> tuple[int, int]:
    p, n = _mods_ptr(mods)
    a, b = ctypes.c_int64(0), ctypes.c_int64(0)
    lib().lf_export_pool_bound(p, n, pol, ctypes.addressof(a), ctypes.addressof(b))
    return a.value, b.value


def lf_truncate_export(mods, pol, B_base, A_base, R_B, R_A, sigma, U, V, ranks, off_A, off_Bt,
                       A_pool, Bt_pool, A_pool_bf16, Bt_pool_bf16, ws, stream=None, check=True) -> int:
    p, n = _mods_ptr(mods)
    st = lib().lf_truncate_export(p, n, pol, _ptr(B_base), _ptr(A_base), _ptr(R_B), _ptr(R_A), _ptr(sigma),
                                  _ptr(U), _ptr(V), _ptr(ranks), _ptr(off_A), _ptr(off_Bt), _ptr(A_pool),
                                  _ptr(Bt_pool), _ptr(A_pool_bf16), _ptr(Bt_pool_bf16), A_pool.numel(),
                                  Bt_pool.numel(), _ptr(ws), ws.numel() if ws is not None else 0,
                                  _stream(stream))
    return _check(st, "lf_truncate_export") if check else st


def lf_apply_workspace_size(T: int, n_adapters: int) -> int:
    return lib().lf_apply_workspace_size(T, n_adapters)


def lf_lora_shrink_expand(x, y, ids, n_adapters, ranks, off_A, off_Bt, A_pool, Bt_pool, scale, ws,
                          seg_out=None, stream=None, check=True) -> int:
    T, d_in = x.shape
    d_out = y.shape[1]
    st = lib().lf_lora_shrink_expand(T, d_in, d_out, _ptr(x), _ptr(y), _ptr(ids), n_adapters, _ptr(ranks),
                                     _ptr(off_A), _ptr(off_Bt), _ptr(A_pool), _ptr(Bt_pool), A_pool.numel(),
                                     Bt_pool.numel(), float(scale),
                                     _ptr(seg_out), _ptr(ws), ws.numel() if ws is not None else 0,
                                     _stream(stream))
    return _check(st, "lf_lora_shrink_expand") if check else st


def lf_apply_slices_workspace_size(T: int, n_adapters: int, n_slices: int) -> int:
    return lib().lf_apply_slices_workspace_size(T, n_adapters, n_slices)


def make_slice(d_out, y_offset, ranks, off_A, off_Bt, A_pool, Bt_pool, max_rank=0) -> lf_slice:
    """lf_slice from device tensors (ranks int32, offsets int64, pools bf16); max_rank: 0, or
    an upper bound of the slice's ranks the caller knows.  It holds the tensors, as what is made
    of it does."""
    sl = lf_slice(int(d_out), int(max_rank), int(y_offset), _ptr(ranks), _ptr(off_A), _ptr(off_Bt), _ptr(A_pool),
                  _ptr(Bt_pool), A_pool.numel(), Bt_pool.numel())
    sl.tables = (ranks, off_A, off_Bt, A_pool, Bt_pool)
    return sl


_TABLE_TYPES: list = []


def _adapters(sl: lf_slice):
    """Number of adapters that the tables of a slice hold (None where they are raw addresses),
    checked once per slice: a wrong type or length is read out of range on the device."""
    n = getattr(sl, "adapters", False)
    if n is not False:
        return n
    if not _TABLE_TYPES:
        import torch
        _TABLE_TYPES.extend((torch.int32, torch.int64, torch.int64, torch.bfloat16, torch.bfloat16))
    n = None
    for t, dtype in zip(getattr(sl, "tables", ()), _TABLE_TYPES):
        if t is None or t.__class__ is int:
            continue
        if t.dtype is not dtype or not t.is_contiguous():
            raise ValueError("contiguous int32 ranks, int64 offsets and bfloat16 pools expected, "
                             f"got {t.dtype} with strides {t.stride()}")
        if dtype is not _TABLE_TYPES[3] and (n is None or t.numel() < n):
            n = t.numel()
    sl.adapters = n
    return n


def _cover(projections, n_adapters: int):
    """Checks that every slice's tables hold n_adapters entries (read whatever the ids name)."""
    for p in getattr(projections, "entries", projections):
        n = getattr(p, "adapters", None)
        if n is not None and n < n_adapters:
            raise ValueError(f"the call names {n_adapters} adapters, the tables of a slice hold {n}")


def _one_device(x, others):
    """x's device, which the other tensors (None: absent) must share."""
    dev = x.device
    for t in others:
        if t is not None and getattr(t, "device", dev) != dev:   # raw addresses pass
            raise ValueError(f"every tensor must live on x's device, {dev}, got {t.device}")
    return dev


def lf_lora_shrink_expand_slices(x, y, ids, n_adapters, slices, scale, ws, adapter_scale=None, seg_out=None,
                                 stream=None, check=True) -> int:
    """slices: list of lf_slice (make_slice); y: T x y_ld bf16 holding every slice."""
    T, d_in = x.shape
    arr = (lf_slice * len(slices))(*slices)
    st = lib().lf_lora_shrink_expand_slices(T, d_in, _ptr(x), _ptr(y), y.shape[1], _ptr(ids), n_adapters, arr,
                                            len(slices), float(scale), _ptr(adapter_scale), _ptr(seg_out), _ptr(ws),
                                            ws.numel() if ws is not None else 0, _stream(stream))
    return _check(st, "lf_lora_shrink_expand_slices") if check else st


def lf_route_tokens(ids, n_adapters, ws, stream=None, check=True) -> int:
    """Routing of a token batch into `ws`, for routed calls on the same batch."""
    st = lib().lf_route_tokens(int(ids.numel()), _ptr(ids), n_adapters, _ptr(ws), ws.numel() if ws is not None else 0,
                               _stream(stream))
    return _check(st, "lf_route_tokens") if check else st


def lf_lora_shrink_expand_slices_routed(x, y, ids, n_adapters, slices, scale, ws, adapter_scale=None, stream=None,
                                        check=True) -> int:
    """lf_lora_shrink_expand_slices on a workspace that already holds this batch's routing."""
    T, d_in = x.shape
    arr = (lf_slice * len(slices))(*slices)
    st = lib().lf_lora_shrink_expand_slices_routed(T, d_in, _ptr(x), _ptr(y), y.shape[1], _ptr(ids), n_adapters, arr,
                                                   len(slices), float(scale), _ptr(adapter_scale), _ptr(ws),
                                                   ws.numel() if ws is not None else 0, _stream(stream))
    return _check(st, "lf_lora_shrink_expand_slices_routed") if check else st


def make_projection(x, y, sl: lf_slice) -> lf_projection:
    """lf_projection from device tensors: x T x d_in bf16, y T x y_ld bf16, and the slice
    (make_slice) saying where in y and with which factors."""
    p = lf_projection(_ptr(x), _ptr(y), int(x.shape[1]), 0, int(y.shape[1]), sl)
    p.holds = (x, y, sl)
    return p


def lf_lora_shrink_expand_projections(T, ids, n_adapters, projections, scale, ws=None, adapter_scale=None,
                                      stream=None, check=True) -> int:
    """Up to MAX_PROJECTIONS projections (make_projection) of one token batch in one call."""
    arr = _array(lf_projection, projections)
    st = lib().lf_lora_shrink_expand_projections(int(T), _ptr(ids), n_adapters, arr, len(projections), float(scale),
                                                 _ptr(adapter_scale), _ptr(ws), ws.numel() if ws is not None else 0,
                                                 _stream(stream))
    return _check(st, "lf_lora_shrink_expand_projections") if check else st


def lf_lora_sigma_sandwich(x, y, ids, n_adapters, Vt, Ut, sigma, diagonal, scale, ws, stream=None,
                           check=True) -> int:
    """Sigma-sandwich serving: y += scale * U (Sigma_a (V^T x)); Vt rank x d_in, Ut rank x d_out
    (bf16), sigma n_adapters x rank (diagonal) or n_adapters x rank x rank (fp32)."""
    T, d_in = x.shape
    d_out = y.shape[1]
    st = lib().lf_lora_sigma_sandwich(T, d_in, d_out, _ptr(x), _ptr(y), _ptr(ids), n_adapters, Vt.shape[0],
                                      _ptr(Vt), _ptr(Ut), _ptr(sigma), 1 if diagonal else 0, float(scale), _ptr(ws),
                                      ws.numel() if ws is not None else 0, _stream(stream))
    return _check(st, "lf_lora_sigma_sandwich") if check else st


_ARRAY_TYPES: dict = {}


def _array(kind, items):
    """C array of the structures in `items` (itself, if it is one already).  It holds them: a
    structure in an array is a copy of the bytes, without the tensors that the item holds."""
    if isinstance(items, ctypes.Array):
        if items._type_ is not kind:
            raise TypeError(f"an array of {kind.__name__} expected, got {items._type_.__name__}")
        return items
    key = (kind, len(items))
    typ = _ARRAY_TYPES.get(key)
    if typ is None:
        typ = _ARRAY_TYPES[key] = kind * len(items)
    arr = typ(*items)
    arr.entries = tuple(items)
    return arr


def _rows_device(items):
    """(rows, device) that the descriptions in `items` (make_*, or an array that _array made) share."""
    items = getattr(items, "entries", items)
    first = None
    for p in items:
        have = getattr(p, "rows", None), getattr(p, "device", None)
        if have[0] is None or have != (first or have):
            raise ValueError("projections of one call must come from make_* and share their rows and device, "
                             f"got {have} beside {first}")
        first = have
    if first is None:
        raise ValueError("one projection or more expected")
    return first


def _rows(t, what: str) -> tuple[int, int, int]:
    """(rows, columns, row stride) of a 2-D bf16 tensor whose columns lie side by side."""
    shape = t.shape
    if len(shape) != 2 or (_TYPE_CODES.get(t.dtype) if _TYPE_CODES else type_code(t.dtype)) != LF_BF16:
        raise ValueError(f"{what}: a 2-D bfloat16 tensor expected")
    n, c = shape
    ld, step = t.stride()
    if step != 1 and n > 0 and c > 1:
        raise ValueError(f"{what}: a unit column stride expected")
    return n, c, (ld if n > 1 else (c + 7) & ~7)   # a single row has no stride: any that is allowed


def make_router(n_experts: int, top_k: int, score: str = "softmax", n_groups: int = 1, top_groups: int = 1,
                group_top: int = 1, renorm: bool = True, weight_scale: float = 1.0) -> lf_router:
    """lf_router; score "softmax" or "sigmoid"."""
    codes = {"softmax": 0, "sigmoid": 1}
    if score not in codes:
        raise ValueError(f"score must be softmax or sigmoid, got {score!r}")
    return lf_router(int(n_experts), int(top_k), codes[score], int(n_groups), int(top_groups), int(group_top),
                     1 if renorm else 0, float(weight_scale))


def _logits_ld(t) -> int:
    return t.stride(0) if t.shape[0] > 1 else max(t.stride(0), t.shape[1])


def lf_route_experts(logits, router: lf_router, bias, ids, weights, counts=None, stream=None, check=True) -> int:
    """Routing of T tokens (logits: T rows of fp32, bf16 or fp16, unit column stride): ids T x top_k
    int32, weights T x top_k fp32, counts (nullable) n_experts int32."""
    st = lib().lf_route_experts(logits.shape[0], ctypes.byref(router), _ptr(logits), type_code(logits.dtype),
                                _logits_ld(logits), _ptr(bias), _ptr(ids), _ptr(weights), _ptr(counts), _stream(stream))
    return _check(st, "lf_route_experts") if check else st


def lf_route_experts_backward(logits, router: lf_router, ids, grad_weights, grad_logits, stream=None,
                              check=True) -> int:
    """grad_logits (the logits' type, unit column stride) from grad_weights at the forward's ids."""
    st = lib().lf_route_experts_backward(logits.shape[0], ctypes.byref(router), _ptr(logits), type_code(logits.dtype),
                                         _logits_ld(logits), _ptr(ids), _ptr(grad_weights), _ptr(grad_logits),
                                         _logits_ld(grad_logits), _stream(stream))
    return _check(st, "lf_route_experts_backward") if check else st


def make_mixture_projection(x, y, sl: lf_slice, base=None) -> lf_mixture_projection:
    """lf_mixture_projection from device tensors: x T x d_in bf16, y T x y_ld bf16 (rows may be
    strided), base None (zeros) or laid out like y (y itself: in place)."""
    T, d_in, x_ld = _rows(x, "x")
    n, cols, y_ld = _rows(y, "y")
    if n != T:
        raise ValueError("x and y must have the same rows")
    if sl.y_offset + sl.d_out > cols:
        raise ValueError(f"the slice ends at column {sl.y_offset + sl.d_out}, y has {cols}")
    if base is not None and base is not y and (_rows(base, "base")[2] != y_ld or base.shape != y.shape):
        raise ValueError("base must have y's shape and row stride")
    p = lf_mixture_projection(x.data_ptr(), _ptr(base), y.data_ptr(), d_in, 0, x_ld, y_ld, sl)
    p.holds = (x, y, base, sl)
    p.rows, p.device, p.adapters = T, _one_device(x, (y, base, *getattr(sl, "tables", ()))), _adapters(sl)
    return p


def make_mixture_grad(x, dy, dx, sl: lf_slice, dx_base=None) -> lf_mixture_grad:
    """lf_mixture_grad from device tensors: x and dx T x d_in, dy T x dy_ld (bf16, rows may be
    strided); dx None = not wanted, dx_base None (zeros) or laid out like dx."""
    T, d_in, x_ld = _rows(x, "x")
    n, cols, dy_ld = _rows(dy, "dy")
    if n != T:
        raise ValueError("x and dy must have the same rows")
    if sl.y_offset + sl.d_out > cols:
        raise ValueError(f"the slice ends at column {sl.y_offset + sl.d_out}, dy has {cols}")
    dx_ld = 0
    if dx is not None:
        if dx.shape != x.shape:
            raise ValueError("dx must have x's shape")
        dx_ld = _rows(dx, "dx")[2]
    if dx_base is not None and (dx is None or _rows(dx_base, "dx_base")[2] != dx_ld or dx_base.shape != dx.shape):
        raise ValueError("dx_base must have dx's shape and row stride")
    p = lf_mixture_grad(x.data_ptr(), dy.data_ptr(), _ptr(dx_base), _ptr(dx), d_in, 0, x_ld, dy_ld, dx_ld, sl)
    p.holds = (x, dy, dx, dx_base, sl)
    p.rows, p.device, p.adapters = T, _one_device(x, (dy, dx, dx_base, *getattr(sl, "tables", ()))), _adapters(sl)
    return p


def lf_lora_mixture_workspace_size(T: int, top_k: int, n_adapters: int, projections) -> int:
    arr = _array(lf_mixture_projection, projections)
    return lib().lf_lora_mixture_workspace_size(T, top_k, n_adapters, arr, len(projections))


def lf_lora_mixture_backward_workspace_size(T: int, top_k: int, n_adapters: int, grads) -> int:
    arr = _array(lf_mixture_grad, grads)
    return lib().lf_lora_mixture_backward_workspace_size(T, top_k, n_adapters, arr, len(grads))


def lf_lora_mixture(ids, weights, n_adapters, projections, scale, ws=None, adapter_scale=None, stream=None,
                    check=True) -> int:
    """Routed side path: ids T x top_k int32, weights T x top_k fp32 or None, up to MAX_PROJECTIONS
    projections (make_mixture_projection)."""
    T, K = ids.shape
    _cover(projections, n_adapters)
    arr = _array(lf_mixture_projection, projections)
    st = lib().lf_lora_mixture(T, K, _ptr(ids), _ptr(weights), n_adapters, arr, len(projections), float(scale),
                               _ptr(adapter_scale), _ptr(ws), ws.numel() if ws is not None else 0, _stream(stream))
    return _check(st, "lf_lora_mixture") if check else st


def lf_lora_mixture_backward(ids, weights, n_adapters, grads, scale, grad_weights=None, ws=None, adapter_scale=None,
                             stream=None, check=True) -> int:
    """Gradients of lf_lora_mixture for x (per projection, make_mixture_grad) and the weights."""
    T, K = ids.shape
    _cover(grads, n_adapters)
    arr = _array(lf_mixture_grad, grads)
    st = lib().lf_lora_mixture_backward(T, K, _ptr(ids), _ptr(weights), n_adapters, arr, len(grads), float(scale),
                                        _ptr(adapter_scale), _ptr(grad_weights), _ptr(ws),
                                        ws.numel() if ws is not None else 0, _stream(stream))
    return _check(st, "lf_lora_mixture_backward") if check else st


def lf_w4_quantize(W, group: int, q, scales, zeros=None, stream=None, check=True) -> int:
    """4-bit codes q (d_out x d_in / 2 uint8), scales (d_out x ng bf16) and, unless None, zero
    points (d_out x ng uint8) of W (d_out x d_in fp32, bf16 or fp16)."""
    d_out, d_in = W.shape
    st = lib().lf_w4_quantize(_ptr(W), type_code(W.dtype), d_out, d_in, int(group), _ptr(q), _ptr(scales), _ptr(zeros),
                              _stream(stream))
    return _check(st, "lf_w4_quantize") if check else st


def lf_w4_dequantize(q, scales, zeros, group: int, W, stream=None, check=True) -> int:
    """W (d_out x d_in fp32, bf16 or fp16) = (q - zeros) * scales."""
    d_out, d_in = W.shape
    code = type_code(W.dtype)
    _w4_tables(q, scales, zeros, d_out, d_in, int(group))
    st = lib().lf_w4_dequantize(_ptr(q), _ptr(scales), _ptr(zeros), d_out, d_in, int(group), _ptr(W), code,
                                _stream(stream))
    return _check(st, "lf_w4_dequantize") if check else st


def _w4_tables(q, scales, zeros, d_out: int, d_in: int, group: int):
    """Checks that the tables of a 4-bit matrix have the sizes its kernels read."""
    n = d_out * (-(-d_in // group))
    if q.element_size() != 1 or q.numel() != d_out * (d_in // 2) or not q.is_contiguous():
        raise ValueError("q: a contiguous d_out x d_in / 2 uint8 tensor expected")
    if scales.numel() != n or _TYPE_CODES.get(scales.dtype) != LF_BF16 or not scales.is_contiguous():
        raise ValueError("scales: a contiguous d_out x ceil(d_in / group) bfloat16 tensor expected")
    if zeros is not None and (zeros.numel() != n or zeros.element_size() != 1 or not zeros.is_contiguous()):
        raise ValueError("zeros: a contiguous d_out x ceil(d_in / group) uint8 tensor expected")


def make_w4_projection(x, y, q, scales, group: int, zeros=None, bias=None) -> lf_w4_projection:
    """lf_w4_projection from device tensors: x T x d_in and y T x d_out bf16 (rows may be strided),
    the 4-bit weights as lf_w4_quantize lays them out, bias d_out bf16 or None."""
    T, d_in, x_ld = _rows(x, "x")
    n, cols, y_ld = _rows(y, "y")
    d_out, half = q.shape
    if n != T or d_in != 2 * half or cols < d_out:
        raise ValueError(f"shapes do not fit: x {tuple(x.shape)}, y {tuple(y.shape)}, q {tuple(q.shape)}")
    _w4_tables(q, scales, zeros, d_out, d_in, group)
    if bias is not None and (bias.numel() != d_out or _TYPE_CODES.get(bias.dtype) != LF_BF16 or not bias.is_contiguous()):
        raise ValueError("bias: d_out contiguous bfloat16 values expected")
    p = lf_w4_projection(x.data_ptr(), y.data_ptr(), q.data_ptr(), scales.data_ptr(),
                         0 if zeros is None else zeros.data_ptr(), 0 if bias is None else bias.data_ptr(), d_in, d_out,
                         group, 0, x_ld, y_ld)
    p.holds = (x, y, q, scales, zeros, bias)
    p.rows, p.device = T, _one_device(x, (y, q, scales, zeros, bias))
    return p


def lf_w4_projections(T: int, projections, stream=None, check=True) -> int:
    """y = x W0^T + bias for up to MAX_PROJECTIONS projections (make_w4_projection) of T tokens."""
    arr = _array(lf_w4_projection, projections)
    st = lib().lf_w4_projections(int(T), arr, len(projections), _stream(stream))
    return _check(st, "lf_w4_projections") if check else st


def _jd_tables(mods, members, probs):
    pm, nm = _mods_ptr(mods)
    assert members.dtype == np.int32 and members.flags["C_CONTIGUOUS"]
    assert probs.dtype == JD_PROBLEM_DTYPE and probs.flags["C_CONTIGUOUS"]
    return pm, nm, members.ctypes.data, int(members.shape[0]), probs.ctypes.data, int(probs.shape[0])


def lf_jd_workspace_size(mods: np.ndarray, members: np.ndarray, probs: np.ndarray) -> int:
    return lib().lf_jd_workspace_size(*_jd_tables(mods, members, probs))


def lf_pool_workspace_size(side, ranks, offs, d) -> int:
    rk = np.ascontiguousarray(ranks, dtype=np.int32)
    of = np.ascontiguousarray(offs, dtype=np.int64)
    return lib().lf_pool_workspace_size(int(side), len(rk), rk.ctypes.data, of.ctypes.data, int(d))


def lf_pool_subspace(side, ranks, offs, d, base, num, den, k, sigma, basis, coef, resid, ws, stream=None,
                     check=True) -> int:
    """Pool-wide subspace of stacked factors (side 0: rows A_i; side 1: columns of B_i)."""
    rk = np.ascontiguousarray(ranks, dtype=np.int32)
    of = np.ascontiguousarray(offs, dtype=np.int64)
    st = lib().lf_pool_subspace(int(side), len(rk), rk.ctypes.data, of.ctypes.data, int(d), _ptr(base), int(num),
                                int(den), _ptr(k), _ptr(sigma), _ptr(basis), _ptr(coef), _ptr(resid), _ptr(ws),
                                ws.numel() if ws is not None else 0, _stream(stream))
    return _check(st, "lf_pool_subspace") if check else st


def lf_jd_full(mods, members, probs, B_base, A_base, weights, iters, U_base, Vt_base, sigma, ws, stream=None,
               check=True) -> int:
    """JD-Full eigenvalue iteration: U_base / Vt_base hold the starting bases on entry and the
    bases after `iters` steps on return; sigma (nullable) receives Sigma_i = U^T B_i A_i V."""
    st = lib().lf_jd_full(*_jd_tables(mods, members, probs), _ptr(B_base), _ptr(A_base), _ptr(weights),
                          int(iters), _ptr(U_base), _ptr(Vt_base), _ptr(sigma), _ptr(ws),
                          ws.numel() if ws is not None else 0, _stream(stream))
    return _check(st, "lf_jd_full") if check else st


def lf_lora_shrink_expand_noalloc(x, y, ids, n_adapters, ranks, off_A, off_Bt, A_pool, Bt_pool, scale,
                                  seg_out=None, stream=None, check=True) -> int:
    """lf_lora_shrink_expand without a workspace argument, for callers that cannot
    allocate device memory; the library keeps the routing scratch itself."""
    T, d_in = x.shape
    d_out = y.shape[1]
    st = lib().lf_lora_shrink_expand_noalloc(T, d_in, d_out, _ptr(x), _ptr(y), _ptr(ids), n_adapters,
                                             _ptr(ranks), _ptr(off_A), _ptr(off_Bt), _ptr(A_pool), _ptr(Bt_pool),
                                             A_pool.numel(), Bt_pool.numel(), float(scale), _ptr(seg_out),
                                             _stream(stream))
    return _check(st, "lf_lora_shrink_expand_noalloc") if check else st


def lf_status_string(st: int) -> str:
    return lib().lf_status_string(st).decode()


def lf_get_device_status(stream=None) -> int:
    return lib().lf_get_device_status(_stream(stream))


def lf_profile_enable(on: bool) -> None:
    lib().lf_profile_enable(1 if on else 0)


def lf_profile_reset() -> None:
    lib().lf_profile_reset()


def lf_profile_read() -> dict[str, tuple[float, int]]:
    """{phase: (total device ms, launches)} accumulated since the last reset."""
    buf = (lf_phase_time * 64)()
    n = lib().lf_profile_read(ctypes.addressof(buf), 64)
    return {buf[i].name.decode(): (buf[i].total_ms, buf[i].launches) for i in range(min(n, 64))}


def lf_launch_count() -> int:
    return lib().lf_launch_count()
