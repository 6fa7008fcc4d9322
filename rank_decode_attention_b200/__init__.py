"""Python binding of libs4r (S4R compressed-KV decode on B200, sm_100a).

Argument marshalling only: every function here fills the C structures of
``include/s4r.h`` from torch tensors (device pointers, sizes read from tensor
shapes) and calls the entry point of the same name in ``libs4r.so``.  All
arithmetic runs in the library's CUDA kernels; there is no Python or CPU
fallback, and a missing or unloadable library raises immediately.

Build the library with ``python -m rank_decode_attention_b200.build``.
"""
from __future__ import annotations

import ctypes
import os

import torch

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libs4r.so")

S4R_OK, S4R_ERR_INVALID_ARG, S4R_ERR_UNSUPPORTED, S4R_ERR_CUDA, S4R_ERR_TIMEOUT, \
    S4R_ERR_DEVICE, S4R_ERR_WORKSPACE = range(7)
S4R_F32, S4R_BF16, S4R_FP4 = 0, 1, 2
S4R_ROWS_CONCAT, S4R_ROWS_PER_HEAD = 0, 1
S4R_POOL_MAX, S4R_POOL_AVG = 0, 1

_DTYPE = {torch.float32: S4R_F32, torch.bfloat16: S4R_BF16}


class S4RError(RuntimeError):
    def __init__(self, status: int, what: str):
        detail = s4r_last_error() if status == S4R_ERR_CUDA else ""
        super().__init__(f"{what}: {s4r_status_string(status)} (status {status})"
                         + (f" -- {detail}" if detail else ""))
        self.status = status


class DecodeArgs(ctypes.Structure):
    _fields_ = [
        ("batch", ctypes.c_int32), ("n_heads_q", ctypes.c_int32), ("n_heads_kv", ctypes.c_int32),
        ("head_dim", ctypes.c_int32), ("rank_k", ctypes.c_int32), ("rank_v", ctypes.c_int32),
        ("n_sink", ctypes.c_int32), ("local_window", ctypes.c_int32), ("top_k", ctypes.c_int32),
        ("query_window", ctypes.c_int32), ("pool_kernel", ctypes.c_int32),
        ("pool_mode", ctypes.c_int32), ("row_mode", ctypes.c_int32), ("dtype", ctypes.c_int32),
        ("cache_rows", ctypes.c_int64),
        ("lengths", ctypes.c_void_p), ("q", ctypes.c_void_p),
        ("coeff_k", ctypes.c_void_p), ("coeff_v", ctypes.c_void_p),
        ("basis_k", ctypes.c_void_p), ("basis_v", ctypes.c_void_p),
        ("sink_k", ctypes.c_void_p), ("sink_v", ctypes.c_void_p),
        ("out", ctypes.c_void_p), ("idx", ctypes.c_void_p), ("scores", ctypes.c_void_p),
        ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t),
        ("profile_events", ctypes.c_void_p * 2),
    ]


class AppendArgs(ctypes.Structure):
    _fields_ = [
        ("batch", ctypes.c_int32), ("d_model", ctypes.c_int32), ("rank_k", ctypes.c_int32),
        ("rank_v", ctypes.c_int32), ("dtype", ctypes.c_int32), ("cache_rows", ctypes.c_int64),
        ("state_k", ctypes.c_void_p), ("state_v", ctypes.c_void_p),
        ("basis_k", ctypes.c_void_p), ("basis_v", ctypes.c_void_p),
        ("coeff_k", ctypes.c_void_p), ("coeff_v", ctypes.c_void_p),
        ("lengths", ctypes.c_void_p), ("status_workspace", ctypes.c_void_p),
    ]


class BasisArgs(ctypes.Structure):
    _fields_ = [
        ("n_problems", ctypes.c_int32), ("d_model", ctypes.c_int32), ("rank", ctypes.c_int32),
        ("n_sink", ctypes.c_int32), ("n_sample", ctypes.c_int32), ("dtype", ctypes.c_int32),
        ("state_rows", ctypes.c_int64),
        ("lengths", ctypes.c_void_p), ("states", ctypes.c_void_p), ("basis_out", ctypes.c_void_p),
        ("basis_f64", ctypes.c_void_p), ("sigma", ctypes.c_void_p),
        ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t),
    ]


class PagePlanArgs(ctypes.Structure):
    _fields_ = [
        ("batch", ctypes.c_int32), ("page_size", ctypes.c_int32), ("max_pages", ctypes.c_int32),
        ("free_capacity", ctypes.c_int32), ("max_tokens", ctypes.c_int64),
        ("lengths", ctypes.c_void_p), ("new_tokens", ctypes.c_void_p), ("block_table", ctypes.c_void_p),
        ("free_pages", ctypes.c_void_p), ("free_count", ctypes.c_void_p), ("lengths_out", ctypes.c_void_p),
        ("free_count_out", ctypes.c_void_p), ("cu_tokens", ctypes.c_void_p), ("slots", ctypes.c_void_p),
        ("positions", ctypes.c_void_p), ("requests", ctypes.c_void_p), ("status_workspace", ctypes.c_void_p),
    ]


class LatentWriteArgs(ctypes.Structure):
    _fields_ = [
        ("n_tokens", ctypes.c_int64), ("width", ctypes.c_int32), ("page_size", ctypes.c_int32),
        ("n_pages", ctypes.c_int64), ("cache_dtype", ctypes.c_int32), ("cache_scale", ctypes.c_float),
        ("latents", ctypes.c_void_p), ("latents_ld", ctypes.c_int64), ("slots", ctypes.c_void_p),
        ("cache", ctypes.c_void_p), ("stored", ctypes.c_void_p), ("status_workspace", ctypes.c_void_p),
    ]


class LatentAttendArgs(ctypes.Structure):
    _fields_ = [
        ("batch", ctypes.c_int32), ("n_query", ctypes.c_int32), ("n_heads", ctypes.c_int32),
        ("width", ctypes.c_int32), ("rank", ctypes.c_int32), ("page_size", ctypes.c_int32),
        ("max_pages", ctypes.c_int32), ("cache_dtype", ctypes.c_int32), ("n_pages", ctypes.c_int64),
        ("scale", ctypes.c_float), ("cache_scale", ctypes.c_float),
        ("q", ctypes.c_void_p), ("cache", ctypes.c_void_p), ("block_table", ctypes.c_void_p),
        ("lengths", ctypes.c_void_p), ("out", ctypes.c_void_p), ("lse", ctypes.c_void_p),
        ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t),
    ]


class LatentProjectArgs(ctypes.Structure):
    _fields_ = [
        ("n_tokens", ctypes.c_int64), ("n_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
        ("rank", ctypes.c_int32), ("to_latent", ctypes.c_int32), ("x", ctypes.c_void_p),
        ("x_ts", ctypes.c_int64), ("x_hs", ctypes.c_int64), ("basis", ctypes.c_void_p), ("out", ctypes.c_void_p),
        ("out_ts", ctypes.c_int64), ("out_hs", ctypes.c_int64),
    ]


class PrefillAttendArgs(ctypes.Structure):
    _fields_ = [
        ("batch", ctypes.c_int32), ("n_heads_q", ctypes.c_int32), ("n_heads_kv", ctypes.c_int32),
        ("head_dim", ctypes.c_int32), ("rope_dim", ctypes.c_int32), ("value_dim", ctypes.c_int32),
        ("causal", ctypes.c_int32), ("max_q", ctypes.c_int32), ("total_q", ctypes.c_int64),
        ("total_k", ctypes.c_int64), ("scale", ctypes.c_float),
        ("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_rope", ctypes.c_void_p),
        ("k_ts", ctypes.c_int64), ("v_ts", ctypes.c_int64), ("k_rope_ts", ctypes.c_int64),
        ("cu_q", ctypes.c_void_p), ("cu_k", ctypes.c_void_p), ("out", ctypes.c_void_p), ("lse", ctypes.c_void_p),
    ]


# Exported symbols and their C signatures (restype, argtypes).
_vp, _i32, _i64, _sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
SIGNATURES = {
    "s4r_encode": (ctypes.c_int, [_vp, _i64, _i64, _vp, _i32, _i32, _vp, _i64, ctypes.c_int, _vp]),
    "s4r_encode2": (ctypes.c_int, [_vp, _vp, _i64, _i64, _vp, _vp, _i32, _i32, _vp, _vp, _i64, ctypes.c_int, _vp]),
    "s4r_append": (ctypes.c_int, [ctypes.POINTER(AppendArgs), _vp]),
    "s4r_decode_workspace_bytes": (_sz, [ctypes.POINTER(DecodeArgs)]),
    "s4r_decode_kernel_launches": (_i32, [ctypes.POINTER(DecodeArgs)]),
    "s4r_workspace_init": (ctypes.c_int, [_vp, _sz, _vp]),
    "s4r_decode_step": (ctypes.c_int, [ctypes.POINTER(DecodeArgs), _vp]),
    "s4r_decode_step_noalloc": (ctypes.c_int, [ctypes.POINTER(DecodeArgs), _vp]),
    "s4r_basis_workspace_bytes": (_sz, [ctypes.POINTER(BasisArgs)]),
    "s4r_build_basis": (ctypes.c_int, [ctypes.POINTER(BasisArgs), _vp]),
    "s4r_reconstruct": (ctypes.c_int, [_vp, _i64, _vp, _i32, _i32, _vp, _i64, _vp, ctypes.c_int, _vp]),
    "s4r_page_plan": (ctypes.c_int, [ctypes.POINTER(PagePlanArgs), _vp]),
    "s4r_latent_write": (ctypes.c_int, [ctypes.POINTER(LatentWriteArgs), _vp]),
    "s4r_latent_attend_workspace_bytes": (_sz, [ctypes.POINTER(LatentAttendArgs)]),
    "s4r_latent_attend": (ctypes.c_int, [ctypes.POINTER(LatentAttendArgs), _vp]),
    "s4r_latent_project": (ctypes.c_int, [ctypes.POINTER(LatentProjectArgs), _vp]),
    "s4r_prefill_attend": (ctypes.c_int, [ctypes.POINTER(PrefillAttendArgs), _vp]),
    "s4r_read_device_status": (ctypes.c_int, [_vp, _vp]),
    "s4r_clear_device_status": (ctypes.c_int, [_vp, _vp]),
    "s4r_debug_waits": (ctypes.c_int, [_i64, _i32]),
    "s4r_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "s4r_version": (_i32, []),
    "s4r_last_error": (ctypes.c_char_p, []),
}

_lib = None


def lib() -> ctypes.CDLL:
    """Load libs4r.so (raises if it is missing: there is no fallback path)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing; build it with "
                               "`python -m rank_decode_attention_b200.build`")
        h = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(h, name)
            fn.restype, fn.argtypes = res, args
        _lib = h
    return _lib


def _ptr(t) -> int | None:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream) -> int | None:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream if torch.cuda.is_available() else None
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(status: int, what: str) -> int:
    if status != S4R_OK:
        raise S4RError(status, what)
    return status


def s4r_status_string(status: int) -> str:
    return lib().s4r_status_string(status).decode()


def s4r_last_error() -> str:
    return (lib().s4r_last_error() or b"").decode()


def s4r_version() -> int:
    return int(lib().s4r_version())


def s4r_encode(states: torch.Tensor, basis: torch.Tensor, coeffs: torch.Tensor, stream=None) -> int:
    """coeffs[t] = states[t] . basis (Eq. 3).  states [n][D'] (row stride may
    exceed D'), basis [D'][r], coeffs [n][r] (row stride may exceed r)."""
    n, d = states.shape
    r = basis.shape[1]
    return _check(lib().s4r_encode(_ptr(states), n, states.stride(0), _ptr(basis), d, r,
                                   _ptr(coeffs), coeffs.stride(0), _DTYPE[states.dtype],
                                   _stream(stream)), "s4r_encode")


def s4r_encode2(states, bases, coeffs, stream=None) -> int:
    """coeffs[p][t] = states[p][t] . bases[p] for p = 0, 1 (Eq. 3), one
    launch: two token sets of the same shape and strides with their own
    bases (the K and V halves of a prompt)."""
    s0, s1 = states
    n, d = s0.shape
    r = bases[0].shape[1]
    if s1.shape != s0.shape or s1.stride(0) != s0.stride(0) or coeffs[1].stride(0) != coeffs[0].stride(0):
        raise ValueError("s4r_encode2: both problems need the same shape and strides")
    return _check(lib().s4r_encode2(_ptr(s0), _ptr(s1), n, s0.stride(0), _ptr(bases[0]), _ptr(bases[1]), d, r,
                                    _ptr(coeffs[0]), _ptr(coeffs[1]), coeffs[0].stride(0), _DTYPE[s0.dtype],
                                    _stream(stream)), "s4r_encode2")


def append_args(*, state_k, state_v, basis_k, basis_v, coeff_k, coeff_v, lengths,
                status_workspace=None) -> AppendArgs:
    B, cache_rows, rk = coeff_k.shape
    return AppendArgs(B, basis_k.shape[1], rk, coeff_v.shape[2], _DTYPE[coeff_k.dtype], cache_rows,
                      _ptr(state_k), _ptr(state_v), _ptr(basis_k), _ptr(basis_v), _ptr(coeff_k),
                      _ptr(coeff_v), _ptr(lengths), _ptr(status_workspace))


def s4r_append(stream=None, **kw) -> int:
    """Encode one new token per problem and append it at row lengths[b]."""
    a = append_args(**kw)
    return _check(lib().s4r_append(ctypes.byref(a), _stream(stream)), "s4r_append")


def decode_args(*, q, coeff_k, coeff_v, basis_k, basis_v, sink_k, sink_v, lengths, n_heads_kv,
                local_window, top_k, out=None, idx=None, scores=None, workspace=None,
                workspace_bytes=None, pool_kernel=1, pool_mode=S4R_POOL_MAX,
                row_mode=S4R_ROWS_CONCAT, profile_events=None) -> DecodeArgs:
    """Fill s4r_decode_args from tensors: q [B][W][H_q][d_h], coeff_k/v
    [B][cache_rows][r], basis_k/v [B][D'][r], sink_k/v [B][s][D'],
    lengths [B] int32 (device)."""
    B, W, Hq, dh = q.shape
    cache_rows = coeff_k.shape[1]
    n_sink = sink_k.shape[1] if sink_k is not None else 0
    if workspace is not None and workspace_bytes is None:
        workspace_bytes = workspace.numel() * workspace.element_size()
    a = DecodeArgs(B, Hq, n_heads_kv, dh, coeff_k.shape[2], coeff_v.shape[2], n_sink,
                   local_window, top_k, W, pool_kernel, pool_mode, row_mode, _DTYPE[q.dtype],
                   cache_rows,
                   _ptr(lengths), _ptr(q), _ptr(coeff_k), _ptr(coeff_v), _ptr(basis_k),
                   _ptr(basis_v), _ptr(sink_k), _ptr(sink_v), _ptr(out), _ptr(idx),
                   _ptr(scores), _ptr(workspace), workspace_bytes or 0)
    if profile_events is not None:
        a.profile_events[0] = profile_events[0].cuda_event
        a.profile_events[1] = profile_events[1].cuda_event
    return a


def s4r_decode_kernel_launches(args: DecodeArgs) -> int:
    return int(lib().s4r_decode_kernel_launches(ctypes.byref(args)))


def s4r_decode_workspace_bytes(args: DecodeArgs) -> int:
    return int(lib().s4r_decode_workspace_bytes(ctypes.byref(args)))


def s4r_workspace_init(workspace: torch.Tensor, stream=None) -> int:
    nbytes = workspace.numel() * workspace.element_size()
    return _check(lib().s4r_workspace_init(_ptr(workspace), nbytes, _stream(stream)),
                  "s4r_workspace_init")


def s4r_decode_step(args: DecodeArgs, stream=None) -> int:
    """One decode step for every problem (see include/s4r.h)."""
    return _check(lib().s4r_decode_step(ctypes.byref(args), _stream(stream)), "s4r_decode_step")


def s4r_decode_step_noalloc(args: DecodeArgs, stream=None) -> int:
    """The decode step on the library's fixed per-device scratch array (no
    workspace, nothing allocated; see include/s4r.h for its limits)."""
    return _check(lib().s4r_decode_step_noalloc(ctypes.byref(args), _stream(stream)),
                  "s4r_decode_step_noalloc")


def basis_args(*, states, lengths, rank, n_sink, n_sample, basis_out=None, basis_f64=None, sigma=None,
               workspace=None, workspace_bytes=None) -> BasisArgs:
    """Fill s4r_basis_args: states [P][state_rows][D'] (bf16 or fp32), lengths
    [P] int32 (device), outputs basis_out [P][D'][r] (states' dtype),
    basis_f64 [P][D'][r] float64, sigma [P][r] float64."""
    P, state_rows, d = states.shape
    if workspace is not None and workspace_bytes is None:
        workspace_bytes = workspace.numel() * workspace.element_size()
    return BasisArgs(P, d, rank, n_sink, n_sample, _DTYPE[states.dtype], state_rows, _ptr(lengths),
                     _ptr(states), _ptr(basis_out), _ptr(basis_f64), _ptr(sigma), _ptr(workspace),
                     workspace_bytes or 0)


def s4r_basis_workspace_bytes(args: BasisArgs) -> int:
    return int(lib().s4r_basis_workspace_bytes(ctypes.byref(args)))


def s4r_build_basis(args: BasisArgs, stream=None) -> int:
    """Prefill bases: 7:3 sample, unit-norm rows, top-r right singular
    vectors in fp64 (Eqs. 1-2; see include/s4r.h)."""
    return _check(lib().s4r_build_basis(ctypes.byref(args), _stream(stream)), "s4r_build_basis")


def s4r_reconstruct(coeffs: torch.Tensor, basis: torch.Tensor, rows: torch.Tensor,
                    out: torch.Tensor, stream=None) -> int:
    """out[e] = coeffs[rows[e]] . basis^T in fp32 (Eq. 16)."""
    n_total, r = coeffs.shape
    return _check(lib().s4r_reconstruct(_ptr(coeffs), n_total, _ptr(basis), basis.shape[0], r,
                                        _ptr(rows), rows.numel(), _ptr(out), _DTYPE[coeffs.dtype],
                                        _stream(stream)), "s4r_reconstruct")


# ---- paged latent cache and prefill attention

_BF16, _F32, _I32, _I64, _U8 = torch.bfloat16, torch.float32, torch.int32, torch.int64, torch.uint8


def _device() -> int:
    """Index of the current CUDA device; -2 (no tensor's) without one."""
    try:
        return torch.cuda.current_device()
    except (RuntimeError, AssertionError):
        return -2


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream_on(stream, dev: int):
    """Handle of `stream`, or of the current stream of device `dev` (a serving loop makes these calls every step: the
    current stream without a Stream object around it)."""
    if stream is None and _raw_stream is not None and dev >= 0:
        return _raw_stream(dev)
    return _stream(stream)


def _arg(what: str, name: str, t, dtype, shape, dev: int, dense_from: int = 0):
    """Data pointer of tensor `t`, which must have the type, the shape, the device `dev` and contiguous dimensions from
    `dense_from` on."""
    if t.dtype is dtype and t.shape == shape and t.get_device() == dev and t.is_contiguous():
        return t.data_ptr()
    if t.dtype is not dtype:
        raise ValueError(f"{what}: {name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{what}: {name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    step = 1
    for i in range(len(shape) - 1, dense_from - 1, -1):
        if shape[i] != 1 and t.stride(i) != step:
            raise ValueError(f"{what}: {name} must be contiguous" + (f" from dimension {dense_from} on" if dense_from else ""))
        step *= shape[i]
    if t.get_device() != dev:
        raise ValueError(f"{what}: {name} must be on the current CUDA device, got {t.device}")
    return t.data_ptr()


def _dims(what: str, name: str, t, n: int):
    """Shape of a tensor of `n` dimensions."""
    s = t.shape
    if len(s) != n:
        raise ValueError(f"{what}: {name} must have {n} dimensions, got {tuple(s)}")
    return s


def _workspace(what: str, t, dev: int):
    """(pointer, bytes) of a workspace tensor or (None, 0)."""
    if t is None:
        return None, 0
    if t.get_device() != dev or not t.is_contiguous():
        raise ValueError(f"{what}: the workspace must be contiguous and on the current CUDA device, got {t.device}")
    return t.data_ptr(), t.numel() * t.element_size()


def _latent_cache(what: str, cache, width: int, page_size: int, dev: int):
    """(S4R type, pages, pointer) of a paged cache: bf16 [pages][page_size][width], or uint8
    [pages][page_size * width * 9 // 16] (4-bit)."""
    if cache.dtype is _U8:
        if page_size * width % 16:
            raise ValueError(f"{what}: a 4-bit page holds whole groups of 16 columns")
        n = _dims(what, "cache", cache, 2)[0]
        return S4R_FP4, n, _arg(what, "cache", cache, _U8, (n, page_size * width * 9 // 16), dev)
    n = _dims(what, "cache", cache, 3)[0]
    return S4R_BF16, n, _arg(what, "cache", cache, _BF16, (n, page_size, width), dev)


def s4r_page_plan(*, lengths, new_tokens, block_table, free_pages, free_count, lengths_out, free_count_out, cu_tokens,
                  slots, page_size, positions=None, requests=None, status_workspace=None, stream=None) -> int:
    """Block tables and slot maps of a step on the device (see include/s4r.h): lengths, new_tokens, lengths_out [B],
    block_table [B][max_pages], free_pages [capacity], free_count, free_count_out [1], cu_tokens [B+1] int32; slots
    [max_tokens] int64, positions and requests [max_tokens] int32 or None."""
    w, dev = "s4r_page_plan", _device()
    B, n, one = lengths.shape[0], slots.shape[0], (1,)
    cols, capacity = _dims(w, "block_table", block_table, 2)[1], free_pages.shape[0]
    per, per_token = (B,), (n,)
    a = PagePlanArgs(
        B, page_size, cols, capacity, n,
        _arg(w, "lengths", lengths, _I32, per, dev), _arg(w, "new_tokens", new_tokens, _I32, per, dev),
        _arg(w, "block_table", block_table, _I32, (B, cols), dev), _arg(w, "free_pages", free_pages, _I32, (capacity,), dev),
        _arg(w, "free_count", free_count, _I32, one, dev), _arg(w, "lengths_out", lengths_out, _I32, per, dev),
        _arg(w, "free_count_out", free_count_out, _I32, one, dev), _arg(w, "cu_tokens", cu_tokens, _I32, (B + 1,), dev),
        _arg(w, "slots", slots, _I64, per_token, dev),
        None if positions is None else _arg(w, "positions", positions, _I32, per_token, dev),
        None if requests is None else _arg(w, "requests", requests, _I32, per_token, dev),
        None if status_workspace is None else _workspace(w, status_workspace, dev)[0])
    return _check(lib().s4r_page_plan(ctypes.byref(a), _stream_on(stream, dev)), w)


def s4r_latent_write(*, latents, slots, cache, page_size, cache_scale=1.0, stored=None, status_workspace=None,
                     stream=None) -> int:
    """Store latents [n][width] bf16 (row stride may exceed width) at slots [n] int64 of a paged cache: bf16
    [pages][page_size][width] or uint8 [pages][page_size*width*9//16] (4-bit, see include/s4r.h)."""
    w, dev = "s4r_latent_write", _device()
    n, width = _dims(w, "latents", latents, 2)
    dt, pages, cache_ptr = _latent_cache(w, cache, width, page_size, dev)
    a = LatentWriteArgs(
        n, width, page_size, pages, dt, cache_scale, _arg(w, "latents", latents, _BF16, (n, width), dev, 1),
        latents.stride(0) if n > 1 else width, _arg(w, "slots", slots, _I64, (n,), dev), cache_ptr,
        None if stored is None else _arg(w, "stored", stored, _BF16, (n, width), dev),
        None if status_workspace is None else _workspace(w, status_workspace, dev)[0])
    return _check(lib().s4r_latent_write(ctypes.byref(a), _stream_on(stream, dev)), w)


def latent_attend_args(*, q, cache, block_table, lengths, out, page_size, scale, lse=None, cache_scale=1.0,
                       workspace=None) -> LatentAttendArgs:
    """Fill s4r_latent_attend_args: q [B][n_query][H][width] bf16, cache as in s4r_latent_write, block_table
    [B][max_pages] and lengths [B] int32, out [B][n_query][H][rank] bf16, lse [B][n_query][H] float32 or None."""
    w, dev = "s4r_latent_attend", _device()
    B, T, H, width = _dims(w, "q", q, 4)
    rank, cols = _dims(w, "out", out, 4)[3], _dims(w, "block_table", block_table, 2)[1]
    dt, pages, cache_ptr = _latent_cache(w, cache, width, page_size, dev)
    ws, ws_bytes = _workspace(w, workspace, dev)
    return LatentAttendArgs(
        B, T, H, width, rank, page_size, cols, dt, pages, scale, cache_scale,
        _arg(w, "q", q, _BF16, (B, T, H, width), dev), cache_ptr, _arg(w, "block_table", block_table, _I32, (B, cols), dev),
        _arg(w, "lengths", lengths, _I32, (B,), dev), _arg(w, "out", out, _BF16, (B, T, H, rank), dev),
        None if lse is None else _arg(w, "lse", lse, _F32, (B, T, H), dev), ws, ws_bytes)


def s4r_latent_attend_workspace_bytes(args: LatentAttendArgs) -> int:
    return int(lib().s4r_latent_attend_workspace_bytes(ctypes.byref(args)))


def s4r_latent_attend(args: LatentAttendArgs, stream=None) -> int:
    """Attention over a paged latent cache, absorbed form (see include/s4r.h)."""
    return _check(lib().s4r_latent_attend(ctypes.byref(args), _stream_on(stream, _device())), "s4r_latent_attend")


def s4r_latent_project(x, basis, out, *, to_latent: bool, stream=None) -> int:
    """Per-head products with basis [H*head_dim][rank] bf16: x [n][H][head_dim] to out [n][H][rank] (to_latent), or x
    [n][H][rank] (or [n][rank], one row for all heads) to out [n][H][head_dim].  Token and head strides are free."""
    w, dev = "s4r_latent_project", _device()
    n, H, n_out = _dims(w, "out", out, 3)
    n_in = x.shape[-1]
    dim, rank = (n_in, n_out) if to_latent else (n_out, n_in)
    shared = x.dim() == 2
    xp = _arg(w, "x", x, _BF16, (n, n_in) if shared else (n, H, n_in), dev, 1 if shared else 2)
    op = _arg(w, "out", out, _BF16, (n, H, n_out), dev, 2)
    a = LatentProjectArgs(
        n, H, dim, rank, 1 if to_latent else 0, xp, x.stride(0) if n > 1 else H * n_in,
        0 if shared else (x.stride(1) if H > 1 else n_in),
        _arg(w, "basis", basis, _BF16, (H * dim, rank), dev), op, out.stride(0) if n > 1 else H * n_out,
        out.stride(1) if H > 1 else n_out)
    return _check(lib().s4r_latent_project(ctypes.byref(a), _stream_on(stream, dev)), w)


def prefill_attend_args(*, q, k, v, cu_q, cu_k, max_q, scale, out, k_rope=None, lse=None,
                        causal=True) -> PrefillAttendArgs:
    """Fill s4r_prefill_attend_args: q [total_q][Hq][head_dim + rope_dim], k [total_k][Hkv][head_dim], v
    [total_k][Hkv][value_dim], k_rope [total_k][rope_dim] or None, out [total_q][Hq][value_dim] bf16 (token strides of k,
    v, k_rope are free), cu_q and cu_k [B+1] int32, lse [total_q][Hq] float32 or None."""
    w, dev = "s4r_prefill_attend", _device()
    nq, Hq, _ = _dims(w, "q", q, 3)
    nk, Hkv, dim = _dims(w, "k", k, 3)
    vd = _dims(w, "v", v, 3)[2]
    rope = 0 if k_rope is None else _dims(w, "k_rope", k_rope, 2)[1]
    B = cu_q.shape[0] - 1
    return PrefillAttendArgs(
        B, Hq, Hkv, dim, rope, vd, 1 if causal else 0, max_q, nq, nk, scale,
        _arg(w, "q", q, _BF16, (nq, Hq, dim + rope), dev), _arg(w, "k", k, _BF16, (nk, Hkv, dim), dev, 1),
        _arg(w, "v", v, _BF16, (nk, Hkv, vd), dev, 1),
        None if k_rope is None else _arg(w, "k_rope", k_rope, _BF16, (nk, rope), dev, 1),
        k.stride(0) if nk > 1 else Hkv * dim, v.stride(0) if nk > 1 else Hkv * vd,
        0 if k_rope is None else (k_rope.stride(0) if nk > 1 else rope),
        _arg(w, "cu_q", cu_q, _I32, (B + 1,), dev), _arg(w, "cu_k", cu_k, _I32, (B + 1,), dev),
        _arg(w, "out", out, _BF16, (nq, Hq, vd), dev), None if lse is None else _arg(w, "lse", lse, _F32, (nq, Hq), dev))


def s4r_prefill_attend(args: PrefillAttendArgs, stream=None) -> int:
    """Attention of ragged prompts over expanded keys and values (see include/s4r.h)."""
    return _check(lib().s4r_prefill_attend(ctypes.byref(args), _stream_on(stream, _device())), "s4r_prefill_attend")


def s4r_read_device_status(workspace, stream=None) -> int:
    """Synchronise the stream and return the sticky device status code."""
    return int(lib().s4r_read_device_status(_ptr(workspace), _stream(stream)))


def s4r_debug_waits(limit_cycles: int = 0, unreachable_barrier: bool = False) -> int:
    """Testing hook: limit of the device-side bounded waits (SM cycles, 0 =
    default) and the switch that makes the scoring kernel's grid barrier and a
    signal in each kernel of latent attention, prefill attention and the
    projection unreachable (see include/s4r.h)."""
    return _check(lib().s4r_debug_waits(int(limit_cycles), 1 if unreachable_barrier else 0),
                  "s4r_debug_waits")


def s4r_clear_device_status(workspace, stream=None) -> int:
    return _check(lib().s4r_clear_device_status(_ptr(workspace), _stream(stream)),
                  "s4r_clear_device_status")
