"""Python binding of libfa (exact IO-aware attention on B200, sm_100a).

Argument marshalling only: every step of the attention computation runs in the
CUDA kernels behind the C ABI declared in ``include/fa.h``.  PyTorch supplies
device memory and the current stream.  There is no CPU fallback: if the
library is missing or no GPU is present, every call raises.
"""
from __future__ import annotations

import ctypes
import math
import os
import struct
from typing import NamedTuple, Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libfa.so")

FA_BF16, FA_F32 = 0, 1
BWD_DKDV_PAIR, BWD_DKDV_SINGLE = 1, 2   # fa.h FA_BWD_DKDV_*
_STATUS = {0: "FA_OK", -1: "FA_ERR_INVALID", -2: "FA_ERR_UNSUPPORTED", -3: "FA_ERR_ALIGN",
           -4: "FA_ERR_CUDA", -5: "FA_ERR_TIMEOUT", -6: "FA_ERR_WORKSPACE"}

# exported symbol -> (restype, argtypes)
_vp, _i, _f, _sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
_l = ctypes.c_int64
SIGNATURES = {
    "fa_fwd": (_i, [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _f, _i, _vp, _vp, _i, _vp]),
    "fa_fwd_gqa": (_i, [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _f, _i, _vp, _vp, _i, _vp]),
    "fa_bwd_workspace_size": (_sz, [_i, _i, _i, _i]),
    "fa_bwd_gqa": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _f, _i,
                        _vp, _vp, _i, _vp, _sz, _vp]),
    "fa_bwd_deterministic": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i,
                                  _f, _i, _vp, _vp, _i, _vp, _sz, _vp]),
    "fa_bwd": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _f, _i, _vp,
                    _vp, _i, _vp, _sz, _vp]),
    "fa_bwd_noalloc": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _f, _i,
                            _vp, _vp, _i, _vp]),
    "fa_bwd_deterministic_ex": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i,
                                     _i, _f, _i, _vp, _vp, _i, _vp, _sz, _i, _vp]),
    "fa_rope": (_i, [_vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _vp, _vp, _l, _f, _i, _i, _vp]),
    "fa_paged_plan": (_i, [_vp, _vp, _vp, _i, _vp, _vp, _l, _i, _i, _i, _i, _vp, _vp, _vp, _vp,
                           _vp, _vp]),
    "fa_paged_append": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _vp,
                             _l, _l, _i, _i, _f, _i, _i, _vp]),
    "fa_paged_workspace_size": (_sz, [_i, _i, _i, _i, _i]),
    "fa_paged_fwd": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _l, _l, _l,
                          _l, _l, _i, _i, _i, _i, _f, _i, _i, _vp, _sz, _vp]),
    "fa_rope_packed": (_i, [ctypes.c_char_p]),
    "fa_paged_plan_packed": (_i, [ctypes.c_char_p]),
    "fa_paged_append_packed": (_i, [ctypes.c_char_p]),
    "fa_paged_fwd_packed": (_i, [ctypes.c_char_p]),
    "fa_fwd_tile_reference": (_i, [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _f, _i, _vp, _vp,
                                   _i, _i, _vp]),
    "fa_naive_workspace_size": (_sz, [_i, _i, _i]),
    "fa_naive_fwd": (_i, [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _f, _i, _vp, _vp, _vp, _sz,
                          _vp]),
    "fa_diag_exp2": (_i, [_vp, _vp, _vp, _vp, _i, _vp]),
    "fa_diag_wait_timeout": (_i, [_i, _vp]),
    "fa_launch_count": (ctypes.c_ulonglong, []),
    "fa_kernel_timing": (_i, [_i]),
    "fa_kernel_timing_read": (_i, [ctypes.c_char_p, ctypes.POINTER(ctypes.c_int),
                                   ctypes.POINTER(ctypes.c_double)]),
    "fa_get_last_error": (ctypes.c_char_p, []),
    "fa_device_status": (_i, [ctypes.POINTER(ctypes.c_uint)]),
}

_lib = None


class FaError(RuntimeError):
    pass


def load(path: str = LIB_PATH):
    """Load libfa.so (built by ``exact_io_aware_98_b200.build``); raises if absent."""
    global _lib
    if _lib is None:
        if not os.path.exists(path):
            raise FaError(f"libfa.so not found at {path}: build it first "
                          "(python -m exact_io_aware_98_b200.build)")
        lib = ctypes.CDLL(path)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _lib = lib
    return _lib


def _check(rc: int, what: str):
    if rc != 0:
        msg = load().fa_get_last_error().decode(errors="replace")
        raise FaError(f"{what}: {_STATUS.get(rc, rc)}: {msg}")


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream():
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def _require(t: torch.Tensor, name: str, dtype=None):
    if not t.is_cuda:
        raise FaError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise FaError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise FaError(f"{name} must be {dtype}, got {t.dtype}")


def _masks(block_mask, kv_len):
    if block_mask is not None:
        _require(block_mask, "block_mask", torch.uint8)
    if kv_len is not None:
        _require(kv_len, "kv_len", torch.int32)
    return _ptr(block_mask), _ptr(kv_len)


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return FA_BF16
    if t.dtype == torch.float32:
        return FA_F32
    raise FaError(f"unsupported dtype {t.dtype}")


def default_scale(d: int) -> float:
    return float(torch.tensor(1.0 / math.sqrt(d), dtype=torch.float32).item())


def _kv_heads(q, k, v) -> int:
    """K/V head count; k and v are [B, H_kv, N, d] with H a multiple of H_kv."""
    B, H, N, d = q.shape
    H_kv = k.shape[1]
    for t, n in ((k, "k"), (v, "v")):
        if t.dim() != 4 or (t.shape[0], t.shape[2], t.shape[3]) != (B, N, d) or t.shape[1] != H_kv:
            raise FaError(f"{n} shape {tuple(t.shape)} does not match q {tuple(q.shape)}")
    if H_kv < 1 or H % H_kv != 0:
        raise FaError(f"H = {H} is not a multiple of H_kv = {H_kv}")
    return H_kv


def fwd(q, k, v, scale: Optional[float] = None, causal: bool = False, block_mask=None,
        kv_len=None, out=None, lse=None):
    """O, lse = fa_fwd(q, k, v); q [B, H, N, d], k and v [B, H_kv, N, d] (bf16 or fp32) on the
    GPU.  H_kv < H is grouped-query attention (fa_fwd_gqa): query head h reads K/V head
    h // (H / H_kv)."""
    lib = load()
    B, H, N, d = q.shape
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _require(t, n, q.dtype)
    H_kv = _kv_heads(q, k, v)
    o = torch.empty_like(q) if out is None else out
    l = torch.empty((B, H, N), dtype=torch.float32, device=q.device) if lse is None else lse
    _require(o, "out", q.dtype)
    _require(l, "lse", torch.float32)
    bm, kl = _masks(block_mask, kv_len)
    s = default_scale(d) if scale is None else float(scale)
    if H_kv == H:
        rc = lib.fa_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(l), B, H, N, d, s, int(causal),
                        bm, kl, _dtype_code(q), _stream())
        _check(rc, "fa_fwd")
    else:
        rc = lib.fa_fwd_gqa(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(l), B, H, H_kv, N, d, s,
                            int(causal), bm, kl, _dtype_code(q), _stream())
        _check(rc, "fa_fwd_gqa")
    return o, l


def bwd_workspace_size(B: int, H: int, N: int, d: int) -> int:
    return int(load().fa_bwd_workspace_size(B, H, N, d))


def _bwd_operands(q, k, v, o, lse, do, dq, dk, dv):
    """Checks shared by every backward call: dtypes, contiguity, and the shapes of o, do, lse
    and of caller-supplied gradients against q, k and v (so that no kernel is ever handed a
    buffer smaller than the tensor maps it builds from q's sizes).  Returns H_kv and dq, dk, dv
    (allocated here when not supplied)."""
    B, H, N, d = q.shape
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (o, "o"), (do, "do")):
        _require(t, n, q.dtype)
    H_kv = _kv_heads(q, k, v)
    for t, n in ((o, "o"), (do, "do")):
        if t.shape != q.shape:
            raise FaError(f"{n} shape {tuple(t.shape)} does not match q {tuple(q.shape)}")
    _require(lse, "lse", torch.float32)
    if tuple(lse.shape) != (B, H, N):
        raise FaError(f"lse shape {tuple(lse.shape)} must be {(B, H, N)}")
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    for t, n in ((dq, "dq"), (dk, "dk"), (dv, "dv")):
        _require(t, n, q.dtype)
    if dq.shape != q.shape or dk.shape != k.shape or dv.shape != v.shape:
        raise FaError("gradient shapes must match q, k and v")
    return H_kv, dq, dk, dv


def bwd(q, k, v, o, lse, do, scale: Optional[float] = None, causal: bool = False,
        block_mask=None, kv_len=None, workspace=None, dq=None, dk=None, dv=None,
        deterministic: bool = False, dkdv_pair: Optional[bool] = None):
    """dQ, dK, dV = fa_bwd(...); tensors on the GPU, q/o/do [B, H, N, d], k/v and dK/dV
    [B, H_kv, N, d] (fa_bwd_gqa when H_kv < H).  ``deterministic`` calls fa_bwd_deterministic:
    bit-reproducible gradients, dQ without atomics; with it, ``dkdv_pair`` True / False picks
    the 2-CTA or the single-CTA dK/dV kernel at d = 128 (fa_bwd_deterministic_ex), None the
    library's default."""
    lib = load()
    B, H, N, d = q.shape
    H_kv, dq, dk, dv = _bwd_operands(q, k, v, o, lse, do, dq, dk, dv)
    need = bwd_workspace_size(B, H, N, d)
    ws = torch.empty(need, dtype=torch.uint8, device=q.device) if workspace is None else workspace
    _require(ws, "workspace", torch.uint8)
    bm, kl = _masks(block_mask, kv_len)
    s = default_scale(d) if scale is None else float(scale)
    if deterministic and dkdv_pair is not None:
        opt = BWD_DKDV_PAIR if dkdv_pair else BWD_DKDV_SINGLE
        rc = lib.fa_bwd_deterministic_ex(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(do),
                                         _ptr(dq), _ptr(dk), _ptr(dv), B, H, H_kv, N, d, s,
                                         int(causal), bm, kl, _dtype_code(q), _ptr(ws),
                                         ws.numel(), opt, _stream())
        _check(rc, "fa_bwd_deterministic_ex")
    elif deterministic:
        rc = lib.fa_bwd_deterministic(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(do),
                                      _ptr(dq), _ptr(dk), _ptr(dv), B, H, H_kv, N, d, s,
                                      int(causal), bm, kl, _dtype_code(q), _ptr(ws), ws.numel(),
                                      _stream())
        _check(rc, "fa_bwd_deterministic")
    elif H_kv == H:
        rc = lib.fa_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(do), _ptr(dq),
                        _ptr(dk), _ptr(dv), B, H, N, d, s, int(causal), bm, kl, _dtype_code(q),
                        _ptr(ws), ws.numel(), _stream())
        _check(rc, "fa_bwd")
    else:
        rc = lib.fa_bwd_gqa(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(do), _ptr(dq),
                            _ptr(dk), _ptr(dv), B, H, H_kv, N, d, s, int(causal), bm, kl,
                            _dtype_code(q), _ptr(ws), ws.numel(), _stream())
        _check(rc, "fa_bwd_gqa")
    return dq, dk, dv


def bwd_noalloc(q, k, v, o, lse, do, scale: Optional[float] = None, causal: bool = False,
                block_mask=None, kv_len=None, dq=None, dk=None, dv=None):
    """fa_bwd without a workspace, for callers that cannot allocate device memory: the
    library's own fixed 32 MiB scratch is used instead, and calls on one device must not
    overlap.  Ordinary attention only (k and v have q's H heads).  dq, dk and dv may be passed
    in; otherwise this wrapper allocates them with torch, which a caller that cannot allocate
    avoids by passing its own."""
    lib = load()
    B, H, N, d = q.shape
    H_kv, dq, dk, dv = _bwd_operands(q, k, v, o, lse, do, dq, dk, dv)
    if H_kv != H:
        raise FaError(f"fa_bwd_noalloc takes ordinary attention only (k/v have {H_kv} heads, "
                      f"q has {H})")
    bm, kl = _masks(block_mask, kv_len)
    s = default_scale(d) if scale is None else float(scale)
    rc = lib.fa_bwd_noalloc(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(do), _ptr(dq),
                            _ptr(dk), _ptr(dv), B, H, N, d, s, int(causal), bm, kl,
                            _dtype_code(q), _stream())
    _check(rc, "fa_bwd_noalloc")
    return dq, dk, dv


# ----------------------------------------------------------------- rotary positions, paged cache
ROPE_INTERLEAVED, ROPE_BACKWARD = 1, 2   # fa.h FA_ROPE_*


# The calls below are a few microseconds of GPU work at a decoding step's sizes, so their checks are
# written for the host: device numbers, shapes and dtypes are compared directly, and only a
# comparison that fails goes through the functions that say which.  The arguments go over in one
# packed structure (fa.h, fa_*_args), which costs a third of what as many ctypes arguments do.
_ROPE = struct.Struct("@Q5Q7q7if")
_PLAN = struct.Struct("@Q11Qq6i")
_APPEND = struct.Struct("@Q10Q10q9if")
_FWD = struct.Struct("@Q11Q5q11if")


def _refuse(dev: int, *specs):
    """Raises for the first (name, tensor, dtype, shape or None, contiguous) that does not hold on
    CUDA device ``dev``; returns if all do."""
    for name, t, dtype, shape, contiguous in specs:
        if not t.is_cuda:
            raise FaError(f"{name} must be a CUDA tensor")
        if t.get_device() != dev:
            raise FaError(f"{name} is on {t.device}, not cuda:{dev}")
        if dtype is not None and t.dtype is not dtype:
            raise FaError(f"{name} must be {dtype}, got {t.dtype}")
        if shape is not None and tuple(t.shape) != tuple(shape):
            raise FaError(f"{name} shape {tuple(t.shape)} must be {tuple(shape)}")
        if contiguous and not t.is_contiguous():
            raise FaError(f"{name} must be contiguous")


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)  # absent without CUDA
_get_device = getattr(torch._C, "_cuda_getDevice", None)


def _call(dev: int, fn, args: struct.Struct, *values):
    """One packed call with CUDA device ``dev`` current; its stream is among the values."""
    try:
        packed = args.pack(args.size, *values)
    except (struct.error, OverflowError) as e:  # a size that is no int32, a scale that is no float
        raise FaError(f"{fn.__name__.removesuffix('_packed')}: {e}") from None
    if dev == _get_device():
        rc = fn(packed)
    else:
        with torch.cuda.device(dev):
            rc = fn(packed)
    if rc != 0:
        _check(rc, fn.__name__.removesuffix("_packed"))


def rope_frequencies(rotary_dim: int, base: float = 10000.0, scaling: Optional[str] = None,
                     factor: float = 1.0, original_length: Optional[int] = None,
                     beta_fast: float = 32.0, beta_slow: float = 1.0, device="cuda"):
    """(inv_freq, magnitude) for ``rope`` and ``paged_append``: float64 [rotary_dim / 2] radians
    per position on ``device``, base^(-2i / rotary_dim), scaled for contexts ``factor`` times
    longer:
      None        unscaled
      "linear"    every frequency divided by ``factor``
      "ntk"       base times factor^(rotary_dim / (rotary_dim - 2)): the lowest frequency is
                  divided by ``factor``, the highest stays
      "by_parts"  (YaRN, arXiv 2309.00071) frequencies that turn at least ``beta_fast`` times in
                  ``original_length`` positions stay, those that turn at most ``beta_slow`` times
                  are divided by ``factor``, linearly between; magnitude 0.1 ln(factor) + 1."""
    if rotary_dim < 2 or rotary_dim % 2:
        raise FaError(f"rotary_dim must be even and positive, got {rotary_dim}")
    if not (base > 0.0 and math.isfinite(base)) or not (factor >= 1.0 and math.isfinite(factor)):
        raise FaError("base must be positive, factor at least 1, both finite")
    i = torch.arange(rotary_dim // 2, dtype=torch.float64)
    if scaling == "ntk" and rotary_dim > 2:
        base = base * factor ** (rotary_dim / (rotary_dim - 2.0))
    f = base ** (-2.0 * i / rotary_dim)
    magnitude = 1.0
    if scaling == "linear":
        f = f / factor
    elif scaling == "by_parts":
        if original_length is None or original_length < 1 or not beta_fast > beta_slow:
            raise FaError('"by_parts" needs original_length >= 1 and beta_fast > beta_slow')
        keep = ((original_length * f / (2.0 * math.pi) - beta_slow) / (beta_fast - beta_slow)).clamp(0.0, 1.0)
        f = f * keep + f / factor * (1.0 - keep)
        magnitude = 0.1 * math.log(factor) + 1.0
    elif scaling not in (None, "ntk"):
        raise FaError(f"unknown scaling {scaling!r}")
    return f.to(device), magnitude


def _rope(x, inv_freq, positions, interleaved, magnitude, out, options):
    lib = _lib or load()
    dev = x.get_device()
    dtype, shape, xs = x.dtype, x.shape, x.stride()
    y = out
    if y is None:
        y = torch.empty(shape, dtype=dtype, device=x.device)
    ys = y.stride()
    if dev < 0 or dev != inv_freq.get_device() or dev != y.get_device() or y.dtype is not dtype or \
            inv_freq.dtype is not torch.float64 or not inv_freq.is_contiguous() or y.shape != shape:
        _refuse(dev, ("x", x, None, None, False), ("inv_freq", inv_freq, torch.float64, None, True),
                ("out", y, dtype, shape, False))
    if len(shape) == 3:
        N, H, d = shape
        B = 1
        xs, ys = (0, xs[1], xs[0], xs[2]), (0, ys[1], ys[0], ys[2])
    elif len(shape) == 4:
        B, H, N, d = shape
    else:
        raise FaError(f"x must be [B, H, N, d] or [T, H, d], got {tuple(shape)}")
    if d > 1 and (xs[-1] != 1 or ys[-1] != 1):
        raise FaError("the last dimension of x and out must be contiguous")
    ps = pp = 0
    if positions is not None:
        if positions.get_device() != dev or positions.dtype is not torch.int32:
            _refuse(dev, ("positions", positions, torch.int32, None, False))
        if positions.shape != (N,):
            if len(shape) == 3 or positions.shape != (B, N):
                raise FaError(f"positions shape {tuple(positions.shape)} does not match x {tuple(shape)}")
            ps = positions.stride(0)
        if N > 1 and positions.stride(-1) != 1:
            raise FaError("positions must be contiguous along the tokens")
        pp = positions.data_ptr()
    _call(dev, lib.fa_rope_packed, _ROPE, x.data_ptr(), y.data_ptr(), pp, inv_freq.data_ptr(), _raw_stream(dev),
          xs[0], xs[1], xs[2], ys[0], ys[1], ys[2], ps, B, H, N, d, 2 * inv_freq.numel(),
          options | ROPE_INTERLEAVED if interleaved else options, _dtype_code(x), magnitude)
    return y


def rope(x, inv_freq, positions=None, interleaved: bool = False, magnitude: float = 1.0, out=None):
    """Rotary positions (fa_rope) on x [B, H, N, d] or packed [T, H, d], bf16 or fp32, any
    strides with d contiguous; the first 2 * len(inv_freq) columns turn.  positions int32 [N]
    or [B, N] ([T] when packed), default 0 .. N-1.  ``out`` may be x."""
    return _rope(x, inv_freq, positions, interleaved, magnitude, out, 0)


def rope_bwd(dy, inv_freq, positions=None, interleaved: bool = False, magnitude: float = 1.0,
             out=None):
    """dL/dx of ``rope`` from dL/dy, with the same arguments."""
    return _rope(dy, inv_freq, positions, interleaved, magnitude, out, ROPE_BACKWARD)


class PagedPlan(NamedTuple):
    """Outputs of ``paged_plan`` (int32, slots int64)."""
    cu_q: torch.Tensor       # [B + 1] first row of each request's new tokens
    kv_len: torch.Tensor     # [B] cached keys including the new tokens
    positions: torch.Tensor  # [max_tokens]
    slots: torch.Tensor      # [max_tokens], -1: not stored
    counts: torch.Tensor     # [4] tokens asked for, pages taken, pages short, cursor after

    @classmethod
    def empty(cls, B: int, max_tokens: int, device="cuda"):
        i32 = lambda n: torch.empty(n, dtype=torch.int32, device=device)
        return cls(i32(B + 1), i32(B), i32(max_tokens),
                   torch.empty(max_tokens, dtype=torch.int64, device=device), i32(4))


def paged_plan(ctx_len, new_len, free_pages, block_table, page_size: int, max_tokens: int,
               cursor=None, out: Optional[PagedPlan] = None) -> PagedPlan:
    """One step's bookkeeping on the GPU (fa_paged_plan): ctx_len and new_len int32 [B],
    free_pages int32 [F] (handed out from ``cursor``, int32 [1], on), block_table int32
    [B, max_pages] updated in place.  ``out`` reuses an earlier plan's tensors."""
    lib = _lib or load()
    dev = ctx_len.get_device()
    B = ctx_len.numel()
    max_tokens = int(max_tokens)
    if out is None:
        if max_tokens < 1 or B < 1:
            raise FaError("paged_plan needs at least one request and max_tokens >= 1")
        out = PagedPlan.empty(B, max_tokens, ctx_len.device)
    cu_q, kv_len, positions, slots, counts = out
    i32 = torch.int32
    if not (dev >= 0 and dev == new_len.get_device() == free_pages.get_device() == block_table.get_device()
            == cu_q.get_device() == kv_len.get_device() == positions.get_device() == slots.get_device()
            == counts.get_device()
            and ctx_len.dtype is i32 and new_len.dtype is i32 and free_pages.dtype is i32
            and block_table.dtype is i32 and cu_q.dtype is i32 and kv_len.dtype is i32
            and positions.dtype is i32 and slots.dtype is torch.int64 and counts.dtype is i32
            and ctx_len.is_contiguous() and new_len.is_contiguous() and free_pages.is_contiguous()
            and cu_q.is_contiguous() and kv_len.is_contiguous() and positions.is_contiguous()
            and slots.is_contiguous() and counts.is_contiguous()
            and ctx_len.dim() == 1 and new_len.shape == (B,) and cu_q.shape == (B + 1,) and kv_len.shape == (B,)
            and positions.shape == (max_tokens,) and slots.shape == (max_tokens,) and counts.shape == (4,)):
        _refuse(dev, ("ctx_len", ctx_len, i32, (B,), True), ("new_len", new_len, i32, (B,), True),
                ("free_pages", free_pages, i32, None, True), ("block_table", block_table, i32, None, False),
                ("cu_q", cu_q, i32, (B + 1,), True), ("kv_len", kv_len, i32, (B,), True),
                ("positions", positions, i32, (max_tokens,), True),
                ("slots", slots, torch.int64, (max_tokens,), True), ("counts", counts, i32, (4,), True))
    ts, stride = block_table.shape, block_table.stride()
    if len(ts) != 2 or ts[0] != B or ts[1] < 1 or (ts[1] > 1 and stride[1] != 1):
        raise FaError(f"block_table must be [{B}, max_pages] with contiguous rows")
    cp = 0
    if cursor is not None:
        _refuse(dev, ("cursor", cursor, i32, None, True))
        if cursor.numel() != 1:
            raise FaError("cursor must hold one number")
        cp = cursor.data_ptr()
    _call(dev, lib.fa_paged_plan_packed, _PLAN, ctx_len.data_ptr(), new_len.data_ptr(), free_pages.data_ptr(), cp,
          block_table.data_ptr(), cu_q.data_ptr(), kv_len.data_ptr(), positions.data_ptr(), counts.data_ptr(),
          slots.data_ptr(), _raw_stream(dev), stride[0], free_pages.numel(), B, ts[1], page_size, max_tokens, 0)
    return out


def _cache(dev: int, k_cache, v_cache, dtype, H_kv: int, d: int):
    """Checks of a paged cache pair [num_pages, H_kv, page_size, d]; (num_pages, page_size and the
    page strides)."""
    shape, ks, vs = k_cache.shape, k_cache.stride(), v_cache.stride()
    if k_cache.get_device() != dev or v_cache.get_device() != dev or k_cache.dtype is not dtype or \
            v_cache.dtype is not dtype or v_cache.shape != shape:
        _refuse(dev, ("k_cache", k_cache, dtype, None, False), ("v_cache", v_cache, dtype, shape, False))
    if len(shape) != 4 or shape[1] != H_kv or shape[3] != d:
        raise FaError(f"k_cache shape {tuple(shape)} must be [pages, {H_kv}, page_size, {d}]")
    page = shape[2]
    inner = (page * d, d, 1)
    if ks[1:] != inner or vs[1:] != inner:
        for n, st in (("k_cache", ks), ("v_cache", vs)):
            if st[3] != 1 or st[2] != d or (H_kv > 1 and st[1] != page * d):
                raise FaError(f"each page of {n} must be contiguous")
    return shape[0], page, ks[0], vs[0]


def paged_append(k, v, k_cache, v_cache, slots, positions=None, inv_freq=None,
                 interleaved: bool = False, magnitude: float = 1.0, q=None, q_out=None):
    """Stores k and v [T, H_kv, d] at their slots (int64 [T]) of the caches [pages, H_kv,
    page_size, d] (fa_paged_append); with inv_freq and positions (int32 [T]) the keys are rotated
    as ``rope`` does.  q [T, H, d] is rotated alongside into q_out (allocated when None; may be
    q), which is returned (None without q)."""
    lib = _lib or load()
    dev = k.get_device()
    dtype, shape = k.dtype, k.shape
    if dev < 0 or v.get_device() != dev or v.dtype is not dtype or v.shape != shape or \
            slots.get_device() != dev or slots.dtype is not torch.int64 or slots.shape != shape[:1] or \
            not slots.is_contiguous():
        _refuse(dev, ("k", k, None, None, False), ("v", v, dtype, shape, False),
                ("slots", slots, torch.int64, shape[:1], True))
    if len(shape) != 3:
        raise FaError(f"k {tuple(shape)} and v must both be [T, H_kv, d]")
    T, H_kv, d = shape
    pages, page, k_page, v_page = _cache(dev, k_cache, v_cache, dtype, H_kv, d)
    rot = pp = fp = 0
    if inv_freq is not None:
        if positions is None:
            raise FaError("inv_freq needs positions")
        if inv_freq.get_device() != dev or positions.get_device() != dev or \
                inv_freq.dtype is not torch.float64 or positions.dtype is not torch.int32 or \
                positions.shape != (T,) or not inv_freq.is_contiguous() or not positions.is_contiguous():
            _refuse(dev, ("inv_freq", inv_freq, torch.float64, None, True),
                    ("positions", positions, torch.int32, (T,), True))
        rot, pp, fp = 2 * inv_freq.numel(), positions.data_ptr(), inv_freq.data_ptr()
    ks, vs = k.stride(), v.stride()
    H, qp, qop, qs, qos = 0, 0, 0, (0, 0, 1), (0, 0, 1)
    if q is not None:
        qshape = q.shape
        if q_out is None:
            q_out = torch.empty(qshape, dtype=q.dtype, device=q.device)
        if q.get_device() != dev or q_out.get_device() != dev or q.dtype is not dtype or \
                q_out.dtype is not dtype or q_out.shape != qshape:
            _refuse(dev, ("q", q, dtype, None, False), ("q_out", q_out, dtype, qshape, False))
        if len(qshape) != 3 or qshape[0] != T or qshape[2] != d:
            raise FaError(f"q shape {tuple(qshape)} must be [{T}, H, {d}]")
        H, qp, qop, qs, qos = qshape[1], q.data_ptr(), q_out.data_ptr(), q.stride(), q_out.stride()
    elif q_out is not None:
        raise FaError("q_out without q")
    if d > 1 and (qs[2] != 1 or ks[2] != 1 or vs[2] != 1 or qos[2] != 1):
        raise FaError("the last dimension of q, k, v and q_out must be contiguous")
    _call(dev, lib.fa_paged_append_packed, _APPEND, qp, k.data_ptr(), v.data_ptr(), qop, k_cache.data_ptr(),
          v_cache.data_ptr(), slots.data_ptr(), pp, fp, _raw_stream(dev), qs[0], qs[1], ks[0], ks[1], vs[0], vs[1],
          qos[0], qos[1], k_page, v_page, T, H, H_kv, d, rot, page, pages,
          ROPE_INTERLEAVED if interleaved else 0, _dtype_code(k), magnitude)
    return q_out


def paged_workspace_size(T: int, B: int, H: int, H_kv: int, d: int) -> int:
    return int(load().fa_paged_workspace_size(T, B, H, H_kv, d))


def paged_fwd(q, k_cache, v_cache, block_table, kv_len, cu_q, scale: Optional[float] = None,
              causal: bool = True, max_q: Optional[int] = None, out=None, lse=None, workspace=None):
    """O, lse of each request's new tokens over its paged cache (fa_paged_fwd): q [T, H, d] (any
    token and head strides), caches [pages, H_kv, page_size, d], block_table int32
    [B, max_pages], kv_len int32 [B], cu_q int32 [B + 1].  O is [T, H, d], lse [T, H]; rows that
    no request owns are not written.  ``max_q``, the most new tokens of any request, helps to
    choose the kernel."""
    lib = _lib or load()
    dev = q.get_device()
    dtype, shape, qs, ts, stride = q.dtype, q.shape, q.stride(), block_table.shape, block_table.stride()
    if dev < 0:
        _refuse(dev, ("q", q, None, None, False))
    if len(shape) != 3:
        raise FaError(f"q must be [T, H, d], got {tuple(shape)}")
    T, H, d = shape
    if d > 1 and qs[2] != 1:
        raise FaError("the last dimension of q must be contiguous")
    if k_cache.dim() != 4:
        raise FaError("k_cache must be [pages, H_kv, page_size, d]")
    H_kv = k_cache.shape[1]
    pages, page, k_page, v_page = _cache(dev, k_cache, v_cache, dtype, H_kv, d)
    B = kv_len.numel()
    if len(ts) != 2 or ts[0] != B or (ts[1] > 1 and stride[1] != 1):
        raise FaError(f"block_table must be [{B}, max_pages] with contiguous rows")
    if out is None:
        out = torch.empty((T, H, d), dtype=dtype, device=q.device)
    if lse is None:
        lse = torch.empty((T, H), dtype=torch.float32, device=q.device)
    if workspace is None:
        workspace = torch.empty(paged_workspace_size(T, B, H, H_kv, d), dtype=torch.uint8, device=q.device)
    i32 = torch.int32
    if not (dev == kv_len.get_device() == cu_q.get_device() == block_table.get_device() == out.get_device()
            == lse.get_device() == workspace.get_device()
            and kv_len.dtype is i32 and cu_q.dtype is i32 and block_table.dtype is i32 and out.dtype is dtype
            and lse.dtype is torch.float32 and workspace.dtype is torch.uint8
            and kv_len.dim() == 1 and cu_q.shape == (B + 1,) and out.shape == shape and lse.shape == shape[:2]
            and kv_len.is_contiguous() and cu_q.is_contiguous() and out.is_contiguous()
            and lse.is_contiguous() and workspace.is_contiguous()):
        _refuse(dev, ("kv_len", kv_len, i32, (B,), True), ("cu_q", cu_q, i32, (B + 1,), True),
                ("block_table", block_table, i32, None, False), ("out", out, dtype, shape, True),
                ("lse", lse, torch.float32, shape[:2], True), ("workspace", workspace, torch.uint8, None, True))
    _call(dev, lib.fa_paged_fwd_packed, _FWD, q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
          block_table.data_ptr(), kv_len.data_ptr(), cu_q.data_ptr(), out.data_ptr(), lse.data_ptr(),
          workspace.data_ptr(), _raw_stream(dev), workspace.numel(), qs[0], qs[1], k_page, v_page, stride[0], T, B,
          H, H_kv, d, page, pages, ts[1], 0 if max_q is None else max_q, 1 if causal else 0, _dtype_code(q),
          default_scale(d) if scale is None else scale)
    return out, lse


TILE_REVERSE = 1          # fa.h FA_TILE_REVERSE: key tiles visited last to first
TILE_L_ROUNDED = 2        # fa.h FA_TILE_L_ROUNDED: l sums the bf16-rounded P
TILE_TENSOR_CORE = 4      # fa.h FA_TILE_TENSOR_CORE: the tcgen05 forward with bc-key tiles
TILE_O_F32 = 8            # fa.h FA_TILE_O_F32: fp32 O/l before its bf16 rounding


def fwd_tile_reference(q, k, v, bc: int, scale: Optional[float] = None, causal: bool = False,
                       block_mask=None, kv_len=None, reverse: bool = False,
                       l_rounded: bool = False, tensor_core: bool = False, o_f32: bool = False):
    """bf16 forward that rescales after every `bc` keys (deviation study): the CUDA-core
    reference (`reverse` visits the key tiles last to first, `l_rounded` sums l over the
    bf16-rounded P) or, with `tensor_core`, the tcgen05 forward with bc-key tiles (d = 64,
    bc 64 or 128).  `o_f32` returns the fp32 O/l before its bf16 rounding."""
    lib = load()
    B, H, N, d = q.shape
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _require(t, n, torch.bfloat16)
    o = torch.empty(q.shape, dtype=torch.float32 if o_f32 else torch.bfloat16, device=q.device)
    l = torch.empty((B, H, N), dtype=torch.float32, device=q.device)
    bm, kl = _masks(block_mask, kv_len)
    s = default_scale(d) if scale is None else float(scale)
    flags = ((TILE_REVERSE if reverse else 0) | (TILE_L_ROUNDED if l_rounded else 0) |
             (TILE_TENSOR_CORE if tensor_core else 0) | (TILE_O_F32 if o_f32 else 0))
    rc = lib.fa_fwd_tile_reference(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(l), B, H, N, d, s,
                                   int(causal), bm, kl, int(bc), flags, _stream())
    _check(rc, "fa_fwd_tile_reference")
    return o, l


def naive_fwd(q, k, v, scale: Optional[float] = None, causal: bool = False, block_mask=None,
              kv_len=None, workspace=None):
    """Materialised baseline: S and P go through HBM in bf16."""
    lib = load()
    B, H, N, d = q.shape
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _require(t, n, torch.bfloat16)
    need = int(lib.fa_naive_workspace_size(B, H, N))
    ws = torch.empty(need, dtype=torch.uint8, device=q.device) if workspace is None else workspace
    o = torch.empty_like(q)
    l = torch.empty((B, H, N), dtype=torch.float32, device=q.device)
    bm, kl = _masks(block_mask, kv_len)
    s = default_scale(d) if scale is None else float(scale)
    rc = lib.fa_naive_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(l), B, H, N, d, s,
                          int(causal), bm, kl, _ptr(ws), ws.numel(), _stream())
    _check(rc, "fa_naive_fwd")
    return o, l


def diag_exp2(x):
    """(FMA-pipe 2^x, ex2.approx, exp2f) of a float32 CUDA tensor; diagnostic only."""
    lib = load()
    _require(x, "x", torch.float32)
    y = [torch.empty_like(x) for _ in range(3)]
    rc = lib.fa_diag_exp2(_ptr(x), _ptr(y[0]), _ptr(y[1]), _ptr(y[2]), x.numel(), _stream())
    _check(rc, "fa_diag_exp2")
    return tuple(y)


def diag_wait_timeout(site: int):
    """Launch the bounded-wait diagnostic (gives up after ~2 s); read it with device_status()."""
    _check(load().fa_diag_wait_timeout(int(site), _stream()), "fa_diag_wait_timeout")


def device_status() -> int:
    """Synchronise; return the bounded-wait status code (0 = no wait gave up) and clear it."""
    code = ctypes.c_uint(0)
    rc = load().fa_device_status(ctypes.byref(code))
    if rc not in (0, -5):
        _check(rc, "fa_device_status")
    return int(code.value)


def launch_count() -> int:
    """Kernels this library has launched in the process (fa_launch_count)."""
    return int(load().fa_launch_count())


def kernel_timing(enable: bool):
    """Start (True) or stop (False) bracketing each tensor-core launch with CUDA events."""
    _check(load().fa_kernel_timing(int(bool(enable))), "fa_kernel_timing")


def kernel_timing_read(name: str = ""):
    """(launches, total ms) of the recorded launches of kernels whose name contains ``name``;
    waits for them and forgets them."""
    n = ctypes.c_int(0)
    ms = ctypes.c_double(0.0)
    _check(load().fa_kernel_timing_read(name.encode(), ctypes.byref(n), ctypes.byref(ms)),
           "fa_kernel_timing_read")
    return int(n.value), float(ms.value)
