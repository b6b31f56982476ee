"""Exact training attention (forward O, L and backward dQ, dK, dV) on one GB300.

Thin Python binding of the C-ABI library `libfa_gb300.so` (declared in include/fa_train.h).
This module only marshals arguments: PyTorch provides device memory and streams, and every
step of the computation runs in the library's sm_103a kernels. There is no fallback: if the
library is missing or was not built for this GPU, the calls raise.
"""
from __future__ import annotations

import ctypes
import os
import threading

from .build import LIB_PATH, build

__all__ = [
    "FaParams", "fa_train_fwd", "fa_train_bwd", "fa_device_status", "fa_error_string",
    "fa_version", "fa_profile_enable", "fa_profile_read", "attention_fwd", "attention_bwd", "load_library", "build", "LIB_PATH",
    "FA_OK", "FA_ERR_INVALID", "FA_ERR_CUDA", "FA_ERR_DEVICE_TIMEOUT", "FA_ERR_UNSUPPORTED",
    "FA_ERR_TOO_LARGE", "FA_ERR_BAD_INPUT", "FaOptions", "FaPagedParams", "paged_attention",
    "fa_paged_attention", "fa_paged_attention_bwd", "fa_train_fwd_ex", "fa_train_bwd_ex", "make_options",
    "FA_MASK_F32", "FA_MASK_BF16", "FA_MASK_BOOL", "FaQ8Cache", "FaQ8Rows", "make_q8_cache",
    "q8_cache_write", "q8_cache_read", "q8_paged_attention",
]

FA_OK = 0
FA_ERR_INVALID = 1
FA_ERR_CUDA = 2
FA_ERR_DEVICE_TIMEOUT = 3
FA_ERR_UNSUPPORTED = 4
FA_ERR_TOO_LARGE = 5
FA_ERR_BAD_INPUT = 6


FA_MASK_F32 = 0
FA_MASK_BF16 = 1
FA_MASK_BOOL = 2
FA_LAYOUT_Q_BSHD = 1   # q, o, dO, dq as [batch, seq, heads, dim] in memory
FA_LAYOUT_KV_BSHD = 2  # k, v, dk, dv as [batch, seq, kv_heads, dim] in memory


class FaOptions(ctypes.Structure):
    """Mirror of `fa_options` in include/fa_train.h."""

    _fields_ = [
        ("window_left", ctypes.c_int32),
        ("window_right", ctypes.c_int32),
        ("mask_type", ctypes.c_int32),
        ("value_dim", ctypes.c_int32),
        ("mask_stride_b", ctypes.c_int64),
        ("mask_stride_h", ctypes.c_int64),
        ("mask_stride_q", ctypes.c_int64),
        ("sinks", ctypes.c_void_p),
        ("dsinks", ctypes.c_void_p),
        ("deterministic", ctypes.c_int32),
        ("layout", ctypes.c_int32),
        ("cu_seqlens_q", ctypes.c_void_p),
        ("cu_seqlens_k", ctypes.c_void_p),
        ("total_q", ctypes.c_int32),
        ("total_k", ctypes.c_int32),
    ]


class FaPagedParams(ctypes.Structure):
    """Mirror of `fa_paged_params` in include/fa_train.h."""

    _fields_ = [
        ("batch", ctypes.c_int32),
        ("n_heads", ctypes.c_int32),
        ("n_kv_heads", ctypes.c_int32),
        ("q_len", ctypes.c_int32),
        ("head_dim", ctypes.c_int32),
        ("page_size", ctypes.c_int32),
        ("max_pages", ctypes.c_int32),
        ("num_pages", ctypes.c_int32),
        ("scale", ctypes.c_float),
        ("causal", ctypes.c_int32),
        ("num_splits", ctypes.c_int32),
        ("reserved", ctypes.c_int32),
    ]


class FaParams(ctypes.Structure):
    """Mirror of `fa_params` in include/fa_train.h."""

    _fields_ = [
        ("batch", ctypes.c_int32),
        ("n_heads", ctypes.c_int32),
        ("n_kv_heads", ctypes.c_int32),
        ("ql", ctypes.c_int32),
        ("kl", ctypes.c_int32),
        ("head_dim", ctypes.c_int32),
        ("scale", ctypes.c_float),
        ("causal", ctypes.c_int32),
    ]


class FaQ8Cache(ctypes.Structure):
    """Mirror of `fa_q8_cache` in include/fa_train.h."""

    _fields_ = [
        ("k", ctypes.c_void_p),
        ("v", ctypes.c_void_p),
        ("k_scale", ctypes.c_void_p),
        ("v_scale", ctypes.c_void_p),
        ("num_pages", ctypes.c_int32),
        ("n_kv_heads", ctypes.c_int32),
        ("page_size", ctypes.c_int32),
        ("head_dim", ctypes.c_int32),
        ("scale_block", ctypes.c_int32),
        ("reserved", ctypes.c_int32),
    ]


class FaQ8Rows(ctypes.Structure):
    """Mirror of `fa_q8_rows` in include/fa_train.h."""

    _fields_ = [
        ("k", ctypes.c_void_p),
        ("v", ctypes.c_void_p),
        ("k_stride", ctypes.c_int64 * 3),
        ("v_stride", ctypes.c_int64 * 3),
        ("cu_seqlens", ctypes.c_void_p),
        ("block_table", ctypes.c_void_p),
        ("lengths", ctypes.c_void_p),
        ("batch", ctypes.c_int32),
        ("max_pages", ctypes.c_int32),
        ("total", ctypes.c_int32),
        ("new_len", ctypes.c_int32),
    ]


_lib = None
_lock = threading.Lock()


class FaError(RuntimeError):
    def __init__(self, code, where):
        lib = load_library()
        text = lib.fa_error_string(code).decode()
        cuda = lib.fa_last_cuda_error().decode() if code == FA_ERR_CUDA else ""
        super().__init__(f"{where}: {text}" + (f" [{cuda}]" if cuda else ""))
        self.code = code


def load_library():
    """Load libfa_gb300.so (it must have been built: `flash_attention_gb300.build()`)."""
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(
                    f"{LIB_PATH} is missing: build the CUDA library first "
                    "(python -c 'import flash_attention_gb300 as f; f.build()')")
            lib = ctypes.CDLL(LIB_PATH)
            vp, fp = ctypes.c_void_p, ctypes.c_void_p
            pp = ctypes.POINTER(FaParams)
            lib.fa_train_fwd.argtypes = [vp, vp, vp, fp, vp, fp, pp, vp]
            lib.fa_train_fwd.restype = ctypes.c_int
            lib.fa_train_bwd.argtypes = [vp, vp, vp, vp, fp, vp, fp, vp, vp, vp, pp, vp]
            lib.fa_train_bwd.restype = ctypes.c_int
            po = ctypes.POINTER(FaOptions)
            lib.fa_train_fwd_ex.argtypes = [vp, vp, vp, vp, vp, fp, pp, po, vp]
            lib.fa_train_fwd_ex.restype = ctypes.c_int
            lib.fa_train_bwd_ex.argtypes = [vp, vp, vp, vp, fp, vp, vp, vp, vp, vp, pp, po, vp]
            lib.fa_train_bwd_ex.restype = ctypes.c_int
            lib.fa_paged_attention.argtypes = [vp, vp, vp, vp, vp, vp, fp, vp, vp]
            lib.fa_paged_attention.restype = ctypes.c_int
            lib.fa_paged_attention_bwd.argtypes = [vp, vp, vp, vp, vp, vp, fp, vp, vp, vp, vp,
                                                   vp, vp]
            lib.fa_paged_attention_bwd.restype = ctypes.c_int
            pc, pr = ctypes.POINTER(FaQ8Cache), ctypes.POINTER(FaQ8Rows)
            lib.fa_q8_cache_write.argtypes = [pc, pr, vp]
            lib.fa_q8_cache_write.restype = ctypes.c_int
            lib.fa_q8_cache_read.argtypes = [pc, pr, vp]
            lib.fa_q8_cache_read.restype = ctypes.c_int
            lib.fa_q8_paged_attention.argtypes = [vp, pc, vp, vp, vp, vp,
                                                  ctypes.POINTER(FaPagedParams), vp]
            lib.fa_q8_paged_attention.restype = ctypes.c_int
            lib.fa_device_status.argtypes = [ctypes.c_int]
            lib.fa_device_status.restype = ctypes.c_int
            lib.fa_error_string.argtypes = [ctypes.c_int]
            lib.fa_error_string.restype = ctypes.c_char_p
            lib.fa_last_cuda_error.restype = ctypes.c_char_p
            lib.fa_version.restype = ctypes.c_char_p
            lib.fa_profile_enable.argtypes = [ctypes.c_int]
            lib.fa_profile_enable.restype = ctypes.c_int
            lib.fa_profile_read.argtypes = [ctypes.POINTER(ctypes.c_double),
                                            ctypes.POINTER(ctypes.c_int64)]
            lib.fa_profile_read.restype = ctypes.c_int
            lib.fa_kernel_name.argtypes = [ctypes.c_int]
            lib.fa_kernel_name.restype = ctypes.c_char_p
            lib.fa_train_bwd_noalloc.argtypes = [vp, vp, vp, vp, fp, vp, fp, vp, vp, vp, pp, vp]
            lib.fa_train_bwd_noalloc.restype = ctypes.c_int
            lib.fa_set_wait_limit_ns.argtypes = [ctypes.c_uint64]
            lib.fa_set_wait_limit_ns.restype = ctypes.c_int
            lib.fa_get_wait_limit_ns.argtypes = []
            lib.fa_get_wait_limit_ns.restype = ctypes.c_uint64
            lib.fa_debug_ex2.argtypes = [vp, vp, vp, vp, ctypes.c_int64, vp]
            lib.fa_debug_ex2.restype = ctypes.c_int
            lib.fa_debug_wait_timeout.argtypes = [vp, vp]
            lib.fa_debug_wait_timeout.restype = ctypes.c_int
            _lib = lib
    return _lib


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream_handle(stream):
    if stream is None:
        import torch

        stream = torch.cuda.current_stream()
    h = getattr(stream, "cuda_stream", stream)
    return ctypes.c_void_p(int(h))


def make_params(q, k, *, scale, causal) -> FaParams:
    B, H, ql, d = q.shape
    Bk, Hk, kl, dk = k.shape
    if B != Bk or d != dk:
        raise ValueError("q and k disagree on batch or head_dim")
    return FaParams(B, H, Hk, ql, kl, d, float(scale), int(bool(causal)))


def _check(t, dtype, name):
    import torch

    if t.dtype != dtype or not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous CUDA {dtype} tensor")


def _layout_bit(t) -> int:
    """0 if `t` ([..., heads, rows, dim]) is contiguous, 1 if it is the transposed view of a
    contiguous [..., rows, heads, dim] tensor (the memory layout the FA_LAYOUT_* flags name)."""
    if t.is_contiguous():
        return 0
    if t.transpose(-3, -2).is_contiguous():
        return 1
    raise ValueError("a [.., heads, rows, dim] tensor must be contiguous or a transposed view of "
                     "a contiguous [.., rows, heads, dim] tensor")


def _check_bf16(t, bshd, name):
    import torch

    if t.dtype != torch.bfloat16 or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA bfloat16 tensor")
    ok = t.transpose(-3, -2).is_contiguous() if bshd else t.is_contiguous()
    if not ok:
        raise ValueError(f"{name} must be laid out as " +
                         ("[.., rows, heads, dim]" if bshd else "[.., heads, rows, dim]"))


def _check_sides(options, q_side, kv_side):
    """Checks the q-side (q, o, dO, dq) and kv-side (k, v, dk, dv) tensors against the layout
    flags of `options`."""
    for t, n in q_side:
        _check_bf16(t, options.layout & FA_LAYOUT_Q_BSHD, n)
    for t, n in kv_side:
        _check_bf16(t, options.layout & FA_LAYOUT_KV_BSHD, n)


def fa_train_fwd(q, k, v, mask, o, lse, params: FaParams, stream=None) -> None:
    """C call `fa_train_fwd` on torch tensors (q, k, v, o bf16; mask, lse f32)."""
    import torch

    for t, n in ((q, "q"), (k, "k"), (v, "v"), (o, "o")):
        _check(t, torch.bfloat16, n)
    _check(lse, torch.float32, "lse")
    if mask is not None:
        _check(mask, torch.float32, "mask")
    rc = load_library().fa_train_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(mask), _ptr(o), _ptr(lse),
                                     ctypes.byref(params), _stream_handle(stream))
    if rc:
        raise FaError(rc, "fa_train_fwd")


def fa_train_bwd(q, k, v, o, lse, dO, mask, dq, dk, dv, params: FaParams, stream=None) -> None:
    """C call `fa_train_bwd` on torch tensors."""
    import torch

    for t, n in ((q, "q"), (k, "k"), (v, "v"), (o, "o"), (dO, "dO"), (dq, "dq"), (dk, "dk"),
                 (dv, "dv")):
        _check(t, torch.bfloat16, n)
    _check(lse, torch.float32, "lse")
    if mask is not None:
        _check(mask, torch.float32, "mask")
    rc = load_library().fa_train_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(dO),
                                     _ptr(mask), _ptr(dq), _ptr(dk), _ptr(dv),
                                     ctypes.byref(params), _stream_handle(stream))
    if rc:
        raise FaError(rc, "fa_train_bwd")


def make_options(q, k, mask=None, window=(-1, -1), v=None, sinks=None, dsinks=None,
                 deterministic=False) -> FaOptions:
    """fa_options for a mask tensor of any supported dtype (float32, bfloat16, bool) whose shape
    broadcasts to [B, H, ql, kl] with the keys contiguous, a (left, right) window, the value
    head dim of `v` (when it differs from q's), float32 [H] sinks / dsinks tensors, the
    deterministic backward, and the memory layouts of q and k (contiguous, or transposed views
    of [B, seq, heads, dim] tensors)."""
    import torch

    B, H, ql, d = q.shape
    kl = k.shape[2]
    wl, wr = window if window is not None else (-1, -1)
    layout = FA_LAYOUT_Q_BSHD * _layout_bit(q) | FA_LAYOUT_KV_BSHD * _layout_bit(k)
    opt = FaOptions(int(wl), int(wr), FA_MASK_F32, 0, 0, 0, 0, None, None,
                    1 if deterministic else 0, layout, None, None, 0, 0)
    if v is not None and v.shape[-1] != d:
        opt.value_dim = int(v.shape[-1])
    if mask is not None:
        types = {torch.float32: FA_MASK_F32, torch.bfloat16: FA_MASK_BF16, torch.bool: FA_MASK_BOOL,
                 torch.uint8: FA_MASK_BOOL}
        if mask.dtype not in types or not mask.is_cuda:
            raise ValueError("mask must be a CUDA float32, bfloat16 or bool tensor")
        e = mask.expand(B, H, ql, kl)
        sb, sh, sq, sk = e.stride()
        if kl > 1 and sk != 1:
            raise ValueError("the mask's key dimension must be contiguous")
        opt.mask_type = types[mask.dtype]
        opt.mask_stride_b, opt.mask_stride_h, opt.mask_stride_q = sb, sh, sq
    for name, t in (("sinks", sinks), ("dsinks", dsinks)):
        if t is None:
            continue
        if t.dtype != torch.float32 or not t.is_cuda or tuple(t.shape) != (H,) or \
                not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous CUDA float32 tensor of shape [{H}]")
        setattr(opt, name, t.data_ptr())
    return opt


def fa_train_fwd_ex(q, k, v, mask, o, lse, params: FaParams, options: FaOptions,
                    stream=None) -> None:
    """C call `fa_train_fwd_ex` (window, mask type and broadcast in `options`)."""
    import torch

    _check_sides(options, ((q, "q"), (o, "o")), ((k, "k"), (v, "v")))
    _check(lse, torch.float32, "lse")
    rc = load_library().fa_train_fwd_ex(_ptr(q), _ptr(k), _ptr(v), _ptr(mask), _ptr(o), _ptr(lse),
                                        ctypes.byref(params), ctypes.byref(options),
                                        _stream_handle(stream))
    if rc:
        raise FaError(rc, "fa_train_fwd_ex")


def fa_train_bwd_ex(q, k, v, o, lse, dO, mask, dq, dk, dv, params: FaParams, options: FaOptions,
                    stream=None) -> None:
    """C call `fa_train_bwd_ex`."""
    import torch

    _check_sides(options, ((q, "q"), (o, "o"), (dO, "dO"), (dq, "dq")),
                 ((k, "k"), (v, "v"), (dk, "dk"), (dv, "dv")))
    _check(lse, torch.float32, "lse")
    rc = load_library().fa_train_bwd_ex(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(dO),
                                        _ptr(mask), _ptr(dq), _ptr(dk), _ptr(dv),
                                        ctypes.byref(params), ctypes.byref(options),
                                        _stream_handle(stream))
    if rc:
        raise FaError(rc, "fa_train_bwd_ex")


def fa_device_status(clear: bool = True) -> int:
    return load_library().fa_device_status(int(bool(clear)))


FA_NUM_KERNELS = 14


def fa_profile_enable(on: bool) -> None:
    load_library().fa_profile_enable(int(bool(on)))


def fa_profile_read():
    """{kernel name: (total device ms, launches)} since the last read (then cleared)."""
    lib = load_library()
    ms = (ctypes.c_double * FA_NUM_KERNELS)()
    n = (ctypes.c_int64 * FA_NUM_KERNELS)()
    rc = lib.fa_profile_read(ms, n)
    if rc:
        raise FaError(rc, "fa_profile_read")
    return {lib.fa_kernel_name(k).decode(): (ms[k], n[k]) for k in range(FA_NUM_KERNELS)}


def fa_error_string(code: int) -> str:
    return load_library().fa_error_string(int(code)).decode()


def fa_version() -> str:
    return load_library().fa_version().decode()


def fa_train_bwd_noalloc(q, k, v, o, lse, dO, mask, dq, dk, dv, params: FaParams,
                         stream=None) -> None:
    """C call `fa_train_bwd_noalloc` (the backward with its scratch in the library's fixed
    device array; no allocation)."""
    import torch

    for t, n in ((q, "q"), (k, "k"), (v, "v"), (o, "o"), (dO, "dO"), (dq, "dq"), (dk, "dk"),
                 (dv, "dv")):
        _check(t, torch.bfloat16, n)
    _check(lse, torch.float32, "lse")
    if mask is not None:
        _check(mask, torch.float32, "mask")
    rc = load_library().fa_train_bwd_noalloc(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse),
                                             _ptr(dO), _ptr(mask), _ptr(dq), _ptr(dk), _ptr(dv),
                                             ctypes.byref(params), _stream_handle(stream))
    if rc:
        raise FaError(rc, "fa_train_bwd_noalloc")


def fa_set_wait_limit_ns(ns: int) -> None:
    """Limit of one barrier wait in the kernels launched from now on (0: the default 2 s)."""
    rc = load_library().fa_set_wait_limit_ns(int(ns))
    if rc:
        raise FaError(rc, "fa_set_wait_limit_ns")


def fa_get_wait_limit_ns() -> int:
    return int(load_library().fa_get_wait_limit_ns())


def fa_debug_ex2(x, stream=None):
    """The softmax's two exp2 forms and CUDA's exp2f on a CUDA float32 tensor:
    (polynomial, hardware approximation, exp2f)."""
    import torch

    _check(x, torch.float32, "x")
    outs = [torch.empty_like(x) for _ in range(3)]
    rc = load_library().fa_debug_ex2(_ptr(x), *(_ptr(t) for t in outs), x.numel(),
                                     _stream_handle(stream))
    if rc:
        raise FaError(rc, "fa_debug_ex2")
    return tuple(outs)


def fa_debug_wait_timeout(stream=None):
    """Launches the kernel that waits on a barrier nothing completes; returns a CUDA int64
    tensor that receives how long it waited (ns)."""
    import torch

    waited = torch.zeros(1, dtype=torch.int64, device="cuda")
    rc = load_library().fa_debug_wait_timeout(_ptr(waited), _stream_handle(stream))
    if rc:
        raise FaError(rc, "fa_debug_wait_timeout")
    return waited


def _plain_call(q, k, v, mask, window, sinks):
    """True when the base entry point covers the call (dense f32 mask or none, no window, no
    sinks, value head dim = head dim)."""
    import torch

    B, H, ql, d = q.shape
    dense = mask is None or (mask.dtype == torch.float32 and mask.dim() == 4
                             and mask.is_contiguous()
                             and tuple(mask.shape) == (B, H, ql, k.shape[2]))
    contiguous = q.is_contiguous() and k.is_contiguous() and v.is_contiguous()
    return dense and contiguous and window is None and sinks is None and v.shape[-1] == d


def attention_fwd(q, k, v, *, scale, causal, mask=None, window=None, sinks=None, stream=None):
    """Allocate O and L and run the forward: returns (o, lse). `mask`: None, or a float32 /
    bfloat16 additive or bool mask broadcastable to [B, H, ql, kl]; `window`: None or
    (left, right) with -1 for an unbounded side; `sinks`: None or float32 [H] logits. v may
    have its own head dim (o then has it too)."""
    import torch

    B, H, ql, d = q.shape
    if _layout_bit(q):  # o in q's layout
        o = torch.empty((B, ql, H, v.shape[-1]), dtype=q.dtype, device=q.device).transpose(1, 2)
    else:
        o = torch.empty((B, H, ql, v.shape[-1]), dtype=q.dtype, device=q.device)
    lse = torch.empty((B, H, ql), dtype=torch.float32, device=q.device)
    params = make_params(q, k, scale=scale, causal=causal)
    if _plain_call(q, k, v, mask, window, sinks):
        fa_train_fwd(q, k, v, mask, o, lse, params, stream)
    else:
        fa_train_fwd_ex(q, k, v, mask, o, lse, params,
                        make_options(q, k, mask, window, v=v, sinks=sinks), stream)
    return o, lse


def attention_bwd(q, k, v, o, lse, dO, *, scale, causal, mask=None, window=None, sinks=None,
                  deterministic=False, stream=None):
    """Allocate dQ, dK, dV and run the backward: returns (dq, dk, dv), or (dq, dk, dv, dsinks)
    when `sinks` is given. `mask`, `window` and `sinks` as given to attention_fwd;
    `deterministic` makes every output bitwise reproducible (dQ from its own kernel)."""
    import torch

    dq = torch.empty_like(q)
    dk = torch.empty_like(k)
    dv = torch.empty_like(v)
    params = make_params(q, k, scale=scale, causal=causal)
    if _plain_call(q, k, v, mask, window, sinks) and not deterministic:
        fa_train_bwd(q, k, v, o, lse, dO, mask, dq, dk, dv, params, stream)
        return dq, dk, dv
    dsinks = None if sinks is None else torch.empty_like(sinks)
    fa_train_bwd_ex(q, k, v, o, lse, dO, mask, dq, dk, dv, params,
                    make_options(q, k, mask, window, v=v, sinks=sinks, dsinks=dsinks,
                                 deterministic=deterministic), stream)
    return (dq, dk, dv) if sinks is None else (dq, dk, dv, dsinks)


def fa_paged_attention(q, k_cache, v_cache, block_table, lengths, o, lse, params: FaPagedParams,
                       stream=None) -> None:
    """C call `fa_paged_attention` (q, caches, o bf16; block_table, lengths int32; lse f32 or
    None)."""
    import torch

    for t, n in ((q, "q"), (k_cache, "k_cache"), (v_cache, "v_cache"), (o, "o")):
        _check(t, torch.bfloat16, n)
    _check(block_table, torch.int32, "block_table")
    _check(lengths, torch.int32, "lengths")
    if lse is not None:
        _check(lse, torch.float32, "lse")
    rc = load_library().fa_paged_attention(_ptr(q), _ptr(k_cache), _ptr(v_cache),
                                           _ptr(block_table), _ptr(lengths), _ptr(o), _ptr(lse),
                                           ctypes.byref(params), _stream_handle(stream))
    if rc:
        raise FaError(rc, "fa_paged_attention")


def paged_attention(q, k_cache, v_cache, block_table, lengths, *, scale, causal=True,
                    num_splits=0, stream=None):
    """Attention of q [B, H, q_len, d] over paged caches [num_pages, Hk, page_size, d] with a
    block table [B, max_pages] and lengths [B] (int32, on the device): returns (o, lse). The
    q_len queries are each sequence's last positions (causal: bottom-right per sequence)."""
    import torch

    B, H, lq, d = q.shape
    P, Hk, bs, _ = k_cache.shape
    params = FaPagedParams(B, H, Hk, lq, d, bs, block_table.shape[1], P, float(scale),
                           int(bool(causal)), int(num_splits), 0)
    o = torch.empty_like(q)
    lse = torch.empty((B, H, lq), dtype=torch.float32, device=q.device)
    fa_paged_attention(q, k_cache, v_cache, block_table, lengths, o, lse, params, stream)
    return o, lse


def fa_paged_attention_bwd(q, k_cache, v_cache, block_table, lengths, o, lse, dO, dq, dk_cache,
                           dv_cache, params: FaPagedParams, stream=None) -> None:
    """C call `fa_paged_attention_bwd` (gradients for q and both caches)."""
    import torch

    for t, n in ((q, "q"), (k_cache, "k_cache"), (v_cache, "v_cache"), (o, "o"), (dO, "dO"),
                 (dq, "dq"), (dk_cache, "dk_cache"), (dv_cache, "dv_cache")):
        _check(t, torch.bfloat16, n)
    _check(block_table, torch.int32, "block_table")
    _check(lengths, torch.int32, "lengths")
    _check(lse, torch.float32, "lse")
    rc = load_library().fa_paged_attention_bwd(
        _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_table), _ptr(lengths), _ptr(o),
        _ptr(lse), _ptr(dO), _ptr(dq), _ptr(dk_cache), _ptr(dv_cache), ctypes.byref(params),
        _stream_handle(stream))
    if rc:
        raise FaError(rc, "fa_paged_attention_bwd")


def paged_attention_bwd(q, k_cache, v_cache, block_table, lengths, o, lse, dO, *, scale,
                        causal=True, stream=None):
    """Gradients of paged_attention: returns (dq, dk_cache, dv_cache), the cache gradients
    shaped like the caches (0 in every slot no sequence reads)."""
    import torch

    B, H, lq, d = q.shape
    P, Hk, bs, _ = k_cache.shape
    params = FaPagedParams(B, H, Hk, lq, d, bs, block_table.shape[1], P, float(scale),
                           int(bool(causal)), 0, 0)
    dq = torch.empty_like(q)
    dk = torch.empty_like(k_cache)
    dv = torch.empty_like(v_cache)
    fa_paged_attention_bwd(q, k_cache, v_cache, block_table, lengths, o, lse, dO, dq, dk, dv,
                           params, stream)
    return dq, dk, dv


def varlen_params_options(q, k, v, cu_q, cu_k, max_q, max_k, *, scale, causal, window=None,
                          sinks=None, dsinks=None, deterministic=False):
    """FaParams and FaOptions of a variable-length batch: q [H, total_q, d], k and v
    [Hk, total_k, d(v)], cu_q / cu_k int32 CUDA tensors of batch + 1 offsets, max_q / max_k the
    longest sequence."""
    import torch

    H, Tq, d = q.shape
    Hk, Tk, _ = k.shape
    for t, n in ((cu_q, "cu_q"), (cu_k, "cu_k")):
        _check(t, torch.int32, n)
    B = cu_q.numel() - 1
    params = FaParams(B, H, Hk, int(max_q), int(max_k), d, float(scale), int(bool(causal)))
    opt = make_options(q[None], k[None], None, window, v=v[None], sinks=sinks, dsinks=dsinks,
                       deterministic=deterministic)
    opt.cu_seqlens_q = cu_q.data_ptr()
    opt.cu_seqlens_k = cu_k.data_ptr()
    opt.total_q, opt.total_k = Tq, Tk
    return params, opt


def varlen_attention_fwd(q, k, v, cu_q, cu_k, max_q, max_k, *, scale, causal, window=None,
                         sinks=None, stream=None):
    """Forward of a variable-length batch (see varlen_params_options): returns (o, lse) with
    o [H, total_q, dv] and lse [H, total_q]."""
    import torch

    H, Tq, _ = q.shape
    if _layout_bit(q):  # o in q's layout: [total_q, H, dv] memory
        o = torch.empty((Tq, H, v.shape[2]), dtype=q.dtype, device=q.device).transpose(0, 1)
    else:
        o = torch.empty((H, Tq, v.shape[2]), dtype=q.dtype, device=q.device)
    lse = torch.empty((H, Tq), dtype=torch.float32, device=q.device)
    params, opt = varlen_params_options(q, k, v, cu_q, cu_k, max_q, max_k, scale=scale,
                                        causal=causal, window=window, sinks=sinks)
    fa_train_fwd_ex(q, k, v, None, o, lse, params, opt, stream)
    return o, lse


def varlen_attention_bwd(q, k, v, o, lse, dO, cu_q, cu_k, max_q, max_k, *, scale, causal,
                         window=None, sinks=None, deterministic=False, stream=None):
    """Backward of a variable-length batch: returns (dq, dk, dv) (+ dsinks with sinks)."""
    import torch

    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    dsinks = None if sinks is None else torch.empty_like(sinks)
    params, opt = varlen_params_options(q, k, v, cu_q, cu_k, max_q, max_k, scale=scale,
                                        causal=causal, window=window, sinks=sinks,
                                        dsinks=dsinks, deterministic=deterministic)
    fa_train_bwd_ex(q, k, v, o, lse, dO, None, dq, dk, dv, params, opt, stream)
    return (dq, dk, dv) if sinks is None else (dq, dk, dv, dsinks)


# ----------------------------------------------------------------- 8-bit key/value cache
def make_q8_cache(num_pages, n_kv_heads, page_size, head_dim, scale_block=None, device="cuda"):
    """An empty 8-bit paged cache: (k_cache, v_cache, k_scale, v_scale), codes float8_e4m3fn
    [num_pages, Hk, page_size, d] and float32 scales [num_pages, Hk, page_size // scale_block]
    (by default one scale for each page and head)."""
    import torch

    block = page_size if scale_block is None else int(scale_block)
    if block < 1 or page_size % block:
        raise ValueError("scale_block must divide page_size")
    codes = [torch.zeros((num_pages, n_kv_heads, page_size, head_dim), dtype=torch.uint8,
                         device=device).view(torch.float8_e4m3fn) for _ in range(2)]
    scales = [torch.ones((num_pages, n_kv_heads, page_size // block), dtype=torch.float32,
                         device=device) for _ in range(2)]
    return (*codes, *scales)


# These calls are short (a decoding step's take microseconds), so their checks are written to cost
# little where they pass.
def _q8_cache(k, v, ks, vs, torch) -> FaQ8Cache:
    shape, blocks = k.shape, ks.shape
    if not (k.dtype is v.dtype is torch.float8_e4m3fn and len(shape) == 4 and v.shape == shape):
        raise ValueError("k_cache and v_cache must be float8_e4m3fn [num_pages, Hk, page_size, d]")
    P, Hk, ps, d = shape
    if not (ks.dtype is vs.dtype is torch.float32 and len(blocks) == 3 and vs.shape == blocks
            and blocks[0] == P and blocks[1] == Hk and blocks[2] > 0 and ps % blocks[2] == 0):
        raise ValueError("k_scale and v_scale must be float32 "
                         "[num_pages, Hk, page_size // scale_block]")
    if not (k.is_contiguous() and v.is_contiguous() and ks.is_contiguous()
            and vs.is_contiguous()):
        raise ValueError("the cache's tensors must be contiguous")
    return FaQ8Cache(k.data_ptr(), v.data_ptr(), ks.data_ptr(), vs.data_ptr(), P, Hk, ps, d,
                     ps // blocks[2], 0)


def _q8_table(table, torch):
    if not (table.dtype is torch.int32 and table.dim() == 2 and table.is_contiguous()):
        raise ValueError("block_table must be a contiguous int32 tensor [B, max_pages]")
    return table.shape


def _q8_index(t, n, name, torch):
    if not (t.dtype is torch.int32 and t.dim() == 1 and t.shape[0] == n and t.is_contiguous()):
        raise ValueError(f"{name} must be a contiguous int32 tensor of {n} entries")
    return t.data_ptr()


def _q8_rows(t, name, torch):
    """(sequence, head, row) strides of bf16 rows [B, Hk, n, d] or [Hk, total, d]: any with the
    last dimension contiguous and the others multiples of 8 elements."""
    st = t.stride()
    if st[0] % 8 or st[1] % 8 or st[-2] % 8:  # a dimension of one element may have any stride
        st = tuple(s if n > 1 else 0 for s, n in zip(st[:-1], t.shape)) + st[-1:]
    if t.dtype is not torch.bfloat16 or st[-1] != 1 or st[0] % 8 or st[1] % 8 or st[-2] % 8:
        raise ValueError(f"{name} must be bfloat16 with contiguous rows and strides that are "
                         "multiples of 8 elements")
    return (0, st[0], st[1]) if len(st) == 3 else st[:3]


def _q8_stream(stream, torch, *tensors):
    """(handle, context) of a call's stream: new outputs are made in the context, so that they
    belong to that stream (None: it is the current one). Every tensor must be on the current CUDA
    device, the one the kernels are launched on."""
    dev = tensors[0].get_device()
    for t in tensors:
        if t.get_device() != dev or dev < 0:
            raise ValueError("the tensors must be on the current CUDA device")
    if torch.cuda.current_device() != dev:
        raise ValueError("the tensors must be on the current CUDA device")
    now = torch._C._cuda_getCurrentRawStream(dev)
    if stream is None:
        return now, None
    handle = int(getattr(stream, "cuda_stream", stream))
    if handle == now:
        return now, None
    return handle, torch.cuda.stream(stream if isinstance(stream, torch.cuda.Stream)
                                     else torch.cuda.ExternalStream(handle))


def q8_cache_write(k, v, k_cache, v_cache, k_scale, v_scale, block_table, lengths, *,
                   cu_seqlens=None, stream=None) -> None:
    """Quantise new keys and values into an 8-bit paged cache, in place. k, v: bf16
    [B, Hk, n, d], n new rows for each sequence, or with cu_seqlens (int32 [B + 1]) packed
    [Hk, total, d]; any strides with contiguous rows. `lengths` (int32 [B]) counts each sequence's
    keys with the new rows, which become its last positions; block_table is int32 [B, max_pages].
    A page written to must belong to one sequence of the call. See fa_q8_cache_write in
    include/fa_train.h for the rounding and the scales. With `stream`, the inputs have to stay as
    they are until that stream has done the call."""
    import torch

    cache = _q8_cache(k_cache, v_cache, k_scale, v_scale, torch)
    B, per = _q8_table(block_table, torch)
    shape = k.shape
    if v.shape != shape:
        raise ValueError("k and v must have the same shape")
    if cu_seqlens is None:
        if not (len(shape) == 4 and shape[0] == B and shape[1] == cache.n_kv_heads
                and shape[3] == cache.head_dim):
            raise ValueError("k and v must be [B, Hk, n, d]")
        cu, total, n = None, 0, shape[2]
    else:
        if not (len(shape) == 3 and shape[0] == cache.n_kv_heads and shape[2] == cache.head_dim):
            raise ValueError("packed k and v must be [Hk, total, d]")
        cu, total, n = _q8_index(cu_seqlens, B + 1, "cu_seqlens", torch), shape[1], 0
    rows = FaQ8Rows(k.data_ptr(), v.data_ptr(), _q8_rows(k, "k", torch), _q8_rows(v, "v", torch),
                    cu, block_table.data_ptr(), _q8_index(lengths, B, "lengths", torch), B, per,
                    total, n)
    handle, _ = _q8_stream(stream, torch, k, v, k_cache, v_cache, k_scale, v_scale, block_table,
                           lengths, *(() if cu is None else (cu_seqlens,)))
    if total == 0 and n == 0:
        return
    rc = (_lib or load_library()).fa_q8_cache_write(ctypes.byref(cache), ctypes.byref(rows),
                                                    handle)
    if rc:
        raise FaError(rc, "fa_q8_cache_write")


def q8_cache_read(k_cache, v_cache, k_scale, v_scale, block_table, cu_seqlens, total, *, out=None,
                  stream=None):
    """The keys and values of a batch back from an 8-bit paged cache: (k, v), bf16
    [Hk, total, d], packed as varlen_attention_fwd takes them. Sequence b's rows
    cu_seqlens[b] .. cu_seqlens[b + 1] - 1 are its first keys. `out`: a pair of such tensors of
    any strides with contiguous rows that do not lie on one another, such as views of one tensor
    (rows behind cu_seqlens[B] are left as they were). With `stream`, the inputs have to stay as they
    are until that stream has done the call, and new outputs belong to it."""
    import torch

    cache = _q8_cache(k_cache, v_cache, k_scale, v_scale, torch)
    B, per = _q8_table(block_table, torch)
    cu = _q8_index(cu_seqlens, B + 1, "cu_seqlens", torch)
    total = int(total)
    shape = (cache.n_kv_heads, total, cache.head_dim)
    handle, ctx = _q8_stream(stream, torch, k_cache, v_cache, k_scale, v_scale, block_table,
                             cu_seqlens, *(out or ()))
    if out is not None:
        k, v = out
        if not (k.shape == v.shape == shape):
            raise ValueError("out must be two tensors [Hk, total, d]")
        ks, vs = _q8_rows(k, "out[0]", torch), _q8_rows(v, "out[1]", torch)
    else:
        if ctx is None:
            k = torch.empty(shape, dtype=torch.bfloat16, device=k_cache.device)
            v = torch.empty_like(k)
        else:
            with ctx:
                k = torch.empty(shape, dtype=torch.bfloat16, device=k_cache.device)
                v = torch.empty_like(k)
        ks = vs = (0, total * shape[2], shape[2])
    if total == 0:
        return k, v
    rows = FaQ8Rows(k.data_ptr(), v.data_ptr(), ks, vs, cu, block_table.data_ptr(), None, B, per,
                    total, 0)
    rc = (_lib or load_library()).fa_q8_cache_read(ctypes.byref(cache), ctypes.byref(rows), handle)
    if rc:
        raise FaError(rc, "fa_q8_cache_read")
    return k, v


def q8_paged_attention(q, k_cache, v_cache, k_scale, v_scale, block_table, lengths, *, scale,
                       causal=True, stream=None):
    """paged_attention over an 8-bit paged cache: q bf16 [B, H, q_len, d], codes float8_e4m3fn
    [num_pages, Hk, page_size, d] with float32 scales [num_pages, Hk, page_size // scale_block],
    block_table [B, max_pages] and lengths [B] (int32): returns (o, lse). The q_len queries are
    each sequence's last positions (causal: bottom-right per sequence). Scales outside [0, 2^100]
    are reported by fa_device_status. With `stream`, the inputs have to stay as they are until that
    stream has done the call, and the outputs belong to it. For a long prompt against the cache
    (more than about 640 query rows a kv head, 140 at head_dim 256) q8_cache_read and
    varlen_attention_fwd are faster."""
    import torch

    cache = _q8_cache(k_cache, v_cache, k_scale, v_scale, torch)
    shape = q.shape
    if not (q.dtype is torch.bfloat16 and len(shape) == 4 and q.is_contiguous()
            and shape[3] == cache.head_dim):
        raise ValueError("q must be contiguous bfloat16 [B, H, q_len, d]")
    B, H, lq, d = shape
    rows, per = _q8_table(block_table, torch)
    if rows != B:
        raise ValueError("block_table must have a row for each sequence of q")
    lens = _q8_index(lengths, B, "lengths", torch)
    handle, ctx = _q8_stream(stream, torch, q, k_cache, v_cache, k_scale, v_scale, block_table,
                             lengths)
    params = FaPagedParams(B, H, cache.n_kv_heads, lq, d, cache.page_size, per, cache.num_pages,
                           float(scale), 1 if causal else 0, 0, 0)
    if ctx is None:
        o = torch.empty_like(q)
        lse = torch.empty((B, H, lq), dtype=torch.float32, device=q.device)
    else:
        with ctx:
            o = torch.empty_like(q)
            lse = torch.empty((B, H, lq), dtype=torch.float32, device=q.device)
    rc = (_lib or load_library()).fa_q8_paged_attention(
        q.data_ptr(), ctypes.byref(cache), block_table.data_ptr(), lens, o.data_ptr(),
        lse.data_ptr(), ctypes.byref(params), handle)
    if rc:
        raise FaError(rc, "fa_q8_paged_attention")
    return o, lse
