"""Parallax attention on B200 (sm_100a): Python binding of the C ABI in include/parallax.h.

Parallax keeps exact softmax attention and subtracts the softmax-weighted
key/value covariance projected by a learned probe rho_i = W_R x_i (zubnet.ai
news item on Parallax, paragraph 2):  y_i = o_i - (m_i - o_i abar_i).

This module only marshals torch tensors to the shared library
``libparallax.so`` (built by ``softmax_learned_covariance_b200.build``); every
step of the computation runs in its CUDA kernels.  There is no fallback: if the
library is missing or a call fails, a ``ParallaxError`` is raised.

Functions keep the C names:
    parallax_fwd(q, k, v, rho=None, causal=True, out_dtype=torch.float32) -> (y, lse)
    parallax_fwd_fused(q, k, v, x, W_R, causal=True) -> (y, lse)     probe rho = x W_R in the kernel
    parallax_fwd_train(q, k, v, rho, causal=True) -> (y, lse, o, abar)  the forward kept for the backward
    parallax_bwd(q, k, v, rho, y, o, abar, lse, dy, causal=True) -> (dq, dk, dv, drho)
    parallax_decode(q, rho, kcache, vcache, seqlens, out_dtype=torch.float32) -> (y, lse)
    parallax_softmax_decode(q, kcache, vcache, seqlens) -> (y, lse)   reference: softmax attention, d 64/128/256
    parallax_decode_ex(..., workspace) -> (y, lse)          caller-owned split scratch
    parallax_decode_paged(q, rho, kpages, vpages, block_table, seqlens) -> (y, lse)
                                                            paged cache, grouped query heads
    parallax_kv_append(k, v, kpages, vpages, block_table, seqlens, kexp=, vexp=, ...) -> new_seqlens
                                                            new tokens into a paged cache (e4m3 or bf16)
    parallax_decode_paged_q8(q, rho, kpages, vpages, kexp, vexp, block_table, seqlens, wacc=None) -> (y, lse)
                                                            decode over an e4m3 cache; adds attention weights to wacc
    parallax_decode_paged_acc(q, rho, kpages, vpages, block_table, seqlens, wacc) -> (y, lse)
                                                            the same over a bf16 cache
    parallax_kv_evict(kpages, vpages, block_table, seqlens, wacc, new_table, budget, recent)
        -> (new_seqlens, kept, new_wacc)                    keep the newest and most attended tokens
    parallax_rho_proj(x, W_R, H, d) -> rho
"""
from __future__ import annotations

import contextlib
import ctypes
import os
import threading

__all__ = [
    "ParallaxError", "lib", "parallax_fwd", "parallax_fwd_fused", "parallax_fwd_train", "parallax_bwd",
    "parallax_decode", "parallax_softmax_decode", "parallax_decode_ex", "parallax_decode_paged",
    "parallax_kv_append", "parallax_decode_paged_q8", "parallax_decode_paged_acc", "parallax_kv_evict",
    "parallax_rho_proj", "parallax_decode_workspace_bytes", "parallax_last_device_error",
    "parallax_strerror", "parallax_device_sm_count", "LIB_PATH", "F32", "BF16", "E4M3",
]

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libparallax.so")
F32, BF16, E4M3 = 0, 1, 2
_lock = threading.Lock()
_lib = None


class ParallaxError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {parallax_strerror(status)} (status {status})")


def lib() -> ctypes.CDLL:
    """The loaded C library (raises if it has not been built)."""
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise ParallaxError(-1, f"{LIB_PATH} is missing; build it with "
                                        "`python -m softmax_learned_covariance_b200.build`")
            L = ctypes.CDLL(LIB_PATH)
            P, I, S = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
            L.parallax_fwd.argtypes = [P, P, P, P, P, P, I, I, I, I, I, I, I, P]
            L.parallax_fwd_fused.argtypes = [P, P, P, P, P, P, P, I, I, I, I, I, I, I, I, P]
            L.parallax_fwd_train.argtypes = [P, P, P, P, P, P, P, P, I, I, I, I, I, I, P]
            L.parallax_bwd.argtypes = [P, P, P, P, P, P, P, P, P, P, P, P, P, I, I, I, I, I, I, P]
            L.parallax_decode.argtypes = [P, P, P, P, P, P, P, I, I, I, I, I, I, P]
            L.parallax_softmax_decode.argtypes = [P, P, P, P, P, P, I, I, I, I, I, I, P]
            L.parallax_decode_ex.argtypes = [P, P, P, P, P, P, P, I, I, I, I, I, I, P, S, P]
            L.parallax_decode_paged.argtypes = [P, P, P, P, P, P, P, P, I, I, I, I, I, I, I, I, I, P]
            L.parallax_decode_paged_q8.argtypes = [P] * 11 + [I] * 9 + [P]
            L.parallax_decode_paged_acc.argtypes = [P] * 9 + [I] * 9 + [P]
            L.parallax_kv_append.argtypes = [P] * 13 + [I] * 9 + [P]
            L.parallax_kv_evict.argtypes = [P] * 11 + [I] * 10 + [P]
            L.parallax_decode_workspace_bytes.argtypes = [I, I, I, I]
            L.parallax_decode_workspace_bytes.restype = S
            L.parallax_rho_proj.argtypes = [P, P, P, I, I, I, I, I, I, P]
            L.parallax_strerror.argtypes = [I]
            L.parallax_strerror.restype = ctypes.c_char_p
            L.parallax_last_device_error.argtypes = [P]
            L.parallax_device_sm_count.argtypes = []
            for f in (L.parallax_fwd, L.parallax_fwd_fused, L.parallax_fwd_train, L.parallax_bwd, L.parallax_decode,
                      L.parallax_softmax_decode, L.parallax_decode_ex, L.parallax_decode_paged,
                      L.parallax_decode_paged_q8, L.parallax_decode_paged_acc, L.parallax_kv_append,
                      L.parallax_kv_evict, L.parallax_rho_proj,
                      L.parallax_last_device_error, L.parallax_device_sm_count):
                f.restype = I
            _lib = L
    return _lib


def parallax_strerror(status: int) -> str:
    if status == -1:
        return "library not built"
    return lib().parallax_strerror(int(status)).decode()


def _torch():
    import torch

    return torch


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    torch = _torch()
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _dtype_code(dt):
    torch = _torch()
    if dt == torch.float32:
        return F32
    if dt == torch.bfloat16:
        return BF16
    raise TypeError(f"unsupported dtype {dt}")


def _check(status, what):
    if status != 0:
        raise ParallaxError(status, what)


def _need(t, name):
    if not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous CUDA tensor")


def parallax_fwd(q, k, v, rho=None, causal: bool = True, out_dtype=None, y=None, lse=None,
                 stream=None, want_lse: bool = True):
    """Prefill/forward.  q,k,v,rho: [B,H,T,d]; returns (y [B,H,T,d], lse [B,H,T] fp32 or None).

    rho=None runs the softmax-only instantiation.  bf16 inputs run on the tensor
    cores (d = 128); fp32 inputs run the fp32 CUDA-core kernel.
    """
    torch = _torch()
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _need(t, n)
    if rho is not None:
        _need(rho, "rho")
    B, H, T, d = q.shape
    out_dtype = out_dtype or torch.float32
    if y is None:
        y = torch.empty((B, H, T, d), dtype=out_dtype, device=q.device)
    if lse is None and want_lse:
        lse = torch.empty((B, H, T), dtype=torch.float32, device=q.device)
    st = lib().parallax_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(rho), _ptr(y), _ptr(lse), B, H, T, d,
                            int(bool(causal)), _dtype_code(q.dtype), _dtype_code(y.dtype), _stream(stream))
    _check(st, "parallax_fwd")
    return y, lse


def parallax_fwd_fused(q, k, v, x, W_R, causal: bool = True, out_dtype=None, y=None, lse=None, stream=None,
                       want_lse: bool = True):
    """Prefill with the probe rho = x W_R computed in the kernel.

    q, k, v: [B, H, T, d] bf16 (d = 128); x: [B, T, d_model] bf16; W_R: [d_model, H*d] bf16.
    """
    torch = _torch()
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (x, "x"), (W_R, "W_R")):
        _need(t, n)
    B, H, T, d = q.shape
    d_model = x.shape[-1]
    out_dtype = out_dtype or torch.float32
    if y is None:
        y = torch.empty((B, H, T, d), dtype=out_dtype, device=q.device)
    if lse is None and want_lse:
        lse = torch.empty((B, H, T), dtype=torch.float32, device=q.device)
    st = lib().parallax_fwd_fused(_ptr(q), _ptr(k), _ptr(v), _ptr(x), _ptr(W_R), _ptr(y), _ptr(lse), B, H, T, d,
                                  d_model, int(bool(causal)), _dtype_code(q.dtype), _dtype_code(y.dtype),
                                  _stream(stream))
    _check(st, "parallax_fwd_fused")
    return y, lse


def parallax_fwd_train(q, k, v, rho, causal: bool = True, stream=None):
    """Training forward: (y, lse, o, abar), fp32; o and abar are what parallax_bwd needs."""
    torch = _torch()
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (rho, "rho")):
        _need(t, n)
    B, H, T, d = q.shape
    f32 = dict(dtype=torch.float32, device=q.device)
    y, o = torch.empty((B, H, T, d), **f32), torch.empty((B, H, T, d), **f32)
    lse, abar = torch.empty((B, H, T), **f32), torch.empty((B, H, T), **f32)
    st = lib().parallax_fwd_train(_ptr(q), _ptr(k), _ptr(v), _ptr(rho), _ptr(y), _ptr(lse), _ptr(o), _ptr(abar),
                                  B, H, T, d, int(bool(causal)), _dtype_code(q.dtype), _stream(stream))
    _check(st, "parallax_fwd_train")
    return y, lse, o, abar


def parallax_bwd(q, k, v, rho, y, o, abar, lse, dy, causal: bool = True, stream=None, out=None):
    """Gradients (dq, dk, dv, drho), fp32, for an upstream dy (bf16, [B, H, T, d]).

    ``out``: optional (dq, dk, dv, drho) fp32 [B, H, T, d] tensors to write into."""
    torch = _torch()
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (rho, "rho"), (y, "y"), (o, "o"), (abar, "abar"), (lse, "lse"),
                 (dy, "dy")):
        _need(t, n)
    B, H, T, d = q.shape
    if out is None:
        outs = [torch.empty((B, H, T, d), dtype=torch.float32, device=q.device) for _ in range(4)]
    else:
        outs = list(out)
        for t, n in zip(outs, ("dq", "dk", "dv", "drho")):
            _need(t, n)
            if t.dtype != torch.float32 or tuple(t.shape) != (B, H, T, d):
                raise ValueError(f"{n} must be float32 of shape {(B, H, T, d)}")
    st = lib().parallax_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(rho), _ptr(y), _ptr(o), _ptr(abar), _ptr(lse), _ptr(dy),
                            *(_ptr(t) for t in outs), B, H, T, d, int(bool(causal)), _dtype_code(q.dtype),
                            _stream(stream))
    _check(st, "parallax_bwd")
    return tuple(outs)


def parallax_decode(q, rho, kcache, vcache, seqlens, out_dtype=None, y=None, lse=None, stream=None,
                    want_lse: bool = True):
    """Decode one token per sequence.  q,rho: [B,H,d]; caches [B,H,Tcap,d]; seqlens int32 [B] on device."""
    torch = _torch()
    for t, n in ((q, "q"), (rho, "rho"), (kcache, "kcache"), (vcache, "vcache"), (seqlens, "seqlens")):
        _need(t, n)
    if seqlens.dtype != torch.int32:
        raise TypeError("seqlens must be int32")
    B, H, Tcap, d = kcache.shape
    out_dtype = out_dtype or torch.float32
    if y is None:
        y = torch.empty((B, H, d), dtype=out_dtype, device=q.device)
    if lse is None and want_lse:
        lse = torch.empty((B, H), dtype=torch.float32, device=q.device)
    st = lib().parallax_decode(_ptr(q), _ptr(rho), _ptr(kcache), _ptr(vcache), _ptr(seqlens), _ptr(y),
                               _ptr(lse), B, H, Tcap, d, _dtype_code(q.dtype), _dtype_code(y.dtype),
                               _stream(stream))
    _check(st, "parallax_decode")
    return y, lse


def parallax_softmax_decode(q, kcache, vcache, seqlens, out_dtype=None, y=None, lse=None, stream=None,
                            want_lse: bool = True):
    """Plain softmax attention decode (no probe), head dims 64, 128, 256: the pages' reference point."""
    torch = _torch()
    for t, n in ((q, "q"), (kcache, "kcache"), (vcache, "vcache"), (seqlens, "seqlens")):
        _need(t, n)
    B, H, Tcap, d = kcache.shape
    out_dtype = out_dtype or torch.float32
    if y is None:
        y = torch.empty((B, H, d), dtype=out_dtype, device=q.device)
    if lse is None and want_lse:
        lse = torch.empty((B, H), dtype=torch.float32, device=q.device)
    st = lib().parallax_softmax_decode(_ptr(q), _ptr(kcache), _ptr(vcache), _ptr(seqlens), _ptr(y), _ptr(lse), B, H,
                                       Tcap, d, _dtype_code(q.dtype), _dtype_code(y.dtype), _stream(stream))
    _check(st, "parallax_softmax_decode")
    return y, lse


def parallax_decode_workspace_bytes(B: int, H: int, Tcap: int, d: int) -> int:
    return int(lib().parallax_decode_workspace_bytes(B, H, Tcap, d))


def parallax_decode_ex(q, rho, kcache, vcache, seqlens, workspace, out_dtype=None, y=None, lse=None,
                       stream=None, want_lse: bool = True):
    """parallax_decode with a caller-owned workspace tensor (any dtype, >= the required bytes)."""
    torch = _torch()
    B, H, Tcap, d = kcache.shape
    out_dtype = out_dtype or torch.float32
    if y is None:
        y = torch.empty((B, H, d), dtype=out_dtype, device=q.device)
    if lse is None and want_lse:
        lse = torch.empty((B, H), dtype=torch.float32, device=q.device)
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    st = lib().parallax_decode_ex(_ptr(q), _ptr(rho), _ptr(kcache), _ptr(vcache), _ptr(seqlens), _ptr(y),
                                  _ptr(lse), B, H, Tcap, d, _dtype_code(q.dtype), _dtype_code(y.dtype),
                                  _ptr(workspace), nbytes, _stream(stream))
    _check(st, "parallax_decode_ex")
    return y, lse


def parallax_decode_paged(q, rho, kpages, vpages, block_table, seqlens, out_dtype=None, y=None, lse=None,
                          stream=None, want_lse: bool = True):
    """Decode over a paged cache with grouped query heads.

    q, rho: [B, Hq, d]; kpages, vpages: [num_pages, Hkv, page_size, d];
    block_table: int32 [B, max_pages] and seqlens: int32 [B], both on the device.
    """
    torch = _torch()
    for t, n in ((q, "q"), (rho, "rho"), (kpages, "kpages"), (vpages, "vpages"), (block_table, "block_table"),
                 (seqlens, "seqlens")):
        _need(t, n)
    if seqlens.dtype != torch.int32 or block_table.dtype != torch.int32:
        raise TypeError("seqlens and block_table must be int32")
    B, Hq, d = q.shape
    num_pages, Hkv, page_size, _ = kpages.shape
    max_pages = block_table.shape[1]
    out_dtype = out_dtype or torch.float32
    if y is None:
        y = torch.empty((B, Hq, d), dtype=out_dtype, device=q.device)
    if lse is None and want_lse:
        lse = torch.empty((B, Hq), dtype=torch.float32, device=q.device)
    st = lib().parallax_decode_paged(_ptr(q), _ptr(rho), _ptr(kpages), _ptr(vpages), _ptr(block_table),
                                     _ptr(seqlens), _ptr(y), _ptr(lse), B, Hq, Hkv, page_size, max_pages,
                                     num_pages, d, _dtype_code(q.dtype), _dtype_code(y.dtype), _stream(stream))
    _check(st, "parallax_decode_paged")
    return y, lse


def _is(t, name, dtype, shape, device):
    """A tensor a kernel reads or writes whole: contiguous, on `device`, of this dtype and shape."""
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}")
    if t.shape != shape or t.device != device or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous tensor of shape {tuple(shape)} on {device}")


def _check_cache(torch, kpages, vpages, kexp, vexp, block_table, seqlens):
    """Shapes of a paged cache; returns (device, B, Hkv, page_size, max_pages, num_pages, d, dtype code)."""
    _need(kpages, "kpages")
    if kpages.dim() != 4 or block_table.dim() != 2 or kpages.shape[2] < 16:
        raise ValueError("kpages must be [num_pages, Hkv, page_size >= 16, d] and block_table [B, max_pages]")
    dev, dtype = kpages.device, kpages.dtype
    num_pages, Hkv, page_size, d = kpages.shape
    B, max_pages = block_table.shape
    _is(vpages, "vpages", dtype, kpages.shape, dev)
    if dtype == torch.float8_e4m3fn:
        if kexp is None or vexp is None:
            raise ValueError("an e4m3 cache needs kexp and vexp")
        _is(kexp, "kexp", torch.int8, (num_pages, Hkv, page_size // 16), dev)
        _is(vexp, "vexp", torch.int8, (num_pages, Hkv, page_size // 16), dev)
        code = E4M3
    elif dtype == torch.bfloat16:
        if kexp is not None or vexp is not None:
            raise ValueError("a bf16 cache has no exponents")
        code = BF16
    else:
        raise TypeError(f"unsupported cache dtype {dtype}")
    _is(block_table, "block_table", torch.int32, (B, max_pages), dev)
    _is(seqlens, "seqlens", torch.int32, (B,), dev)
    return dev, B, Hkv, page_size, max_pages, num_pages, d, code


def _elsewhere(torch, device, stream):
    """Whether a call has to change the current device or stream first (see _on)."""
    return stream is not None or device.index != torch.cuda.current_device()


@contextlib.contextmanager
def _on(torch, device, stream):
    """The tensors' device as the current one and `stream` (default: its current one) as its current
    stream, so that outputs allocated inside belong to the stream that writes them."""
    if stream is not None and stream.device != device:
        raise ValueError(f"the stream must be one of {device}")
    with torch.cuda.device(device), torch.cuda.stream(stream):
        yield


def _raw_stream(torch, device):
    # the handle of torch.cuda.current_stream(device) without building a Stream (0.1 against 2.2 us a call)
    return torch._C._cuda_getCurrentRawStream(device.index)


def _at(t):
    return None if t is None else t.data_ptr()


def parallax_kv_append(k, v, kpages, vpages, block_table, seqlens, kexp=None, vexp=None, counts=None,
                       new_seqlens=None, wacc=None, stream=None):
    """New tokens k, v [B, Hkv, T, d] bf16 behind each sequence's last; returns new_seqlens (int32 [B]).

    k and v may be strided views with a dense last dimension (for instance a [B, T, Hkv, d]
    projection transposed).  kpages, vpages: [num_pages, Hkv, page_size, d] bf16, or e4m3 with kexp,
    vexp int8 [num_pages, Hkv, page_size / 16].  counts: int32 [B], tokens of each sequence (default
    T).  wacc: the weight accumulator, whose entries of the new tokens become 0.
    """
    torch = _torch()
    dev, B, Hkv, ps, mp, npg, d, code = _check_cache(torch, kpages, vpages, kexp, vexp, block_table, seqlens)
    T = k.shape[2] if k.dim() == 4 else 0
    strides = []
    for t, n in ((k, "k"), (v, "v")):
        if t.dtype != torch.bfloat16:
            raise TypeError(f"{n} must be bfloat16")
        if t.shape != (B, Hkv, T, d) or t.device != dev:
            raise ValueError(f"{n} must be [B, Hkv, T, d] = [{B}, {Hkv}, T, {d}] on {dev}")
        if t.is_contiguous():
            strides.append(None)
            continue
        sb, sh, st, si = t.stride()
        if si != 1:
            raise ValueError(f"{n} must have a dense last dimension")
        # the stride of a dimension of size 1 means nothing
        strides.append((ctypes.c_longlong * 3)(sb if B > 1 else 0, sh if Hkv > 1 else 0, st if T > 1 else 0))
    if counts is not None:
        _is(counts, "counts", torch.int32, (B,), dev)
    if wacc is not None:
        _is(wacc, "wacc", torch.float32, (B, Hkv, mp * ps), dev)
    if _elsewhere(torch, dev, stream):
        with _on(torch, dev, stream):
            return parallax_kv_append(k, v, kpages, vpages, block_table, seqlens, kexp, vexp, counts, new_seqlens, wacc)
    if new_seqlens is None:
        new_seqlens = torch.empty_like(seqlens)
    else:
        _is(new_seqlens, "new_seqlens", torch.int32, (B,), dev)
    st = lib().parallax_kv_append(_at(k), _at(v), strides[0], strides[1], _at(kpages), _at(vpages), _at(kexp),
                                  _at(vexp), _at(block_table), _at(seqlens), _at(counts), _at(new_seqlens), _at(wacc),
                                  B, Hkv, T, ps, mp, npg, d, BF16, code, _raw_stream(torch, dev))
    _check(st, "parallax_kv_append")
    return new_seqlens


def _decode_cache(name, q, rho, kpages, vpages, kexp, vexp, block_table, seqlens, wacc, out_dtype, y, lse, stream,
                  want_lse):
    torch = _torch()
    dev, B, Hkv, ps, mp, npg, d, code = _check_cache(torch, kpages, vpages, kexp, vexp, block_table, seqlens)
    if q.dim() != 3:
        raise ValueError(f"q must be [B, Hq, d] = [{B}, Hq, {d}]")
    Hq = q.shape[1]
    _is(q, "q", torch.bfloat16, (B, Hq, d), dev)
    if rho is not None:
        _is(rho, "rho", torch.bfloat16, (B, Hq, d), dev)
    if wacc is not None:
        _is(wacc, "wacc", torch.float32, (B, Hkv, mp * ps), dev)
    if _elsewhere(torch, dev, stream):
        with _on(torch, dev, stream):
            return _decode_cache(name, q, rho, kpages, vpages, kexp, vexp, block_table, seqlens, wacc, out_dtype, y,
                                 lse, None, want_lse)
    if y is None:
        y = torch.empty_like(q, dtype=out_dtype or torch.float32)
    else:
        _is(y, "y", y.dtype, (B, Hq, d), dev)
    if lse is not None:
        _is(lse, "lse", torch.float32, (B, Hq), dev)
    elif want_lse:
        lse = q.new_empty((B, Hq), dtype=torch.float32)
    if code == E4M3:
        st = lib().parallax_decode_paged_q8(_at(q), _at(rho), _at(kpages), _at(vpages), _at(kexp), _at(vexp),
                                            _at(block_table), _at(seqlens), _at(y), _at(lse), _at(wacc), B, Hq, Hkv,
                                            ps, mp, npg, d, BF16, _dtype_code(y.dtype), _raw_stream(torch, dev))
    else:
        st = lib().parallax_decode_paged_acc(_at(q), _at(rho), _at(kpages), _at(vpages), _at(block_table),
                                             _at(seqlens), _at(y), _at(lse), _at(wacc), B, Hq, Hkv, ps, mp, npg, d,
                                             BF16, _dtype_code(y.dtype), _raw_stream(torch, dev))
    _check(st, name)
    return y, lse


def parallax_decode_paged_q8(q, rho, kpages, vpages, kexp, vexp, block_table, seqlens, wacc=None, out_dtype=None,
                             y=None, lse=None, stream=None, want_lse: bool = True):
    """Decode over an e4m3 paged cache (value = code * 2^exp per block of 16 tokens and KV head).

    q: [B, Hq, d] bf16; rho: the same, or None for softmax attention; kpages, vpages: [num_pages, Hkv,
    page_size, d] float8_e4m3fn; kexp, vexp: int8 [num_pages, Hkv, page_size / 16]; wacc: None, or fp32
    [B, Hkv, max_pages * page_size], to which the attention weight of each cached token, summed over
    the query heads of its KV head, is added.
    """
    if kpages.dtype != _torch().float8_e4m3fn:
        raise TypeError("kpages must be float8_e4m3fn")
    return _decode_cache("parallax_decode_paged_q8", q, rho, kpages, vpages, kexp, vexp, block_table, seqlens, wacc,
                         out_dtype, y, lse, stream, want_lse)


def parallax_decode_paged_acc(q, rho, kpages, vpages, block_table, seqlens, wacc, out_dtype=None, y=None, lse=None,
                              stream=None, want_lse: bool = True):
    """parallax_decode_paged_q8 over a bf16 paged cache; wacc is required."""
    if kpages.dtype != _torch().bfloat16:
        raise TypeError("kpages must be bfloat16")
    if wacc is None:
        raise ValueError("wacc is required; without it use parallax_decode_paged")
    return _decode_cache("parallax_decode_paged_acc", q, rho, kpages, vpages, None, None, block_table, seqlens, wacc,
                         out_dtype, y, lse, stream, want_lse)


def parallax_kv_evict(kpages, vpages, block_table, seqlens, wacc, new_table, budget: int, recent: int, kexp=None,
                      vexp=None, new_seqlens=None, kept=None, new_wacc=None, stream=None):
    """Keep min(L, budget) tokens per sequence and KV head: the newest `recent` and the heaviest others.

    They move, in order, to the pages of new_table (int32 [B, new_max_pages], pages no entry of
    block_table reaches).  Returns (new_seqlens int32 [B], kept int32 [B, Hkv, budget]: old positions,
    new_wacc fp32 [B, Hkv, new_max_pages * page_size]); kept and new_wacc are written up to each
    sequence's new length, and start as zero when they are allocated here.
    """
    torch = _torch()
    dev, B, Hkv, ps, mp, npg, d, code = _check_cache(torch, kpages, vpages, kexp, vexp, block_table, seqlens)
    _is(wacc, "wacc", torch.float32, (B, Hkv, mp * ps), dev)
    if new_table.dim() != 2:
        raise ValueError("new_table must be [B, new_max_pages]")
    nmp = new_table.shape[1]
    _is(new_table, "new_table", torch.int32, (B, nmp), dev)
    budget, recent = int(budget), int(recent)
    if not 1 <= budget <= nmp * ps or not 0 <= recent <= budget:
        raise ValueError("1 <= budget <= new_max_pages * page_size and 0 <= recent <= budget are wanted")
    if _elsewhere(torch, dev, stream):
        with _on(torch, dev, stream):
            return parallax_kv_evict(kpages, vpages, block_table, seqlens, wacc, new_table, budget, recent, kexp, vexp,
                                     new_seqlens, kept, new_wacc)
    if new_seqlens is None:
        new_seqlens = torch.empty_like(seqlens)
    else:
        _is(new_seqlens, "new_seqlens", torch.int32, (B,), dev)
    if kept is None:
        kept = torch.zeros((B, Hkv, budget), dtype=torch.int32, device=dev)
    else:
        _is(kept, "kept", torch.int32, (B, Hkv, budget), dev)
    if new_wacc is None:
        new_wacc = torch.zeros((B, Hkv, nmp * ps), dtype=torch.float32, device=dev)
    else:
        _is(new_wacc, "new_wacc", torch.float32, (B, Hkv, nmp * ps), dev)
    st = lib().parallax_kv_evict(_at(kpages), _at(vpages), _at(kexp), _at(vexp), _at(block_table), _at(seqlens),
                                 _at(wacc), _at(new_table), _at(new_seqlens), _at(kept), _at(new_wacc), B, Hkv, ps, mp,
                                 nmp, npg, d, budget, recent, code, _raw_stream(torch, dev))
    _check(st, "parallax_kv_evict")
    return new_seqlens, kept, new_wacc


def parallax_rho_proj(x, W_R, H: int, d: int, rho=None, stream=None):
    """rho [B,H,T,d] bf16 = per-head slices of x [B,T,d_model] @ W_R [d_model, H*d]."""
    torch = _torch()
    _need(x, "x")
    _need(W_R, "W_R")
    B, T, dm = x.shape
    if rho is None:
        rho = torch.empty((B, H, T, d), dtype=torch.bfloat16, device=x.device)
    st = lib().parallax_rho_proj(_ptr(x), _ptr(W_R), _ptr(rho), B, T, dm, H, d, _dtype_code(x.dtype),
                                 _stream(stream))
    _check(st, "parallax_rho_proj")
    return rho


def parallax_last_device_error(stream=None) -> int:
    """Sync the stream; return and clear the device error word (0 or a status code)."""
    return int(lib().parallax_last_device_error(_stream(stream)))


def parallax_device_sm_count() -> int:
    return int(lib().parallax_device_sm_count())
