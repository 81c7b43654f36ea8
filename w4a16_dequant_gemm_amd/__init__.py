"""MI355X-native W4A16 weight-only linear layer: Python binding of ``libw4a16.so``.

The binding only marshals arguments: it checks dtypes, shapes and contiguity of torch
tensors, passes raw device pointers and the current HIP stream to the C ABI and turns
negative status codes into :class:`W4A16Error`.  Every step of the computation runs in
the library's HIP kernels; there is no CPU or PyTorch fallback.

``quantize_pack(W, group_size, scheme)`` -> ``(qweight, scales, zeros)``
    group-wise INT4 RTN quantization of an fp32 ``[N, K]`` CUDA tensor.
``linear(X, qweight, scales, zeros, group_size, path=PATH_AUTO)`` -> ``Y``
    ``Y = X . dequant(qweight)^T`` for fp16/bf16 ``X [M, K]``.
``linear_batch([(X, qweight, scales, zeros, group_size), ...])`` -> ``[Y, ...]``
    independent layers in one call; one-row layers share grouped launches.
``gptq_hessian(X, H=None)`` / ``gptq_factor(H, damp)`` / ``gptq_quantize(W, U, group_size, scheme)``
    GPTQ: ``H = 2 X^T X`` (fp64, lower triangle), the upper Cholesky factor ``U`` of the
    damped inverse, and the compensated column-wise quantization in the packed format.
``awq_stats(X)`` / ``awq_search(W, X, xmean, group_size, scheme)`` / ``awq_scale(X, s)``
    AWQ: per-channel activation statistic, grid search over channel scalings, and the
    activation side of the rescaling.
``w8a8_smooth`` / ``w8a8_quantize_weight`` / ``w8a8_quantize_act`` / ``w8a8_linear``
    W8A8 with SmoothQuant on the INT8 matrix cores.
``kv_quantize(x, bits)`` / ``kv_attention_decode(q, cache, T)``
    per-token KV8 / KV4 cache quantization and the decode attention over the quantized cache.
``attention_prompt(q, k, v, cu_seqlens)``
    causal attention over packed prompts, on the 16-bit keys and values before they are cached.
``kv_attention_decode_shared(q, kprefix, vprefix, P, kcache, vcache, lengths)``
    decode attention of a batch whose sequences share a cached prefix, read once for all.
``kv_attention_decode_weights(q, kcache, vcache, lengths, weights)`` / ``kv_evict(kcache, vcache, weights, ...)``
    decode attention that adds up the attention weight of every cached token, and the compaction
    of a cache to the recent and the most attended tokens.
``rope_frequencies(R, base, scaling)`` / ``rope(x, positions, freqs)``
    rotary positions: half or interleaved pairs, part of a head, scaled for long contexts.
``kv_pages(...)`` / ``kv_append_paged(k, v, kpages, vpages, table, lengths, ...)`` / ``kv_read_paged(...)``
    a paged 8-bit cache with one scale a page and head: pools, appending with the keys (and queries)
    rotated on the way, reading tokens back as 16-bit rows.
``kv_attention_paged(q, kpages, vpages, table, lengths, cu_seqlens)``
    causal attention over the pages, of a decode step's tokens or of chunks of prompts.
"""

from __future__ import annotations

import functools
import math
import struct

import torch

from . import _lib as _lib_mod
from ._lib import (ASYM, BF16, F16, KV_E4M3, KV_INT8, KvCache, KvPaged, OK, PATH_AUTO, PATH_GEMV, PATH_NAMES, PATH_PREFILL,
                   PATH_SKINNY, SYM, W4A16Error, check, lib)

__all__ = [
    "ASYM", "SYM", "F16", "BF16", "PATH_AUTO", "PATH_GEMV", "PATH_SKINNY", "PATH_PREFILL",
    "PATH_NAMES", "W4A16Error", "quantize_pack", "linear", "linear_batch", "dequantize", "select_path",
    "w8a16_quantize_pack", "w8a16_linear", "w8a16_select_path", "linear_workspace", "linear_ws",
    "abi_version", "lib", "gptq_hessian", "gptq_factor", "gptq_quantize", "awq_stats",
    "awq_search", "awq_scale", "w8a8_smooth", "w8a8_quantize_weight", "w8a8_quantize_act",
    "w8a8_linear", "kv_quantize", "kv_attention_decode", "attention_prompt",
    "kv_attention_decode_shared", "kv_attention_decode_weights", "kv_evict",
    "rope_frequencies", "rope", "kv_pages", "kv_append_paged", "kv_read_paged", "kv_attention_paged",
    "kv_attention_paged_workspace",
]


_INT8, _INT32, _HALF = torch.int8, torch.int32, torch.float16


def _stream() -> int:
    return torch.cuda.current_stream().cuda_stream


def _call(fn, what: str, device: torch.device, *args) -> None:
    """``fn(*args, stream)`` on ``device``, on the stream current there, whichever device is
    current; raises on a negative status."""
    i = device.index
    stream = torch._C._cuda_getCurrentRawStream(i)      # the handle alone, without a Stream object
    if i == torch._C._cuda_getDevice():
        status = fn(*args, stream)
    else:
        with torch.cuda.device(device):
            status = fn(*args, stream)
    if status != OK:
        raise W4A16Error(status, what)


def _same_device(x: torch.Tensor, name: str, **others) -> None:
    """Every given tensor (None: absent) is a GPU tensor on the device of ``x``."""
    dev = x.get_device()
    for other, t in others.items():
        if t is not None and t.get_device() != dev:
            raise ValueError(f"{other} must be on the device of {name}")


def _need(t: torch.Tensor, name: str, dtype, ndim: int) -> None:
    if isinstance(t, torch.Tensor) and t.dtype is dtype and t.dim() == ndim and t.is_cuda and t.is_contiguous():
        return
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != ndim:
        raise ValueError(f"{name} must be {ndim}-D")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.float16:
        return F16
    if t.dtype == torch.bfloat16:
        return BF16
    raise TypeError(f"activations must be float16 or bfloat16, got {t.dtype}")


def _check_linear(X, qweight, scales, zeros, group_size: int, codes_per_word: int):
    """Argument checks shared by the linear calls: dtypes, 2-D contiguous GPU tensors on the
    device of ``X``, ``qweight [N, K/codes_per_word]``, ``scales`` and ``zeros`` (if given)
    ``[N, K/group_size]``.  Returns ``(M, K, N)``."""
    _need(X, "X", X.dtype, 2)
    _need(qweight, "qweight", torch.int32, 2)
    _need(scales, "scales", torch.float16, 2)
    if zeros is not None:
        _need(zeros, "zeros", torch.float16, 2)
    M, K = X.shape
    N = qweight.shape[0]
    if qweight.shape[1] * codes_per_word != K:
        raise ValueError(f"qweight must be [N, K/{codes_per_word}]")
    if group_size <= 0 or K % group_size or tuple(scales.shape) != (N, K // group_size):
        raise ValueError("scales must be [N, K/group_size]")
    if zeros is not None and zeros.shape != scales.shape:
        raise ValueError("zeros must match scales")
    for t, name in ((qweight, "qweight"), (scales, "scales"), (zeros, "zeros")):
        if t is not None and t.device != X.device:
            raise ValueError(f"{name} must be on the device of X")
    return M, K, N


def _out(out, X, M: int, N: int) -> torch.Tensor:
    """The output tensor: allocated ``[M, N]`` in the dtype of ``X``, or a caller tensor
    checked for dtype, shape, device and contiguity."""
    if out is None:
        return torch.empty((M, N), dtype=X.dtype, device=X.device)
    _need(out, "out", X.dtype, 2)
    if tuple(out.shape) != (M, N):
        raise ValueError("out must be [M, N]")
    if out.device != X.device:
        raise ValueError("out must be on the device of X")
    return out


def abi_version() -> int:
    return lib().w4a16_abi_version()


def select_path(M: int, N: int, K: int, group_size: int, dtype: int = F16) -> int:
    """Kernel path the dispatcher picks (host only); raises on invalid arguments."""
    p = lib().w4a16_select_path(M, N, K, group_size, dtype)
    if p < 0:
        raise W4A16Error(p, "select_path")
    return p


def quantize_pack(W: torch.Tensor, group_size: int = 128, scheme: int = ASYM,
                  write_zeros: bool = True):
    """Quantize fp32 ``W [N, K]`` on the GPU.

    Returns ``(qweight int32 [N, K/8], scales fp16 [N, K/g], zeros fp16 [N, K/g] or None)``.
    ``zeros`` is None only for the symmetric scheme with ``write_zeros=False``.
    """
    _need(W, "W", torch.float32, 2)
    N, K = W.shape
    if K % 8 or group_size <= 0 or K % group_size:
        raise ValueError("K must be a multiple of 8 and of group_size")
    G = K // group_size
    qweight = torch.empty((N, K // 8), dtype=torch.int32, device=W.device)
    scales = torch.empty((N, G), dtype=torch.float16, device=W.device)
    zeros = None
    if scheme == ASYM or write_zeros:
        zeros = torch.empty((N, G), dtype=torch.float16, device=W.device)
    st = lib().w4a16_quantize_pack(W.data_ptr(), N, K, group_size, scheme, qweight.data_ptr(),
                                   scales.data_ptr(), zeros.data_ptr() if zeros is not None else None,
                                   _stream())
    check(st, "w4a16_quantize_pack")
    return qweight, scales, zeros


def linear(X: torch.Tensor, qweight: torch.Tensor, scales: torch.Tensor, zeros, group_size: int,
           path: int = PATH_AUTO, out: torch.Tensor | None = None) -> torch.Tensor:
    """``Y [M, N] = X [M, K] . dequant(qweight)^T`` in the dtype of ``X``."""
    dt = _dtype_code(X)
    M, K, N = _check_linear(X, qweight, scales, zeros, group_size, 8)
    out = _out(out, X, M, N)
    st = lib().w4a16_linear_ex(X.data_ptr(), dt, M, N, K, group_size, qweight.data_ptr(),
                               scales.data_ptr(), zeros.data_ptr() if zeros is not None else None,
                               out.data_ptr(), path, _stream())
    check(st, "w4a16_linear")
    return out


def linear_batch(layers, outs=None) -> list:
    """Several independent layers in one call: ``layers`` is a sequence of
    ``(X, qweight, scales, zeros, group_size)`` with one activation dtype; returns the outputs
    ``Y`` (``outs``, if given, supplies them).  One-row layers share grouped launches."""
    layers = list(layers)
    if not layers:
        raise ValueError("linear_batch needs at least one layer")
    dt = _dtype_code(layers[0][0])
    outs = list(outs) if outs is not None else [None] * len(layers)
    if len(outs) != len(layers):
        raise ValueError("outs must match layers")
    items = (_lib_mod.LinearItem * len(layers))()
    ys = []
    for i, ((X, qweight, scales, zeros, group_size), out) in enumerate(zip(layers, outs)):
        if _dtype_code(X) != dt:
            raise TypeError("all layers of a batch need the same activation dtype")
        M, K, N = _check_linear(X, qweight, scales, zeros, group_size, 8)
        if X.device != layers[0][0].device:
            raise ValueError("all layers of a batch must be on one device")
        y = _out(out, X, M, N)
        items[i] = _lib_mod.LinearItem(X.data_ptr(), M, N, K, group_size, qweight.data_ptr(), scales.data_ptr(),
                                       zeros.data_ptr() if zeros is not None else None, y.data_ptr())
        ys.append(y)
    check(lib().w4a16_linear_batch(items, len(layers), dt, _stream()), "w4a16_linear_batch")
    return ys


def linear_workspace(M: int, N: int, K: int, group_size: int, dtype: int = F16) -> int:
    """Bytes of fp32 workspace :func:`linear_ws` can use (0: it behaves as :func:`linear`)."""
    need = lib().w4a16_linear_workspace(M, N, K, group_size, dtype)
    if need < 0:
        raise W4A16Error(int(need), "w4a16_linear_workspace")
    return int(need)


def linear_ws(X: torch.Tensor, qweight: torch.Tensor, scales: torch.Tensor, zeros, group_size: int,
              work: torch.Tensor | None = None, out: torch.Tensor | None = None) -> torch.Tensor:
    """:func:`linear` with a workspace for the tile-starved prefill shapes (split K, partial
    tiles summed in fixed order).  ``work``: float32 device tensor (allocated here if None)."""
    dt = _dtype_code(X)
    M, K, N = _check_linear(X, qweight, scales, zeros, group_size, 8)
    need = linear_workspace(M, N, K, group_size, dt)
    if work is None and need > 0:
        work = torch.empty((need + 3) // 4, dtype=torch.float32, device=X.device)
    if work is not None:
        _need(work, "work", torch.float32, work.dim())
        if work.device != X.device:
            raise ValueError("work must be on the device of X")
    out = _out(out, X, M, N)
    st = lib().w4a16_linear_ws(X.data_ptr(), dt, M, N, K, group_size, qweight.data_ptr(), scales.data_ptr(),
                               zeros.data_ptr() if zeros is not None else None, out.data_ptr(),
                               work.data_ptr() if work is not None else None,
                               work.numel() * 4 if work is not None else 0, _stream())
    check(st, "w4a16_linear_ws")
    return out


def w8a16_quantize_pack(W: torch.Tensor, group_size: int = 128, scheme: int = ASYM,
                        write_zeros: bool = True):
    """8-bit codes: quantize fp32 ``W [N, K]`` on the GPU.  Returns ``(qweight int32 [N, K/4],
    scales fp16 [N, K/g], zeros fp16 [N, K/g] or None)``; ``zeros`` is None only for the
    symmetric scheme with ``write_zeros=False`` (implicit zero point 128)."""
    _need(W, "W", torch.float32, 2)
    N, K = W.shape
    if K % 4 or group_size <= 0 or K % group_size:
        raise ValueError("K must be a multiple of 4 and of group_size")
    G = K // group_size
    qweight = torch.empty((N, K // 4), dtype=torch.int32, device=W.device)
    scales = torch.empty((N, G), dtype=torch.float16, device=W.device)
    zeros = None
    if scheme == ASYM or write_zeros:
        zeros = torch.empty((N, G), dtype=torch.float16, device=W.device)
    st = lib().w4a16_w8a16_quantize_pack(W.data_ptr(), N, K, group_size, scheme, qweight.data_ptr(),
                                         scales.data_ptr(), zeros.data_ptr() if zeros is not None else None,
                                         _stream())
    check(st, "w4a16_w8a16_quantize_pack")
    return qweight, scales, zeros


def w8a16_select_path(M: int, N: int, K: int, group_size: int, dtype: int = F16) -> int:
    """Kernel the 8-bit dispatcher picks (host only): ``PATH_GEMV`` or ``PATH_PREFILL``."""
    p = lib().w4a16_w8a16_select_path(M, N, K, group_size, dtype)
    if p < 0:
        raise W4A16Error(p, "w8a16_select_path")
    return p


def w8a16_linear(X: torch.Tensor, qweight: torch.Tensor, scales: torch.Tensor, zeros, group_size: int,
                 path: int = PATH_AUTO, out: torch.Tensor | None = None) -> torch.Tensor:
    """``Y [M, N] = X [M, K] . dequant(qweight)^T`` with 8-bit codes ``qweight int32 [N, K/4]``
    (the weight-streaming GEMV for M <= 16, the tiled MFMA GEMM above)."""
    dt = _dtype_code(X)
    M, K, N = _check_linear(X, qweight, scales, zeros, group_size, 4)
    out = _out(out, X, M, N)
    st = lib().w4a16_w8a16_linear_ex(X.data_ptr(), dt, M, N, K, group_size, qweight.data_ptr(),
                                     scales.data_ptr(), zeros.data_ptr() if zeros is not None else None,
                                     out.data_ptr(), path, _stream())
    check(st, "w4a16_w8a16_linear")
    return out


def dequantize(qweight: torch.Tensor, scales: torch.Tensor, zeros, group_size: int) -> torch.Tensor:
    """Exact fp32 ``W_hat [N, K]`` (layout checks and tests)."""
    _need(qweight, "qweight", torch.int32, 2)
    _need(scales, "scales", torch.float16, 2)
    if zeros is not None:
        _need(zeros, "zeros", torch.float16, 2)
    N, KW = qweight.shape
    K = KW * 8
    out = torch.empty((N, K), dtype=torch.float32, device=qweight.device)
    st = lib().w4a16_dequantize(qweight.data_ptr(), scales.data_ptr(),
                                zeros.data_ptr() if zeros is not None else None, N, K, group_size,
                                out.data_ptr(), _stream())
    check(st, "w4a16_dequantize")
    return out


def gptq_hessian(X: torch.Tensor, H: torch.Tensor | None = None) -> torch.Tensor:
    """``H = 2 X^T X`` (``H += 2 X^T X`` when ``H`` is given) for fp16/bf16 calibration
    activations ``X [n, K]``; fp64 ``[K, K]``, lower triangle defined."""
    dt = _dtype_code(X)
    _need(X, "X", X.dtype, 2)
    n, K = X.shape
    acc = H is not None
    if H is None:
        H = torch.empty((K, K), dtype=torch.float64, device=X.device)
    else:
        _need(H, "H", torch.float64, 2)
        if tuple(H.shape) != (K, K):
            raise ValueError("H must be [K, K]")
    check(lib().w4a16_gptq_hessian(X.data_ptr(), dt, n, K, H.data_ptr(), 1 if acc else 0, _stream()),
          "w4a16_gptq_hessian")
    return H


def gptq_factor(H: torch.Tensor, damp: float = 0.01) -> torch.Tensor:
    """Upper ``U`` with ``(H + damp * mean(diag H) I)^-1 = U^T U``; ``H`` is overwritten."""
    _need(H, "H", torch.float64, 2)
    K = H.shape[0]
    if tuple(H.shape) != (K, K):
        raise ValueError("H must be square")
    U = torch.empty_like(H)
    check(lib().w4a16_gptq_factor(H.data_ptr(), K, float(damp), U.data_ptr(), _stream()),
          "w4a16_gptq_factor")
    return U


def gptq_quantize(W: torch.Tensor, U: torch.Tensor, group_size: int = 128, scheme: int = ASYM,
                  work: torch.Tensor | None = None):
    """GPTQ of fp32 ``W [N, K]`` with the factor ``U``; returns ``(qweight, scales, zeros)``
    in the layout of :func:`quantize_pack` (zeros all 8 for the symmetric scheme)."""
    _need(W, "W", torch.float32, 2)
    _need(U, "U", torch.float64, 2)
    N, K = W.shape
    if tuple(U.shape) != (K, K):
        raise ValueError("U must be [K, K]")
    if K % 8 or group_size <= 0 or K % group_size:
        raise ValueError("K must be a multiple of 8 and of group_size")
    need = N * K + 64 * N
    if work is None:
        work = torch.empty(need, dtype=torch.float64, device=W.device)
    elif work.dtype != torch.float64 or work.numel() < need or not work.is_contiguous():
        raise ValueError(f"work must be a contiguous fp64 tensor of >= {need} elements")
    G = K // group_size
    qweight = torch.empty((N, K // 8), dtype=torch.int32, device=W.device)
    scales = torch.empty((N, G), dtype=torch.float16, device=W.device)
    zeros = torch.empty((N, G), dtype=torch.float16, device=W.device)
    check(lib().w4a16_gptq_quantize(W.data_ptr(), N, K, group_size, scheme, U.data_ptr(),
                                    work.data_ptr(), qweight.data_ptr(), scales.data_ptr(),
                                    zeros.data_ptr(), _stream()), "w4a16_gptq_quantize")
    return qweight, scales, zeros


def awq_stats(X: torch.Tensor) -> torch.Tensor:
    """Mean ``|x|`` per input channel of calibration activations ``X [n, K]`` (fp32 ``[K]``)."""
    dt = _dtype_code(X)
    _need(X, "X", X.dtype, 2)
    n, K = X.shape
    out = torch.empty(K, dtype=torch.float32, device=X.device)
    check(lib().w4a16_awq_stats(X.data_ptr(), dt, n, K, out.data_ptr(), _stream()), "w4a16_awq_stats")
    return out


def awq_search(W: torch.Tensor, X: torch.Tensor, xmean: torch.Tensor, group_size: int = 128,
               scheme: int = ASYM):
    """Grid search of the channel scaling; returns ``(qweight, scales, zeros, s, losses,
    best)`` (``s`` fp32 ``[K]``, ``losses`` fp64 ``[9]``, ``best`` int32 ``[1]``, all on the
    GPU)."""
    _need(W, "W", torch.float32, 2)
    dt = _dtype_code(X)
    _need(X, "X", X.dtype, 2)
    _need(xmean, "xmean", torch.float32, 1)
    N, K = W.shape
    n = X.shape[0]
    if X.shape[1] != K or xmean.shape[0] != K:
        raise ValueError("X must be [n, K] and xmean [K]")
    if K % 8 or group_size <= 0 or K % group_size:
        raise ValueError("K must be a multiple of 8 and of group_size")
    L = lib()
    need = L.w4a16_awq_workspace(N, K, n)
    if need < 0:
        raise W4A16Error(int(need), "w4a16_awq_workspace")
    work = torch.empty(need, dtype=torch.float64, device=W.device)
    G = K // group_size
    qweight = torch.empty((N, K // 8), dtype=torch.int32, device=W.device)
    scales = torch.empty((N, G), dtype=torch.float16, device=W.device)
    zeros = torch.empty((N, G), dtype=torch.float16, device=W.device)
    s = torch.empty(K, dtype=torch.float32, device=W.device)
    losses = torch.empty(9, dtype=torch.float64, device=W.device)
    best = torch.empty(1, dtype=torch.int32, device=W.device)
    check(L.w4a16_awq_search(W.data_ptr(), N, K, X.data_ptr(), dt, n, xmean.data_ptr(), group_size,
                             scheme, work.data_ptr(), losses.data_ptr(), best.data_ptr(), s.data_ptr(),
                             qweight.data_ptr(), scales.data_ptr(), zeros.data_ptr(), _stream()),
          "w4a16_awq_search")
    return qweight, scales, zeros, s, losses, best


def awq_scale(X: torch.Tensor, s: torch.Tensor, out: torch.Tensor | None = None) -> torch.Tensor:
    """``X * s`` per input channel, rounded once to the dtype of ``X``."""
    dt = _dtype_code(X)
    _need(X, "X", X.dtype, 2)
    _need(s, "s", torch.float32, 1)
    M, K = X.shape
    if s.shape[0] != K:
        raise ValueError("s must be [K]")
    if out is None:
        out = torch.empty_like(X)
    else:
        _need(out, "out", X.dtype, 2)
    check(lib().w4a16_awq_scale(X.data_ptr(), dt, M, K, s.data_ptr(), out.data_ptr(), _stream()),
          "w4a16_awq_scale")
    return out


def w8a8_smooth(X: torch.Tensor, W: torch.Tensor, alpha_quarters: int = 2) -> torch.Tensor:
    """SmoothQuant factors ``s [K]`` from calibration activations ``X [n, K]`` and ``W [N, K]``."""
    dt = _dtype_code(X)
    _need(X, "X", X.dtype, 2)
    _need(W, "W", torch.float32, 2)
    n, K = X.shape
    N = W.shape[0]
    if W.shape[1] != K:
        raise ValueError("W must be [N, K]")
    s = torch.empty(K, dtype=torch.float32, device=X.device)
    check(lib().w4a16_w8a8_smooth(X.data_ptr(), dt, n, W.data_ptr(), N, K, alpha_quarters, s.data_ptr(),
                                  _stream()), "w4a16_w8a8_smooth")
    return s


def w8a8_quantize_weight(W: torch.Tensor, s: torch.Tensor):
    """``(qweight int8 [N, K], wscale fp32 [N])`` of the smoothed weights ``W * s``."""
    _need(W, "W", torch.float32, 2)
    _need(s, "s", torch.float32, 1)
    N, K = W.shape
    q = torch.empty((N, K), dtype=torch.int8, device=W.device)
    sw = torch.empty(N, dtype=torch.float32, device=W.device)
    check(lib().w4a16_w8a8_quantize_weight(W.data_ptr(), N, K, s.data_ptr(), q.data_ptr(), sw.data_ptr(),
                                           _stream()), "w4a16_w8a8_quantize_weight")
    return q, sw


def w8a8_quantize_act(X: torch.Tensor, s: torch.Tensor):
    """``(qx int8 [M, K], xscale fp32 [M])``: per-token INT8 of ``X / s``."""
    dt = _dtype_code(X)
    _need(X, "X", X.dtype, 2)
    _need(s, "s", torch.float32, 1)
    M, K = X.shape
    q = torch.empty((M, K), dtype=torch.int8, device=X.device)
    sx = torch.empty(M, dtype=torch.float32, device=X.device)
    check(lib().w4a16_w8a8_quantize_act(X.data_ptr(), dt, M, K, s.data_ptr(), q.data_ptr(), sx.data_ptr(),
                                        _stream()), "w4a16_w8a8_quantize_act")
    return q, sx


def w8a8_linear(qx: torch.Tensor, sx: torch.Tensor, qw: torch.Tensor, sw: torch.Tensor,
                dtype=torch.float16, out: torch.Tensor | None = None) -> torch.Tensor:
    """``Y [M, N]`` from INT8 operands and their fp32 scales, on the INT8 matrix cores."""
    _need(qx, "qx", torch.int8, 2)
    _need(qw, "qweight", torch.int8, 2)
    _need(sx, "xscale", torch.float32, 1)
    _need(sw, "wscale", torch.float32, 1)
    M, K = qx.shape
    N = qw.shape[0]
    if qw.shape[1] != K or sx.shape[0] != M or sw.shape[0] != N:
        raise ValueError("shape mismatch")
    if out is None:
        out = torch.empty((M, N), dtype=dtype, device=qx.device)
    dt = _dtype_code(out)
    check(lib().w4a16_w8a8_linear(qx.data_ptr(), sx.data_ptr(), M, N, K, qw.data_ptr(), sw.data_ptr(),
                                  out.data_ptr(), dt, _stream()), "w4a16_w8a8_linear")
    return out


def kv_quantize(x: torch.Tensor, bits: int = 8):
    """Quantize ``x [H, T, D]`` (fp16/bf16) into ``(codes, scales, zeros)``: codes int8
    ``[H, T, D]`` (KV8) or int32 ``[H, T, D/8]`` (KV4), scales / zeros fp16 ``[H, T]`` (zeros
    None for KV8)."""
    dt = _dtype_code(x)
    _need(x, "x", x.dtype, 3)
    H, T, D = x.shape
    if bits == 8:
        codes = torch.empty((H, T, D), dtype=torch.int8, device=x.device)
        zeros = None
    else:
        codes = torch.empty((H, T, D // 8), dtype=torch.int32, device=x.device)
        zeros = torch.empty((H, T), dtype=torch.float16, device=x.device)
    scales = torch.empty((H, T), dtype=torch.float16, device=x.device)
    check(lib().w4a16_kv_quantize(x.data_ptr(), dt, H, T, D, bits, codes.data_ptr(), scales.data_ptr(),
                                  zeros.data_ptr() if zeros is not None else None, _stream()),
          "w4a16_kv_quantize")
    return codes, scales, zeros


def kv_attention_workspace(Hq: int, T: int, D: int) -> int:
    """fp32 elements of the scratch buffer that :func:`kv_attention_decode` needs."""
    need = lib().w4a16_kv_attention_workspace(Hq, T, D)
    if need < 0:
        raise W4A16Error(int(need), "w4a16_kv_attention_workspace")
    return int(need)


def kv_attention_batch_workspace(B: int, Hq: int, Tmax: int, D: int) -> int:
    """fp32 elements of the scratch buffer that :func:`kv_attention_decode_batch` needs."""
    need = lib().w4a16_kv_attention_batch_workspace(B, Hq, Tmax, D)
    if need < 0:
        raise W4A16Error(int(need), "w4a16_kv_attention_batch_workspace")
    return int(need)


def kv_attention_decode_batch(q: torch.Tensor, kcache, vcache, lengths: torch.Tensor, bits: int = 8,
                              out: torch.Tensor | None = None, work: torch.Tensor | None = None) -> torch.Tensor:
    """Decode attention for ``B`` sequences in one call: ``q [B, Hq, D]``, caches
    ``(codes, scales, zeros)`` of shape ``[B, Hkv, Tmax, ...]`` (scales ``[B, Hkv, Tmax]``),
    ``lengths`` int32 ``[B]`` on the device."""
    dt = _dtype_code(q)
    _need(q, "q", q.dtype, 3)
    _need(lengths, "lengths", torch.int32, 1)
    B, Hq, D = q.shape
    kc, ks, kz = kcache
    vc, vs, vz = vcache
    if ks.dim() != 3 or ks.shape[0] != B or lengths.shape[0] != B:
        raise ValueError("caches must be [B, Hkv, Tmax, ...] and lengths [B]")
    _, Hkv, Tmax = ks.shape
    L = lib()
    need = kv_attention_batch_workspace(B, Hq, Tmax, D)
    if work is None:
        work = torch.empty(need, dtype=torch.float32, device=q.device)
    elif work.dtype != torch.float32 or not work.is_cuda or work.numel() < need:
        raise ValueError(f"work must be a float32 device tensor of at least {need} elements")
    if out is None:
        out = torch.empty_like(q)
    ptr = lambda t: t.data_ptr() if t is not None else None
    check(L.w4a16_kv_attention_decode_batch(q.data_ptr(), dt, B, Hq, Hkv, lengths.data_ptr(), Tmax, D, bits,
                                            kc.data_ptr(), ks.data_ptr(), ptr(kz), vc.data_ptr(), vs.data_ptr(),
                                            ptr(vz), work.data_ptr(), out.data_ptr(), _stream()),
          "w4a16_kv_attention_decode_batch")
    return out


def kv_attention_decode(q: torch.Tensor, kcache, vcache, T: int, bits: int = 8,
                        out: torch.Tensor | None = None, work: torch.Tensor | None = None) -> torch.Tensor:
    """``softmax(q K^T / sqrt(D)) V`` over the first ``T`` tokens of quantized caches
    ``(codes, scales, zeros)`` of shape ``[Hkv, Tmax, ...]``; ``q [Hq, D]``.  ``work`` is an
    optional fp32 device buffer of at least :func:`kv_attention_workspace` elements."""
    dt = _dtype_code(q)
    _need(q, "q", q.dtype, 2)
    Hq, D = q.shape
    kc, ks, kz = kcache
    vc, vs, vz = vcache
    Hkv, Tmax = ks.shape
    L = lib()
    need = kv_attention_workspace(Hq, T, D)
    if work is None:
        work = torch.empty(need, dtype=torch.float32, device=q.device)
    elif work.dtype != torch.float32 or not work.is_cuda or work.numel() < need:
        raise ValueError(f"work must be a float32 device tensor of at least {need} elements")
    if out is None:
        out = torch.empty_like(q)
    ptr = lambda t: t.data_ptr() if t is not None else None
    check(L.w4a16_kv_attention_decode(q.data_ptr(), dt, Hq, Hkv, T, Tmax, D, bits, kc.data_ptr(), ks.data_ptr(),
                                      ptr(kz), vc.data_ptr(), vs.data_ptr(), ptr(vz), work.data_ptr(),
                                      out.data_ptr(), _stream()), "w4a16_kv_attention_decode")
    return out


def _need_heads(t: torch.Tensor, name: str, dtype) -> int:
    """``t [T, H, D]``: a GPU tensor of adjacent heads (a row is ``H * D`` consecutive values); rows
    may be further apart, as in a column block of a wider tensor.  Returns the rows' distance."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != 3:
        raise ValueError(f"{name} must be 3-D")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    T, H, D = t.shape
    st, sh, sd = t.stride()
    if (D > 1 and sd != 1) or (H > 1 and sh != D):
        raise ValueError(f"the heads of {name} must be adjacent (strides [*, D, 1])")
    return st if T > 1 else H * D          # (a single row's stride is arbitrary in torch)


def attention_prompt(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cu_seqlens: torch.Tensor,
                     out: torch.Tensor | None = None) -> torch.Tensor:
    """Causal attention over packed prompts: ``out[i, h] = softmax_j(q[i, h] . k[j, h // G] /
    sqrt(D)) . v`` over the tokens ``j <= i`` of the sequence of ``i``, ``G = Hq / Hkv``.

    ``q [T, Hq, D]``, ``k`` and ``v [T, Hkv, D]`` are fp16 or bf16; their heads are adjacent, their
    rows may be strided (column blocks of a fused projection).  Sequence ``b`` is the tokens
    ``cu_seqlens[b] .. cu_seqlens[b + 1] - 1`` (int32 ``[B + 1]`` on the device, not decreasing).
    Rows outside every sequence are neither read nor written: in an ``out`` of the caller's (which
    must not overlap the inputs) they keep what they held, in the returned tensor of a call without
    ``out`` they are undefined.  Scores, softmax statistics and sums are fp32; the softmax weights are
    rounded once to the inputs' type.  A row depends on the tokens up to its own alone, whatever later
    ones hold; an infinity or NaN among the values that it sees makes that element of it one or NaN."""
    dt = _dtype_code(q)
    dtype, dev = q.dtype, q.get_device()
    strides = None
    if (q.dim() == 3 and isinstance(k, torch.Tensor) and isinstance(v, torch.Tensor) and dev >= 0 and k.dtype is dtype
            and v.dtype is dtype and dev == k.get_device() == v.get_device()):
        # the usual case in few steps; anything else is looked at piece by piece below
        T, Hq, D = q.shape
        kshape = k.shape
        if len(kshape) == 3 and T > 1 and D > 1 and kshape[0] == T and kshape[2] == D and v.shape == kshape:
            (sq, hq, dq), (sk, hk, dk), (sv, hv, dv) = q.stride(), k.stride(), v.stride()
            if dq == dk == dv == 1 and hq == hk == hv == D:
                strides, Hkv = (sq, sk, sv), kshape[1]
    if strides is None:
        strides = _need_heads(q, "q", dtype), _need_heads(k, "k", dtype), _need_heads(v, "v", dtype)
        T, Hq, D = q.shape
        Hkv = k.shape[1]
        if k.shape != v.shape or k.shape[0] != T or k.shape[2] != D:
            raise ValueError("k and v must be [T, Hkv, D]")
        _same_device(q, "q", k=k, v=v)
    _need(cu_seqlens, "cu_seqlens", _INT32, 1)
    B = cu_seqlens.shape[0] - 1
    if B < 1:
        raise ValueError("cu_seqlens must be [B + 1] with B >= 1")
    if out is None:
        out = torch.empty((T, Hq, D), dtype=dtype, device=q.device)
    else:
        _need(out, "out", dtype, 3)
        if out.shape != q.shape:
            raise ValueError("out must be [T, Hq, D]")
    if dev != cu_seqlens.get_device() or dev != out.get_device():
        raise ValueError("cu_seqlens and out must be on the device of q")
    _call(lib().w4a16_attention_prompt, "w4a16_attention_prompt", q.device, q.data_ptr(), k.data_ptr(), v.data_ptr(),
          dt, T, B, cu_seqlens.data_ptr(), Hq, Hkv, D, *strides, out.data_ptr())
    return out


def _cache_shape(cache, name: str, bits: int, lead: int, D: int, dev: int):
    """Checks ``(codes, scales, zeros)`` of a quantized cache with ``lead`` leading axes besides the
    tokens', on device ``dev``; returns the shape of its scales."""
    codes, scales, zeros = cache
    _need(codes, f"{name} codes", torch.int8 if bits == 8 else torch.int32, lead + 2)
    _need(scales, f"{name} scales", torch.float16, lead + 1)
    shape = scales.shape
    if codes.shape != (*shape, D if bits == 8 else D // 8):
        raise ValueError(f"{name} codes must be [..., {'D' if bits == 8 else 'D/8'}] over its scales' shape")
    if bits == 4:
        if zeros is None:
            raise ValueError(f"{name} needs zeros for 4-bit codes")
        _need(zeros, f"{name} zeros", torch.float16, lead + 1)
        if zeros.shape != shape:
            raise ValueError(f"{name} zeros must match its scales")
    for t in cache[:2 if bits == 8 else 3]:
        if t.get_device() != dev:
            raise ValueError(f"{name} must be on the device of the other arguments")
    return shape


def _need_caches(k, v, kname: str, vname: str, bits: int, lead: int, D: int, like: torch.Tensor):
    """A K and a V cache of one shape on the device of ``like``; returns the shape of their scales."""
    if bits != 8 and bits != 4:
        raise ValueError("bits must be 8 or 4")
    dev = like.get_device()
    (kc, ks, kz), (vc, vs, vz) = k, v
    if isinstance(kc, torch.Tensor) and isinstance(ks, torch.Tensor) and isinstance(vc, torch.Tensor) and isinstance(
            vs, torch.Tensor):
        # the usual case in one expression; anything else is looked at piece by piece below
        shape = ks.shape
        want = (*shape, D if bits == 8 else D // 8)
        code = _INT8 if bits == 8 else _INT32
        if (len(shape) == lead + 1 and kc.dtype is code and vc.dtype is code and ks.dtype is _HALF and vs.dtype is _HALF
                and vs.shape == shape and kc.shape == want and vc.shape == want
                and dev == kc.get_device() == ks.get_device() == vc.get_device() == vs.get_device()
                and kc.is_contiguous() and ks.is_contiguous() and vc.is_contiguous() and vs.is_contiguous()
                and (bits == 8 or (isinstance(kz, torch.Tensor) and isinstance(vz, torch.Tensor) and kz.dtype is _HALF
                                   and vz.dtype is _HALF and kz.shape == shape and vz.shape == shape
                                   and dev == kz.get_device() == vz.get_device() and kz.is_contiguous()
                                   and vz.is_contiguous()))):
            return shape
    shape = _cache_shape(k, kname, bits, lead, D, dev)
    if _cache_shape(v, vname, bits, lead, D, dev) != shape:
        raise ValueError(f"{kname} and {vname} must have the same shape")
    return shape


def _cache_struct(k, v, bits: int) -> KvCache:
    z = (k[2].data_ptr(), v[2].data_ptr()) if bits == 4 else (None, None)
    return KvCache(k[0].data_ptr(), k[1].data_ptr(), z[0], v[0].data_ptr(), v[1].data_ptr(), z[1])


def _work(work, need: int, what: str, like: torch.Tensor) -> torch.Tensor:
    """The scratch buffer of a call: allocated, or the caller's checked."""
    if need < 0:
        raise W4A16Error(int(need), what)
    if work is None:
        return torch.empty(need, dtype=torch.float32, device=like.device)
    if work.dtype != torch.float32 or work.device != like.device or not work.is_contiguous() or work.numel() < need:
        raise ValueError(f"work must be a contiguous float32 tensor on {like.device} of at least {need} elements")
    return work


def _decode_out(out, q: torch.Tensor) -> torch.Tensor:
    if out is None:
        return torch.empty_like(q)
    _need(out, "out", q.dtype, 3)
    if out.shape != q.shape or out.device != q.device:
        raise ValueError("out must be [B, Hq, D] on the device of q")
    return out


def kv_attention_shared_workspace(B: int, Hq: int, Hkv: int, P: int, Tmax: int, D: int) -> int:
    """fp32 elements of a scratch buffer that holds every :func:`kv_attention_decode_shared` call of these
    heads with at most ``B`` sequences, ``P`` shared and ``Tmax`` own tokens (0: none)."""
    need = lib().w4a16_kv_attention_shared_workspace(B, Hq, Hkv, P, Tmax, D)
    if need < 0:
        raise W4A16Error(int(need), "w4a16_kv_attention_shared_workspace")
    return int(need)


def kv_attention_weights_workspace(B: int, Hq: int, Hkv: int, Tmax: int, D: int) -> int:
    """fp32 elements of a scratch buffer that holds every :func:`kv_attention_decode_weights` call of these
    heads with at most ``B`` sequences and ``Tmax`` tokens (0: none)."""
    need = lib().w4a16_kv_attention_weights_workspace(B, Hq, Hkv, Tmax, D)
    if need < 0:
        raise W4A16Error(int(need), "w4a16_kv_attention_weights_workspace")
    return int(need)


def kv_evict_workspace(B: int, Hkv: int, Tmax: int) -> int:
    """fp32 elements of a scratch buffer that holds every :func:`kv_evict` call of at most ``B`` sequences
    and ``Tmax`` tokens (0: none)."""
    need = lib().w4a16_kv_evict_workspace(B, Hkv, Tmax)
    if need < 0:
        raise W4A16Error(int(need), "w4a16_kv_evict_workspace")
    return int(need)


def kv_attention_decode_shared(q: torch.Tensor, kprefix, vprefix, P: int, kcache, vcache, lengths: torch.Tensor,
                               bits: int = 8, out: torch.Tensor | None = None,
                               work: torch.Tensor | None = None) -> torch.Tensor:
    """Decode attention of ``B`` sequences that begin with the same tokens: ``q [B, Hq, D]`` over the
    first ``P`` tokens of the shared caches ``(codes, scales, zeros)`` of shape ``[Hkv, Pmax, ...]``,
    then the first ``lengths[b]`` (int32, on the device, possibly 0) of the sequence's own
    ``[B, Hkv, Tmax, ...]``.  The prefix is held once for the batch, and a long one read once.  A sequence without any
    token gets zeros.  ``out`` must not overlap the inputs.  ``work`` is an optional fp32 buffer of at least
    :func:`kv_attention_shared_workspace` elements (0 for short sequences); calls that may overlap
    need one each.

    Scores and sums are fp32.  The softmax weights, with V's scales, are rounded once to fp16 (relative
    2^-11), and so is ``c - z`` of 4-bit codes whose zero point is beyond 2048 (rows of nearly equal
    values far from 0); :func:`kv_attention_decode_batch` rounds neither."""
    dt = _dtype_code(q)
    _need(q, "q", q.dtype, 3)
    _need(lengths, "lengths", torch.int32, 1)
    B, Hq, D = q.shape
    Bc, Hkv, Tmax = _need_caches(kcache, vcache, "kcache", "vcache", bits, 2, D, q)
    Hp, Pmax = _need_caches(kprefix, vprefix, "kprefix", "vprefix", bits, 1, D, q)
    if Bc != B or lengths.shape[0] != B or Hp != Hkv:
        raise ValueError("caches must be [B, Hkv, Tmax, ...], prefixes [Hkv, Pmax, ...] and lengths [B]")
    if lengths.get_device() != q.get_device():
        raise ValueError("lengths must be on the device of q")
    if not 0 <= P <= Pmax:
        raise ValueError("P must be in [0, Pmax]")
    L = lib()
    out = _decode_out(out, q)
    need = L.w4a16_kv_attention_shared_call_workspace(B, Hq, Hkv, P, Tmax, D)
    if need or work is not None:
        work = _work(work, need, "w4a16_kv_attention_shared_call_workspace", q)
    _call(L.w4a16_kv_attention_decode_shared, "w4a16_kv_attention_decode_shared", q.device, q.data_ptr(), dt, B, Hq,
          Hkv, D, bits, _cache_struct(kprefix, vprefix, bits), P, Pmax, _cache_struct(kcache, vcache, bits),
          lengths.data_ptr(), Tmax, None if work is None else work.data_ptr(), out.data_ptr())
    return out


def kv_attention_decode_weights(q: torch.Tensor, kcache, vcache, lengths: torch.Tensor, weights: torch.Tensor | None,
                                bits: int = 8, sums: torch.Tensor | None = None, out: torch.Tensor | None = None,
                                work: torch.Tensor | None = None):
    """Decode attention over caches ``[B, Hkv, Tmax, ...]`` that adds up the attention every cached
    token receives; returns ``(out, sums)``.

    ``sums[b, hk, t] = weights[b, hk, t] + sum of the softmax weights of the heads of kv head hk`` for
    ``t < lengths[b]`` (entries behind are not written), fp32 ``[B, Hkv, Tmax]``.  ``sums`` defaults to
    ``weights``, which is then updated in place; ``weights=None`` starts from 0 (``sums`` defaults to
    a zero tensor then).  A sequence of length 0 gets zeros.  ``out`` and ``sums`` must not overlap the
    other inputs or each other.  ``work`` is an optional fp32 buffer of at
    least :func:`kv_attention_weights_workspace` elements (0 for short sequences).  Rounding as in
    :func:`kv_attention_decode_shared`; the weights that are added up are fp32 throughout."""
    dt = _dtype_code(q)
    _need(q, "q", q.dtype, 3)
    _need(lengths, "lengths", torch.int32, 1)
    B, Hq, D = q.shape
    Bc, Hkv, Tmax = shape = _need_caches(kcache, vcache, "kcache", "vcache", bits, 2, D, q)
    if Bc != B or lengths.shape[0] != B:
        raise ValueError("caches must be [B, Hkv, Tmax, ...] and lengths [B]")
    if sums is None:
        sums = torch.zeros(shape, dtype=torch.float32, device=q.device) if weights is None else weights
    for t, name in ((weights, "weights"), (sums, "sums")):
        if t is not None:
            _need(t, name, torch.float32, 3)
            if t.shape != shape:
                raise ValueError(f"{name} must be [B, Hkv, Tmax]")
    _same_device(q, "q", lengths=lengths, weights=weights, sums=sums)
    L = lib()
    out = _decode_out(out, q)
    need = L.w4a16_kv_attention_weights_workspace(B, Hq, Hkv, Tmax, D)
    if need or work is not None:
        work = _work(work, need, "w4a16_kv_attention_weights_workspace", q)
    _call(L.w4a16_kv_attention_decode_weights, "w4a16_kv_attention_decode_weights", q.device, q.data_ptr(), dt, B, Hq,
          Hkv, D, bits, _cache_struct(kcache, vcache, bits), lengths.data_ptr(), Tmax,
          None if weights is None else weights.data_ptr(), sums.data_ptr(),
          None if work is None else work.data_ptr(), out.data_ptr())
    return out, sums


def kv_evict(kcache, vcache, weights: torch.Tensor, lengths: torch.Tensor, budget: int, recent: int, bits: int = 8,
             capacity: int | None = None, out=None, work: torch.Tensor | None = None):
    """Shrink caches ``[B, Hkv, Tmax, ...]`` to at most ``budget`` tokens per sequence: every kv head
    keeps its last ``recent`` tokens and, of the earlier ones, those with the largest ``weights``
    (fp32 ``[B, Hkv, Tmax]``, see :func:`kv_attention_decode_weights`; the earlier token among
    equals), in their order.  A sequence of at most ``budget`` tokens keeps all of them.

    Returns ``(kcache, vcache, weights, lengths, kept)`` in memory of their own, never in place: caches
    and weights with room for ``capacity`` tokens (default ``Tmax``), the weights 0 behind the kept
    tokens, ``lengths = min(lengths, budget)`` and the kept tokens' old indices, int32
    ``[B, Hkv, budget]``, -1 behind them.  ``out`` takes such a tuple to write into (its shapes then
    give the capacity); cache rows behind the kept tokens are not written, in a call without
    ``out`` they are undefined.  ``work`` is an optional fp32 buffer of at least
    :func:`kv_evict_workspace` elements (0 for up to 8192 tokens)."""
    _need(weights, "weights", torch.float32, 3)
    _need(lengths, "lengths", torch.int32, 1)
    if bits != 8 and bits != 4:
        raise ValueError("bits must be 8 or 4")
    if not isinstance(kcache[0], torch.Tensor) or kcache[0].dim() != 4:
        raise ValueError("kcache codes must be 4-D")
    D = kcache[0].shape[3] * (1 if bits == 8 else 8)
    B, Hkv, Tmax = shape = _need_caches(kcache, vcache, "kcache", "vcache", bits, 2, D, weights)
    if weights.shape != shape or lengths.shape[0] != B:
        raise ValueError("weights must be [B, Hkv, Tmax] and lengths [B]")
    if lengths.get_device() != weights.get_device():
        raise ValueError("lengths must be on the device of weights")
    if not 0 <= recent <= budget or budget < 1:
        raise ValueError("0 <= recent <= budget and budget >= 1 must hold")
    if out is None:
        room = (B, Hkv, Tmax if capacity is None else capacity)
        if room[2] < min(budget, Tmax):
            raise ValueError("capacity must be at least min(budget, Tmax)")

        def new(c):
            return tuple(torch.empty(room + tuple(t.shape[3:]), dtype=t.dtype, device=t.device) if t is not None else None
                         for t in (c if bits == 4 else (c[0], c[1], None)))
        out = (new(kcache), new(vcache), torch.empty(room, dtype=torch.float32, device=weights.device),
               torch.empty_like(lengths), torch.empty((B, Hkv, budget), dtype=torch.int32, device=weights.device))
    ko, vo, wo, lo, kept = out
    Bo, Ho, Tout = _need_caches(ko, vo, "out kcache", "out vcache", bits, 2, D, weights)
    _need(wo, "out weights", torch.float32, 3)
    _need(lo, "out lengths", torch.int32, 1)
    _need(kept, "out kept", torch.int32, 3)
    if (Bo, Ho) != (B, Hkv) or wo.shape != (B, Hkv, Tout) or lo.shape[0] != B or kept.shape != (B, Hkv, budget):
        raise ValueError("out must be caches [B, Hkv, capacity, ...], weights [B, Hkv, capacity], lengths [B] and "
                         "kept [B, Hkv, budget]")
    if capacity is not None and Tout != capacity:
        raise ValueError("out and capacity disagree")
    if Tout < min(budget, Tmax):
        raise ValueError("out must have room for min(budget, Tmax) tokens")
    if not weights.get_device() == wo.get_device() == lo.get_device() == kept.get_device():
        raise ValueError("out must be on the device of weights")
    L = lib()
    need = L.w4a16_kv_evict_workspace(B, Hkv, Tmax)
    if need or work is not None:
        work = _work(work, need, "w4a16_kv_evict_workspace", weights)
    _call(L.w4a16_kv_evict, "w4a16_kv_evict", weights.device, _cache_struct(kcache, vcache, bits),
          weights.data_ptr(), lengths.data_ptr(), B, Hkv, Tmax, D, bits, budget, recent, _cache_struct(ko, vo, bits),
          Tout, wo.data_ptr(), lo.data_ptr(), kept.data_ptr(), None if work is None else work.data_ptr())
    return (ko, vo, wo, lo, kept)


# --------------------------------------------------------------------------- rotary positions, paged cache

def rope_frequencies(rotary_dim: int, base: float = 10000.0, scaling: str = "none", factor: float = 1.0,
                     original: int = 0, low: float = 1.0, high: float = 4.0, device="cuda"):
    """The frequencies of rotary positions, ``base ** (-2 i / rotary_dim)`` radians a position for pair
    ``i``, and the factor of the rotated values: ``(freqs, mscale)``, what :func:`rope` takes.

    ``freqs`` is int64 ``[rotary_dim / 2]``: turns per position in units of 2^-64 (as unsigned numbers),
    with which angles stay exact at any position.  ``scaling`` stretches them over longer contexts than
    the ``original`` positions a model was trained on:

    ``"linear"``  every frequency divided by ``factor``;
    ``"base"``    the base raised by ``factor ** (R / (R - 2))``, so that the slowest pair is divided by
                  ``factor`` and the fastest is left alone;
    ``"bands"``   pairs that turn more than ``high`` times in ``original`` positions are left alone, those
                  that turn less than ``low`` times divided by ``factor``, those between blended linearly in
                  their turns;
    ``"ramp"``    the same blended linearly in the pairs' index between the (whole) indices of ``high`` and
                  ``low`` turns (usual: 32 and 1), with ``mscale = 0.1 ln(factor) + 1``.
    """
    R = rotary_dim
    if R < 2 or R % 2:
        raise ValueError("rotary_dim must be even and at least 2")
    if not base > 0 or not factor > 0:
        raise ValueError("base and factor must be positive")
    if scaling not in ("none", "linear", "base", "bands", "ramp"):
        raise ValueError("scaling must be 'none', 'linear', 'base', 'bands' or 'ramp'")
    if scaling in ("bands", "ramp") and (original < 1 or not 0 < low < high):
        raise ValueError(f"scaling '{scaling}' needs original >= 1 and 0 < low < high")
    if scaling == "ramp" and base == 1:
        raise ValueError("scaling 'ramp' needs a base other than 1: the pairs' turns do not differ")
    mscale = 1.0
    if scaling == "base" and R > 2:
        base = base * factor ** (R / (R - 2))
    f = [base ** (-2.0 * i / R) for i in range(R // 2)]
    if scaling == "linear":
        f = [x / factor for x in f]
    elif scaling == "bands":
        for i, x in enumerate(f):
            keep = min(max((original * x / (2 * math.pi) - low) / (high - low), 0.0), 1.0)
            f[i] = x * (keep + (1.0 - keep) / factor)
    elif scaling == "ramp":
        def index(turns):
            return R * math.log(original / (turns * 2 * math.pi)) / (2 * math.log(base))
        first, last = max(math.floor(index(high)), 0), min(math.ceil(index(low)), R - 1)
        for i, x in enumerate(f):
            keep = 1.0 - min(max((i - first) / max(last - first, 1e-3), 0.0), 1.0)
            f[i] = x * (keep + (1.0 - keep) / factor)
        mscale = 0.1 * math.log(factor) + 1.0 if factor > 1.0 else 1.0
    words = [round(x / (2 * math.pi) * 2.0 ** 64) % 2 ** 64 for x in f]
    return torch.tensor([w - 2 ** 64 if w >= 2 ** 63 else w for w in words], dtype=torch.int64, device=device), mscale


_CODES = {torch.float16: F16, torch.bfloat16: BF16}


def _rows16(t, name: str, dtype, dev: int) -> int:
    """``t [T, H, D]`` with adjacent heads on device ``dev``, in the usual case in few steps; returns the rows'
    distance."""
    if isinstance(t, torch.Tensor) and t.dtype is dtype and t.get_device() == dev >= 0:
        st, shape = t.stride(), t.shape
        if len(st) == 3 and st[2] == 1 and st[1] == shape[2] and shape[0] > 1:
            return st[0]
    st = _need_heads(t, name, dtype)
    if t.get_device() != dev:
        raise ValueError(f"{name} must be on the device of the other arguments")
    return st


def _vector(t, name: str, dtype, n: int, dev: int) -> int:
    """``t [n]`` of a type on device ``dev``: its address."""
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.get_device() == dev and t.shape == (n,)
            and t.is_contiguous()):
        _need(t, name, dtype, 1)
        if t.get_device() != dev:
            raise ValueError(f"{name} must be on the device of the other arguments")
        if t.shape[0] != n:
            raise ValueError(f"{name} must have {n} elements")
    return t.data_ptr()


def _dense(t, name: str, dtype, shape, dev: int) -> int:
    """A contiguous ``t`` of a type and shape on device ``dev``: its address."""
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.get_device() == dev
            and t.is_contiguous()):
        _need(t, name, dtype, len(shape))
        if t.get_device() != dev:
            raise ValueError(f"{name} must be on the device of the other arguments")
        raise ValueError(f"{name} must be {list(shape)}")
    return t.data_ptr()


def rope(x: torch.Tensor, positions: torch.Tensor, freqs: torch.Tensor, interleaved: bool = False, mscale: float = 1.0,
         out: torch.Tensor | None = None) -> torch.Tensor:
    """Rotates the heads of ``x [T, H, D]`` (fp16 / bf16, adjacent heads, rows possibly strided) by their tokens'
    positions (int32 ``[T]``): the first ``R = 2 * len(freqs)`` values of a head in pairs ``(i, i + R / 2)``, or
    ``(2 i, 2 i + 1)`` if ``interleaved``, by the angle position times frequency, times ``mscale``; the rest
    passes through.  ``freqs`` and ``mscale``: :func:`rope_frequencies`.  ``out`` may be ``x`` (in place), else
    it must not overlap the inputs.  The gradient of ``x`` is ``rope(grad, -positions, ...)``."""
    dt = _dtype_code(x)
    dtype, dev = x.dtype, x.get_device()
    xs = _rows16(x, "x", dtype, dev)
    shape = T, H, D = x.shape
    at = _vector(positions, "positions", _INT32, T, dev)
    pairs = freqs.numel() if isinstance(freqs, torch.Tensor) else 0
    f = _vector(freqs, "freqs", torch.int64, pairs, dev)
    if out is None:
        out = torch.empty(shape, dtype=dtype, device=x.device)
        os = H * D
    else:
        os = _rows16(out, "out", dtype, dev)
        if out.shape != shape:
            raise ValueError("out must be [T, H, D]")
    _call(lib().w4a16_rope, "w4a16_rope", x.device, x.data_ptr(), dt, T, H, D, xs, at, f, 2 * pairs,
          1 if interleaved else 0, mscale, out.data_ptr(), os)
    return out


_E4M3 = torch.float8_e4m3fn


def kv_pages(pages: int, Hkv: int, page: int, D: int, codes=torch.int8, device="cuda"):
    """An empty pool of a paged cache, ``(kpages, vpages)``, each ``(codes, scales)``: codes int8 or
    float8_e4m3fn, K ``[pages, Hkv, page, D]`` and V ``[pages, Hkv, D, page]``, scales fp32 ``[pages, Hkv]``."""
    if codes not in (_INT8, _E4M3):
        raise TypeError("codes must be torch.int8 or torch.float8_e4m3fn")
    if page not in (16, 32, 64, 128) or D not in (64, 128):
        raise ValueError("page must be 16, 32, 64 or 128 and D 64 or 128")

    def pool(shape):
        return (torch.zeros(shape, dtype=torch.uint8, device=device).view(codes),
                torch.zeros((pages, Hkv), dtype=torch.float32, device=device))
    return pool((pages, Hkv, page, D)), pool((pages, Hkv, D, page))


def _paged_odd(kpages, vpages, table, lengths, cu, T, dev: int) -> None:
    """Says what is wrong with the description of a paged cache."""
    (kc, ks), (vc, vs) = kpages, vpages
    for t, name, nd in ((kc, "kpages codes", 4), (vc, "vpages codes", 4), (ks, "kpages scales", 2),
                        (vs, "vpages scales", 2)):
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")
        if t.dim() != nd or not t.is_contiguous():
            raise ValueError(f"{name} must be {nd}-D and contiguous")
        if not t.is_cuda or t.get_device() != dev:
            raise ValueError(f"{name} must be on the GPU of the other arguments")
    if kc.dtype not in (_INT8, _E4M3) or vc.dtype != kc.dtype:
        raise TypeError("codes must be torch.int8 or torch.float8_e4m3fn, alike in kpages and vpages")
    if ks.dtype != torch.float32 or vs.dtype != torch.float32:
        raise TypeError("scales must be float32")
    N, Hkv, page, D = kc.shape
    if vc.shape != (N, Hkv, D, page) or ks.shape != (N, Hkv) or vs.shape != (N, Hkv):
        raise ValueError("kpages must be [pages, Hkv, page, D], vpages [pages, Hkv, D, page] and scales [pages, Hkv]")
    _need(table, "table", _INT32, 2)
    _need(lengths, "lengths", _INT32, 1)
    B = table.shape[0]
    if lengths.shape[0] != B:
        raise ValueError("table must be [B, table_pages] and lengths [B]")
    if table.get_device() != dev or lengths.get_device() != dev:
        raise ValueError("table and lengths must be on the device of the other arguments")
    if cu is None:
        raise ValueError("without cu_seqlens every sequence has one token: T must be B")
    if T is None:
        raise ValueError("T is needed where cu_seqlens is given")
    if not isinstance(T, int):
        raise TypeError("T must be an int")
    _vector(cu, "cu_seqlens", _INT32, B + 1, dev)
    raise ValueError("the description of the paged cache is wrong")


_F32 = torch.float32


def _paged(kpages, vpages, table, lengths, cu, T: int | None, dev: int):
    """The checked description of a paged cache and a call's sequences (``T`` None: the number of sequences), as
    bytes, its ``T``, ``Hkv`` and ``D`` and the tokens that a row of the table has room for."""
    (kc, ks), (vc, vs) = kpages, vpages
    try:
        code = kc.dtype
        N, Hkv, page, D = kc.shape
        B, P = table.shape
        per_head = (N, Hkv)
        if cu is None:
            at = 0
            if T is None:
                T = B
            fine = T == B
        else:
            fine = T is not None
            at = _vector(cu, "cu_seqlens", _INT32, B + 1, dev)
        # (what is no tensor fails one of the comparisons with a tensor's type, device or layout)
        if (fine and (code is _INT8 or code is _E4M3) and vc.dtype is code and ks.dtype is _F32 and vs.dtype is _F32
                and vc.shape == (N, Hkv, D, page) and ks.shape == per_head and vs.shape == per_head
                and table.dtype is _INT32 and lengths.dtype is _INT32 and lengths.shape == (B,)
                and 0 <= dev == kc.get_device() == ks.get_device() == vc.get_device() == vs.get_device()
                == table.get_device() == lengths.get_device()
                and kc.is_contiguous() and ks.is_contiguous() and vc.is_contiguous() and vs.is_contiguous()
                and table.is_contiguous() and lengths.is_contiguous()):
            return KvPaged.pack(kc.data_ptr(), ks.data_ptr(), vc.data_ptr(), vs.data_ptr(), table.data_ptr(),
                                lengths.data_ptr(), at, N, page, P, B, T, Hkv, D,
                                KV_INT8 if code is _INT8 else KV_E4M3), T, Hkv, D, P * page
    except (AttributeError, TypeError, ValueError, struct.error):
        pass
    _paged_odd(kpages, vpages, table, lengths, cu, T, dev)


def kv_append_paged(k: torch.Tensor, v: torch.Tensor, kpages, vpages, table: torch.Tensor, lengths: torch.Tensor,
                    cu_seqlens: torch.Tensor | None = None, freqs: torch.Tensor | None = None,
                    positions: torch.Tensor | None = None, interleaved: bool = False, mscale: float = 1.0,
                    q: torch.Tensor | None = None, q_out: torch.Tensor | None = None) -> torch.Tensor | None:
    """Writes the last tokens of every sequence into the pages of :func:`kv_pages`, keys rotated on the way.

    ``k`` and ``v [T, Hkv, D]`` (fp16 / bf16, adjacent heads, rows possibly strided) are the sequences' new
    tokens: one each, or ``cu_seqlens[b + 1] - cu_seqlens[b]`` of sequence ``b`` from row ``cu_seqlens[b]`` on
    (int32 ``[B + 1]``).  ``lengths`` (int32 ``[B]``) counts a sequence's tokens with the new ones, ``table``
    (int32 ``[B, table_pages]``) names the pages of its tokens in turn; an entry that is no page of the pool takes
    none.  A page that is written to must belong to one sequence.

    A page's scale grows with the tokens written to it since its first slot was, earlier codes being rounded again; infinities
    take the largest code, NaN 0.  ``freqs`` (:func:`rope_frequencies`; None: no rotation), ``interleaved`` and
    ``mscale`` as in :func:`rope`, by ``positions`` (int32 ``[T]``) or the tokens' places in their sequences.
    ``q [T, Hq, D]`` is rotated likewise into ``q_out`` (dense, apart from the inputs), which is returned."""
    dt = _dtype_code(k)
    dtype, dev = k.dtype, k.get_device()
    ks, vs = _rows16(k, "k", dtype, dev), _rows16(v, "v", dtype, dev)
    shape = T, H, D = k.shape
    c, _, Hkv, Dc, _ = _paged(kpages, vpages, table, lengths, cu_seqlens, T, dev)
    if v.shape != shape or H != Hkv or D != Dc:
        raise ValueError("k and v must be [T, Hkv, D]")
    R = f = 0
    if freqs is not None:
        R = freqs.numel() if isinstance(freqs, torch.Tensor) else 0
        f = _vector(freqs, "freqs", torch.int64, R, dev)
        R *= 2
    Hq = qs = 0
    qp = qo = None
    if q is not None:
        qs = _rows16(q, "q", dtype, dev)
        _, Hq, _ = qshape = q.shape
        if qshape[0] != T or qshape[2] != D:
            raise ValueError("q must be [T, Hq, D]")
        if q_out is None:
            q_out = torch.empty(qshape, dtype=dtype, device=k.device)
        qp, qo = q.data_ptr(), _dense(q_out, "q_out", dtype, qshape, dev)
    elif q_out is not None:
        raise ValueError("q_out needs q")
    _call(lib().w4a16_kv_append_paged, "w4a16_kv_append_paged", k.device, c, k.data_ptr(), v.data_ptr(), dt, ks, vs,
          None if positions is None else _vector(positions, "positions", _INT32, T, dev), f or None, R,
          1 if interleaved else 0, mscale, qp, Hq, qs, qo)
    return q_out


def kv_read_paged(kpages, vpages, table: torch.Tensor, lengths: torch.Tensor, cu_seqlens: torch.Tensor | None = None,
                  T: int | None = None, dtype=torch.float16, out=None):
    """The last tokens of every sequence as 16-bit rows ``(k, v)``, ``[T, Hkv, D]`` each: the tokens that
    :func:`kv_append_paged` with the same arguments writes.  ``T`` is the number of packed rows where
    ``cu_seqlens`` is given; ``out`` takes ``(k, v)`` to write into (their shape and type then count).  Tokens
    without a page are zeros; rows of no sequence are not written."""
    pool = kpages[0]
    if not isinstance(pool, torch.Tensor):
        raise TypeError("kpages codes must be a torch.Tensor")
    if out is not None:
        ko, vo = out
        if not isinstance(ko, torch.Tensor) or ko.dim() != 3:
            raise ValueError("out must be two tensors [T, Hkv, D]")
        if T is not None and T != ko.shape[0]:
            raise ValueError("out and T disagree")
        T, dtype = ko.size(0), ko.dtype
    dev = pool.get_device()
    c, T, Hkv, D, _ = _paged(kpages, vpages, table, lengths, cu_seqlens, T, dev)
    shape = (T, Hkv, D)
    if out is None:
        ko, vo = (torch.empty(shape, dtype=dtype, device=pool.device) for _ in range(2))
    code = _CODES.get(dtype)
    if code is None:
        raise TypeError(f"rows are float16 or bfloat16, got {dtype}")
    _call(lib().w4a16_kv_read_paged, "w4a16_kv_read_paged", pool.device, c, code, _dense(ko, "out k", dtype, shape, dev),
          _dense(vo, "out v", dtype, shape, dev))
    return ko, vo


@functools.lru_cache(maxsize=256)
def kv_attention_paged_workspace(Hq: int, Hkv: int, D: int, tokens: int, chunks: bool = True) -> int:
    """fp32 elements of a scratch buffer that holds every :func:`kv_attention_paged` call of these heads whose
    table has room for at most ``tokens`` tokens (0: none); without ``chunks``, of those without ``cu_seqlens``."""
    need = lib().w4a16_kv_attention_paged_workspace(Hq, Hkv, D, tokens, 1 if chunks else 0)
    if need < 0:
        raise W4A16Error(int(need), "w4a16_kv_attention_paged_workspace")
    return int(need)


def kv_attention_paged(q: torch.Tensor, kpages, vpages, table: torch.Tensor, lengths: torch.Tensor,
                       cu_seqlens: torch.Tensor | None = None, out: torch.Tensor | None = None,
                       work: torch.Tensor | None = None) -> torch.Tensor:
    """Causal attention of every sequence's last tokens over its pages, which hold their keys and values already
    (:func:`kv_append_paged` with the same arguments): a decode step, or chunks of prompts where
    ``cu_seqlens`` is given.

    ``q [T, Hq, D]`` (fp16 / bf16, adjacent heads, rows possibly strided); a row sees the tokens up to its own,
    heads ``h`` of q those of kv head ``h // (Hq / Hkv)``; tokens without a page (an entry that is none, or behind the
    table) are not attended to.  Rows that see nothing are zeros, rows of no sequence are not written.  ``out`` must
    not overlap the inputs.  ``work`` is an optional fp32 buffer of at least :func:`kv_attention_paged_workspace`
    elements (0 for short tables); calls that may overlap need one each.

    Codes enter the products exactly; the softmax weights, with V's scales, are rounded once to fp16 (relative
    2^-11, down to 2^-23 of the row's largest weight times the largest scale of V that the row sees; in steps and chunks of
    few rows 2^-22); scores, statistics and sums are fp32."""
    dt = _dtype_code(q)
    dtype, dev = q.dtype, q.get_device()
    qs = _rows16(q, "q", dtype, dev)
    shape = T, Hq, D = q.shape
    c, _, Hkv, Dc, tokens = _paged(kpages, vpages, table, lengths, cu_seqlens, T, dev)
    if D != Dc:
        raise ValueError("q must be [T, Hq, D]")
    if out is None:
        out = torch.empty(shape, dtype=dtype, device=q.device)
    o = _dense(out, "out", dtype, shape, dev)
    need = kv_attention_paged_workspace(Hq, Hkv, D, tokens, cu_seqlens is not None)
    if need or work is not None:
        work = _work(work, need, "w4a16_kv_attention_paged_workspace", q)
    _call(lib().w4a16_kv_attention_paged, "w4a16_kv_attention_paged", q.device, c, q.data_ptr(), dt, Hq, qs,
          None if work is None else work.data_ptr(), o)
    return out
