"""Helpers of the tests of the batched cache operators: caches on the device, the rows they stand
for and attention over them in fp64 (NumPy), and the error bound that the tests hold outputs to.

Bound on an output element.  With u the rounding of the output type (fp16 2^-11, bf16 2^-8):

* a softmax weight times V's scale is rounded once to fp16: relative 2^-11 of it, or, where it is
  below fp16's normal range, an absolute 2^-25 in units in which the largest scale is 2^7, that is
  2^-32 smax per token, times the largest code cmax;
* the weight itself carries the fp32 error of its score, (D + 8) 2^-24 sum_d |q_d k_d| / sqrt(D), and
  32 * 2^-24 of exponential, sums and joining the splits, twice (the row's normalization has the
  error of its weights): e = 2 ((D + 8) max_t sum |q k| / sqrt(D) + 32) 2^-24;
* the output's sum runs in fp32 over products of 16 tokens or more: (n / 16 + 40) 2^-24 sum p |v|;
* the output is rounded once (below fp16's normal range by 2^-25 at most):

    |out - ref| <= u |ref| + (1 + u) (2^-11 + e + (n / 16 + 40) 2^-24) sum p |v| + n 2^-32 smax cmax
                   + 2^-25 [fp16].

An accumulated weight has no 16-bit rounding: |sum - ref| <= e sum_h p + 4 * 2^-24 |ref|.
"""

from __future__ import annotations

import numpy as np
import torch

import w4a16_dequant_gemm_amd as W4

U = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}


def f64(t):
    return t.detach().cpu().double().numpy()


def make_cache(shape, bits, dtype, seed, scale=1.0, outliers=True):
    """A quantized cache of normal rows ``[..., T, D]`` by the library's quantizer."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(shape, generator=g) * scale
    if outliers:
        x = torch.where(torch.rand(shape, generator=g) < 0.02, x * 8.0, x)
    c, s, z = W4.kv_quantize(x.to(dtype).reshape(-1, shape[-2], shape[-1]).cuda(), bits)
    lead = shape[:-1]
    return c.view(*lead, -1), s.view(lead), None if z is None else z.view(lead)


def rows(cache, bits):
    """The values a cache stands for, fp64 ``[..., T, D]``."""
    c, s, z = cache
    if bits == 8:
        return f64(c) * f64(s)[..., None]
    w = c.cpu().numpy().view(np.uint32)
    u = np.stack([(w >> np.uint32(4 * i)) & np.uint32(15) for i in range(8)], -1).reshape(*w.shape[:-1], -1)
    return (u.astype(np.float64) - f64(z)[..., None]) * f64(s)[..., None]


def cmax(cache, bits):
    return 127.0 if bits == 8 else 15.0 + float(cache[2].float().abs().max())


def attend(q, k, v):
    """``(out, weights, sum p |v|, max sum |q k| / sqrt(D))`` of queries ``[R, D]`` over ``k, v [n, D]``."""
    D = q.shape[1]
    if k.shape[0] == 0:
        return np.zeros_like(q), np.zeros((q.shape[0], 0)), np.zeros_like(q), 0.0
    s = q @ k.T / np.sqrt(D)
    p = np.exp(s - s.max(1, keepdims=True))
    p /= p.sum(1, keepdims=True)
    return p @ v, p, p @ np.abs(v), float((np.abs(q) @ np.abs(k).T).max() / np.sqrt(D))


def weight_error(D, qk):
    return 2.0 * ((D + 8) * qk + 32) * 2.0 ** -24


def check_out(got, ref, mag, dtype, e, n, smax, c):
    u = U[dtype]
    tol = u * np.abs(ref) + (1 + u) * (2.0 ** -11 + e + (n / 16 + 40) * 2.0 ** -24) * mag + n * 2.0 ** -32 * smax * c
    if dtype == torch.float16:
        tol = tol + 2.0 ** -25
    assert np.all(np.isfinite(got))
    err = np.abs(got - ref)
    assert (err <= tol).all(), f"{(err > tol).sum()} of {err.size} outside, worst {(err / np.maximum(tol, 1e-300)).max():.2f} x"


def spoil(cache, lengths, bits):
    """NaN scales and zero points and arbitrary codes in the rows behind ``lengths`` (one per
    sequence, or one number for a shared cache)."""
    c, s, z = cache
    for b, n in enumerate(lengths if s.dim() == 3 else [lengths]):
        at = (b,) if s.dim() == 3 else ()
        s[at + (slice(None), slice(n, None))] = float("nan")
        c[at + (slice(None), slice(n, None))] = -128 if bits == 8 else -1
        if z is not None:
            z[at + (slice(None), slice(n, None))] = float("nan")
