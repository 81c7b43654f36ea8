"""Helpers of the tests of the paged 8-bit cache: pools of random codes with anything behind the sequences, the
rows they stand for and attention over them in fp64 (NumPy), rotations in fp64, and the error bounds.

Rotation of a pair in fp32: cos and sin are off by 4 * 2^-24 (the angle's last bits, the series, the factor),
the two products and their sum by 2 * 2^-24 of |x0| + |x1| more; u is the rounding of the output:

    |y - ref| <= u |ref| + (1 + u) 8 * 2^-24 m (|x0| + |x1|) + 2^-25 [fp16].

Attention: as for the contiguous caches (a weight has the fp32 error e of its score and the exponential and
is rounded once to fp16 with V's scale, relative 2^-11; the sum of n / 16 products of 16 tokens runs in fp32), but
weights times scales are held times 2^11 (2^15 where there are few rows) over the power of two above the largest
scale, so that roundings below fp16's normal range cost 2^-25 2^-11 2 smax = 2^-35 smax per token, times the largest code:

    |out - ref| <= u |ref| + (1 + u) (2^-11 + e + (n / 16 + 40) 2^-24) sum p |v| + n 2^-35 smax cmax + 2^-25 [fp16].

(Where the sum is of the rounded weights, sum_i p_i d_i (v_i - out), |d_i| <= 2^-11, may reach 2^-11 (sum p |v| + |out|);
the bound stays the one of roundings that do not all have one sign.)
"""

from __future__ import annotations

import numpy as np
import torch

from tests.kv_util import U, weight_error

TOP = {torch.int8: 127.0, torch.float8_e4m3fn: 448.0}
CODES = [torch.int8, torch.float8_e4m3fn]


def f64(t):
    return t.detach().float().cpu().double().numpy()


def rotate(x, positions, words, R, interleaved, m=1.0):
    """Rotation of ``x [T, H, D]`` (fp64) by 64-bit turn fractions, angles by whole-number arithmetic."""
    # (half a turn to either side: small angles of both signs keep their bits)
    turns = [[((int(p) * int(w) + 2 ** 63) % 2 ** 64 - 2 ** 63) / 2.0 ** 64 for w in words] for p in positions]
    a = 2 * np.pi * np.array(turns).reshape(len(positions), 1, R // 2)
    c, s = m * np.cos(a), m * np.sin(a)
    i0, i1 = (np.arange(0, R, 2), np.arange(1, R, 2)) if interleaved else (np.arange(R // 2), np.arange(R // 2, R))
    y = x.copy()
    y[..., i0] = x[..., i0] * c - x[..., i1] * s
    y[..., i1] = x[..., i1] * c + x[..., i0] * s
    size = np.zeros_like(x)
    size[..., i0] = size[..., i1] = abs(m) * (np.abs(x[..., i0]) + np.abs(x[..., i1]))
    return y, size


def check_rotated(got, ref, size, dtype):
    u = U[dtype]
    tol = u * np.abs(ref) + (1 + u) * 8 * 2.0 ** -24 * size + (2.0 ** -25 if dtype == torch.float16 else 0)
    err = np.abs(got - ref)
    assert (err <= tol).all(), f"{(err > tol).sum()} of {err.size} outside, worst {(err / np.maximum(tol, 1e-300)).max():.2f} x"


class Pool:
    """Pages of random codes and scales; sequences of the given lengths lie in pages of random order, and
    what belongs to no token holds NaN (scales, 8-bit floats) or -128."""

    def __init__(self, lengths, Hkv, D, page, codes, seed, scale=1.0, room=0, outliers=True):
        g = torch.Generator().manual_seed(seed)
        self.lengths, self.Hkv, self.D, self.page, self.codes = list(lengths), Hkv, D, page, codes
        counts = [-(-n // page) for n in lengths]
        N = sum(counts) + 3
        order = torch.randperm(N, generator=g).tolist()
        self.P = max(max(counts), 1) + room
        self.table = torch.full((len(lengths), self.P), -1, dtype=torch.int32)
        at = 0
        for b, c in enumerate(counts):
            self.table[b, :c] = torch.tensor(order[at:at + c], dtype=torch.int32)
            at += c
        top = TOP[codes]

        def pool(shape):
            x = torch.randn(shape, generator=g)
            if outliers:
                x = torch.where(torch.rand(shape, generator=g) < 0.02, x * 8.0, x)
            s = x.abs().amax((2, 3)) / top
            c = (x / s[..., None, None]).clamp(-top, top)
            s = s * torch.exp(torch.randn(s.shape, generator=g) * 0.5) * scale
            return (c.round() if codes == torch.int8 else c).to(codes), s
        self.kc, self.ks = pool((N, Hkv, page, D))
        self.vc, self.vs = pool((N, Hkv, D, page))
        # what no token owns
        owner = torch.zeros((N, page), dtype=torch.bool)
        for b, n in enumerate(lengths):
            for i in range(n):
                owner[self.table[b, i // page], i % page] = True
        bad = 0x7F if codes != torch.int8 else 0x80
        self.kc.view(torch.uint8).masked_fill_(~owner[:, None, :, None], bad)
        self.vc.view(torch.uint8).masked_fill_(~owner[:, None, None, :], bad)
        for s in (self.ks, self.vs):
            s[~owner.any(1)] = float("nan")

    def cuda(self):
        """``(kpages, vpages, table, lengths)`` on the GPU."""
        return ((self.kc.cuda(), self.ks.cuda()), (self.vc.cuda(), self.vs.cuda()), self.table.cuda(),
                torch.tensor(self.lengths, dtype=torch.int32).cuda())

    def rows(self, b):
        """K and V of sequence ``b``, fp64 ``[n, Hkv, D]``, and which of its tokens have a page."""
        n, N = self.lengths[b], self.kc.shape[0]
        k, v = np.zeros((n, self.Hkv, self.D)), np.zeros((n, self.Hkv, self.D))
        live = np.zeros(n, bool)
        for i in range(n):
            p, j = int(self.table[b, i // self.page]), i % self.page
            if 0 <= p < N:
                live[i] = True
                k[i] = f64(self.kc[p, :, j]) * f64(self.ks[p])[:, None]
                v[i] = f64(self.vc[p, :, :, j]) * f64(self.vs[p])[:, None]
        return k, v, live


def check_attention(got, q, pool, b, n, Hq, dtype):
    """Holds rows ``got [n, Hq, D]`` of sequence b's last n tokens to the bound."""
    k, v, live = pool.rows(b)
    D, G, L = pool.D, Hq // pool.Hkv, pool.lengths[b]
    smax = float(np.nanmax(f64(pool.vs)))
    cmax = TOP[pool.codes]
    u = U[dtype]
    for h in range(Hq):
        for i in range(n):
            see = live[:max(L - n + i + 1, 0)]
            kk, vv = k[:len(see), h // G][see], v[:len(see), h // G][see]
            if len(kk) == 0:
                assert (got[i, h] == 0).all()
                continue
            s = kk @ q[i, h] / np.sqrt(D)
            p = np.exp(s - s.max())
            p /= p.sum()
            ref, mag = p @ vv, p @ np.abs(vv)
            e = weight_error(D, float((np.abs(kk) @ np.abs(q[i, h])).max() / np.sqrt(D)))
            m = len(kk)
            tol = u * np.abs(ref) + (1 + u) * (2.0 ** -11 + e + (m / 16 + 40) * 2.0 ** -24) * mag + m * 2.0 ** -35 * smax * cmax
            if dtype == torch.float16:
                tol = tol + 2.0 ** -25
            err = np.abs(got[i, h] - ref)
            assert (err <= tol).all(), f"b {b} row {i} head {h}: worst {(err / tol).max():.2f} x"


def e4m3_round(x):
    """The 8-bit floats (4 exponent, 3 mantissa bits) nearest to fp32 values, ties to even, as values."""
    x = np.asarray(x, np.float64)
    step = np.exp2(np.floor(np.log2(np.maximum(np.abs(x), 2.0 ** -6))) - 3)
    return np.clip(np.rint(x / step) * step, -448.0, 448.0)


def to_codes(quotients, codes):
    """Codes' values of fp32 quotients."""
    q = np.where(np.isnan(quotients), 0.0, np.clip(quotients, -TOP[codes], TOP[codes]))
    return np.rint(q) if codes == torch.int8 else e4m3_round(q)


class HostCache:
    """One (sequence, head) of K or V of a paged cache on the host, in the fp32 steps that appending is made of."""

    def __init__(self, page, codes):
        self.page, self.codes, self.pages = page, codes, []       # pages: [values of codes [n, D], scale]

    def write(self, rows, first):
        """Rows ``[n, D]`` (fp32) from place ``first`` on."""
        at = 0
        while at < len(rows):
            place = first + at
            index, off = divmod(place, self.page)
            x = rows[at:at + self.page - off].astype(np.float32)
            while len(self.pages) <= index:
                self.pages.append([np.zeros((0, rows.shape[1])), np.float32(0)])
            c, s = self.pages[index]
            c, s = (c[:off], s) if off else (c[:0], np.float32(0))
            size = np.abs(x)
            top = np.float32(np.where(np.isfinite(size), size, 0).max()) / np.float32(TOP[self.codes])
            if top > s:
                with np.errstate(invalid="ignore"):
                    ratio = s / top
                c = to_codes((c.astype(np.float32) * ratio), self.codes)
                s = top
            with np.errstate(invalid="ignore", divide="ignore"):
                u = x / s if s > 0 else np.zeros_like(x)
            self.pages[index] = [np.concatenate([c, to_codes(u, self.codes)]), s]
            at += len(x)
