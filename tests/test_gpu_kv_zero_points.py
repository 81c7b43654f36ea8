"""KV4 caches whose zero points lie beyond 2048 (rows of nearly equal values far from 0): c - z is rounded to
fp16, so an element of K and V is off by 2^-11 of itself at most.  On top of the bound of kv_util that
is 2^-11 sum p |v| for the values, and 2^-11 sum |q k| / sqrt(D) for a score, twice that for a weight.
"""

from __future__ import annotations

import numpy as np
import pytest
import torch

import w4a16_dequant_gemm_amd as W4
from tests.kv_util import attend, f64, rows, weight_error

pytestmark = pytest.mark.gpu
H = torch.float16


@pytest.fixture(scope="module", autouse=True)
def _needs_gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    W4.lib()


def cache(shape, D, gen, lo, hi):
    codes = torch.randint(-(1 << 31), 1 << 31, (*shape, D // 8), generator=gen).to(torch.int32).cuda()
    z = torch.exp(torch.rand(shape, generator=gen) * np.log(hi / lo)) * lo
    z = torch.where(torch.rand(shape, generator=gen) < 0.5, -z, z).round().half()
    s = ((torch.rand(shape, generator=gen) + 0.5) / z.float().abs()).half()      # elements of 0.5 to 1.5
    return codes, s.cuda(), z.cuda()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("lo,hi", [(1500, 3000), (2049, 60000)])
@pytest.mark.parametrize("B,P,room", [(3, 0, 40), (3, 0, 1100), (6, 1500, 40), (40, 1500, 40)])
def test_large_zero_points(B, P, room, lo, hi, D):
    Hq = 8
    gen = torch.Generator().manual_seed(B + lo)
    q = torch.randn((B, Hq, D), generator=gen).to(H).cuda()
    kp, vp = (cache((1, max(P, 1)), D, gen, lo, hi) for _ in range(2))
    k, v = (cache((B, 1, room), D, gen, lo, hi) for _ in range(2))
    lens = [room - 3 * (b % 10) for b in range(B)]
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    out = W4.kv_attention_decode_shared(q, kp, vp, P, k, v, n, 4)
    if P == 0:
        out2, sums = W4.kv_attention_decode_weights(q, k, v, n, None, 4)
    torch.cuda.synchronize()
    KP, VP, K, V = (rows(c, 4) for c in (kp, vp, k, v))
    for b in range(0, B, max(1, B // 6)):
        kk, vv = np.concatenate([KP[0, :P], K[b, 0, :lens[b]]]), np.concatenate([VP[0, :P], V[b, 0, :lens[b]]])
        ref, p, mag, qk = attend(f64(q)[b], kk, vv)
        e, t = weight_error(D, qk) + 2 * 2.0 ** -11 * qk, P + lens[b]
        tol = 2.0 ** -11 * np.abs(ref) + (1 + 2.0 ** -11) * (2.0 ** -10 + e + (t / 16 + 40) * 2.0 ** -24) * mag
        tol += t * 2.0 ** -32 * max(float(vp[1].max()), float(v[1].max())) * 65504 + 2.0 ** -25
        for o in (out, out2) if P == 0 else (out,):
            assert (np.abs(f64(o)[b] - ref) <= tol).all()
        if P == 0:
            want = p.sum(0)
            assert (np.abs(f64(sums)[b, 0, :lens[b]] - want) <= (e + 2.0 ** -20) * want).all()
