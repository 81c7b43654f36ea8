"""Prompt attention of rows with one token that takes nearly all the weight, of a small value, and many
of weights around 2^-25 whose values are large: together they decide the output.

Tolerance, as in test_gpu_attention_prompt but for the weights: the kernel holds a weight, relative to a
running maximum that is at most the row's, times 2^7 (fp16) before it is rounded to the type, so it is
off by u of itself (u = 2^-11, bf16 2^-8) or, below 2^-21 in fp16, by 2^-32 of the largest:

    |out - ref| <= u |ref| + (1 + u) (u + e) sum_j p_j |v_j| + n 2^-32 max|v|   [fp16; 0 for bf16]

with e < 2 (72 * 24 + 64) 2^-24 for the scores here (sum |q k| / sqrt(D) <= 24, D = 64).  The scores do not
depend on the row, so the reference is a running sum in 64 bits.
"""

from __future__ import annotations

import numpy as np
import pytest
import torch

import w4a16_dequant_gemm_amd as W4

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _needs_gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    W4.lib()


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("n,heads,sink", [(300, 1, 0), (2000, 1, 0), (2000, 1, 700), (16384, 1, 0), (16384, 40, 3)])
def test_many_small_weights(n, heads, sink, dtype):
    D = 64
    g = torch.Generator().manual_seed(n + sink)
    q = torch.zeros((n, heads, D))
    q[..., 0] = 4.0
    k = torch.zeros((n, 1, D))
    k[:, 0, 0] = torch.tensor([0.0, 2.0, -4.0, 4.5, 0.5])[torch.randint(0, 5, (n,), generator=g)]
    k[sink, 0, 0] = 34.5                       # a score of 17.25: the others' weights are 2^-22 .. 2^-28 of its
    v = torch.randn((n, 1, D), generator=g) + 2.0
    v[sink] *= 2.0 ** -12
    q, k, v = (t.to(dtype).cuda() for t in (q, k, v))
    out = W4.attention_prompt(q, k, v, torch.tensor([0, n], dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    w = np.exp(k[:, 0, 0].double().cpu().numpy() * 0.5)[:, None]
    vd = v[:, 0].double().cpu().numpy()
    total = np.cumsum(w, 0)
    ref, mag = np.cumsum(w * vd, 0) / total, np.cumsum(w * np.abs(vd), 0) / total
    u = 2.0 ** -11 if dtype == torch.float16 else 2.0 ** -8
    e = 2 * (72 * 24 + 64) * 2.0 ** -24
    tol = u * np.abs(ref) + (1 + u) * (u + e) * mag
    if dtype == torch.float16:
        tol = tol + n * 2.0 ** -32 * np.abs(vd).max()
    err = np.abs(out.double().cpu().numpy() - ref[:, None])
    assert (err <= tol[:, None]).all(), f"worst {np.max(err / tol[:, None]):.1f} x"
