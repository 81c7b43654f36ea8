"""Prompt attention over keys and values that are not all numbers: what a row sees decides it, what lies
behind it does not, and neither makes the call much slower.

Expected of an element, by the formula with every visible weight above 0: NaN if the row sees a NaN in that
column of the values, or infinities of both signs; that infinity if it sees one; otherwise the number that
the finite values give, within the bound derived in test_gpu_attention_prompt.
"""

from __future__ import annotations

import numpy as np
import pytest
import torch

import w4a16_dequant_gemm_amd as W4
from tests.test_gpu_attention_prompt import E, U, f64, packed, reference

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _needs_gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    W4.lib()


def check(got, q, k, v, lens):
    vd = f64(v)
    fin = np.where(np.isfinite(vd), vd, 0.0)
    ref, mag = reference(f64(q), f64(k), fin, lens)
    u = U[q.dtype]
    tol = u * np.abs(ref) + (1 + u) * (u + E) * mag + max(lens) * 2.0 ** -25 * np.abs(fin).max()
    g, G = f64(got), q.shape[1] // k.shape[1]
    at = 0
    for n in lens:
        seen = [np.logical_or.accumulate(c(vd[at:at + n]), axis=0).repeat(G, axis=1)
                for c in (np.isnan, np.isposinf, np.isneginf)]
        a = g[at:at + n]
        nan = seen[0] | (seen[1] & seen[2])
        assert np.isnan(a[nan]).all()
        assert np.isposinf(a[seen[1] & ~nan]).all() and np.isneginf(a[seen[2] & ~nan]).all()
        num = ~(nan | seen[1] | seen[2])
        assert np.isfinite(a[num]).all(), f"{(~np.isfinite(a[num])).sum()} of {num.sum()} are no numbers"
        err = np.abs(a - ref[at:at + n])[num]
        assert (err <= tol[at:at + n][num]).all(), f"worst {np.max(err / tol[at:at + n][num]):.2f} x"
        at += n


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("lens,Hq,Hkv,D", [([300, 5, 97], 2, 1, 64), ([700], 4, 2, 128), ([1300], 2, 2, 64),
                                           ([1, 1500], 3, 1, 128), ([33, 64, 65, 31], 2, 1, 128)])
def test_scattered_values_without_numbers(lens, Hq, Hkv, D, dtype):
    q, k, v, cu = packed(lens, Hq, Hkv, D, dtype, seed=sum(lens), pad=2)
    g = torch.Generator().manual_seed(7)
    T = sum(lens)
    for x in (float("nan"), float("inf"), -float("inf")):
        for t in torch.randint(0, T, (max(3, T // 100),), generator=g).tolist():
            v[t, int(torch.randint(0, Hkv, (1,), generator=g)), int(torch.randint(0, D, (1,), generator=g))] = x
    v[T - 1] = float("nan")                 # the last token of all
    out = W4.attention_prompt(q, k, v, cu)
    torch.cuda.synchronize()
    check(out[:T], q[:T], k[:T], v[:T], lens)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("n", [40, 200, 1200])
def test_a_score_of_minus_infinity_before_a_hidden_value(n, dtype):
    """The first token scores -inf for every row (weight 0) and a late value is no number."""
    q, k, v, cu = packed([n], 2, 1, 64, dtype, seed=n, fused=False)
    q[..., 5] = q[..., 5].abs() + 1
    k[0, :, 5] = -float("inf")
    v[n - 2, :, 3] = float("inf")
    out = W4.attention_prompt(q, k, v, cu)
    torch.cuda.synchronize()
    # the rows from 1 on as if token 0 were not there (row 0 sees nothing else: no number)
    assert torch.isnan(out[0]).all()
    check(out[1:], q[1:], k[1:], v[1:], [n - 1])


def elapsed(fn):
    fn()
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    a.record()
    for _ in range(3):
        fn()
    b.record()
    torch.cuda.synchronize()
    return a.elapsed_time(b) / 3


@pytest.mark.parametrize("what", ["first token", "one token in 60", "all"])
def test_long_prompts_stay_fast(what):
    """8192 tokens: rows that see a NaN are not walked again, and those before one in their own tile once,
    on the matrix cores (32 keys at a time from memory; at most some 10 times the work of the others)."""
    n, Hq, Hkv, D = 8192, 8, 2, 64
    q, k, v, cu = packed([n], Hq, Hkv, D, torch.bfloat16, seed=4)
    out = torch.empty_like(q)
    clean = elapsed(lambda: W4.attention_prompt(q, k, v, cu, out=out))
    ref = out.clone()
    at = {"first token": slice(0, 1), "one token in 60": slice(59, n, 60), "all": slice(0, n)}[what]
    v[at, :, 3] = float("nan")
    spoiled = elapsed(lambda: W4.attention_prompt(q, k, v, cu, out=out))
    first = at.start
    assert torch.isnan(out[first:, :, 3]).all() and torch.isfinite(out[:first]).all()
    keep = torch.ones(D, dtype=torch.bool, device="cuda")
    keep[3] = False
    # the same weights, perhaps rounded beside another reference: two roundings of each and of the output
    d = (out[..., keep].float() - ref[..., keep].float()).abs()
    assert float(d.max()) <= 4 * 2.0 ** -8 * float(v[..., keep].float().abs().max())
    assert spoiled <= 30 * clean, f"{spoiled:.3f} ms against {clean:.3f}"
