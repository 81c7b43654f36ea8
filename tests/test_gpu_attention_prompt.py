"""GPU parity of the prompt attention against softmax(q k^T / sqrt(D)) v in 64 bits.

The reference is NumPy in fp64 on the inputs as given (fp16 / bf16 values are exact there).

Tolerance.  With u = eps / 2 of the type (fp16 2^-11, bf16 2^-8): a weight p_j is rounded once to
the type (relative error <= u; below fp16's smallest normal number, which a weight relative to the
row's running maximum only reaches under 2^-14, an absolute one of 2^-25), the sum of p_j v_j keeps
fp32, the output is rounded once.  So

    |out - ref| <= u |ref| + (1 + u) (u + e) sum_j p_j |v_j| + n 2^-25 max|v|,

where e bounds the relative error of a weight in fp32.  A score s = q . k / sqrt(D) has an fp32
error of at most (D + 8) 2^-24 sum_d |q_d k_d| / sqrt(D), which the exponential turns into a
relative one of the same size; D = 128 and rows of N(0, 1) entries scaled by up to 4 keep
sum |q k| / sqrt(D) below 400, so e < 136 * 2^-24 * 400 + 2^-18 < 0.0033; a row's normalization
shares the error of its weights, which doubles it.  For these bounds the computed quantity
sum_j p_j |v_j| is used per element, not a norm; the bf16 bound is dominated by u = 2^-8.
For the plain N(0, 1) rows of most cases sum |q k| / sqrt(D) < 24: e < 2 (136 * 24 + 64) 2^-24 <
4.0e-4.
"""

from __future__ import annotations

import numpy as np
import pytest
import torch

import w4a16_dequant_gemm_amd as W4

pytestmark = pytest.mark.gpu

U = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
E = 4.0e-4


@pytest.fixture(scope="module", autouse=True)
def _needs_gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    W4.lib()


def f64(t):
    return t.detach().cpu().double().numpy()


def reference(q, k, v, lens, first=0):
    """``(out, sum_j p_j |v_j|)`` of the packed sequences, in fp64; rows outside are NaN."""
    T, Hq, D = q.shape
    G = Hq // k.shape[1]
    out = np.full((T, Hq, D), np.nan)
    mag = np.full((T, Hq, D), np.nan)
    at = first
    for n in lens:
        hide = np.triu(np.ones((n, n), bool), 1)
        for h in range(Hq):
            s = q[at:at + n, h] @ k[at:at + n, h // G].T / np.sqrt(D)
            s[hide] = -np.inf
            p = np.exp(s - s.max(1, keepdims=True)) if n else s
            p /= p.sum(1, keepdims=True)
            out[at:at + n, h] = p @ v[at:at + n, h // G]
            mag[at:at + n, h] = p @ np.abs(v[at:at + n, h // G])
        at += n
    return out, mag


def check(got, q, k, v, lens, first=0, e=E):
    ref, mag = reference(f64(q), f64(k), f64(v), lens, first)
    a, b = first, first + sum(lens)
    u = U[q.dtype]
    tol = u * np.abs(ref[a:b]) + (1 + u) * (u + e) * mag[a:b] + max(lens, default=0) * 2.0 ** -25 * np.abs(
        f64(v)[a:b]).max(initial=0.0)
    g = f64(got)[a:b]
    assert np.all(np.isfinite(g))
    bad = np.abs(g - ref[a:b]) > tol
    assert not bad.any(), f"{bad.sum()} of {bad.size} outside, worst {np.max(np.abs(g - ref[a:b]) / tol):.2f} x"


def packed(lens, Hq, Hkv, D, dtype, seed, pad=0, fused=True, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    T = sum(lens) + pad
    x = torch.randn((T, (Hq + 2 * Hkv) * D), generator=g).mul_(scale).to(dtype).cuda()
    q, k, v = x.split([Hq * D, Hkv * D, Hkv * D], dim=1)
    if not fused:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")
    return q.unflatten(1, (Hq, D)), k.unflatten(1, (Hkv, D)), v.unflatten(1, (Hkv, D)), cu


# lengths around the wave's 32 rows, the block's rows and the 64-key tiles; empty sequences first,
# in the middle and last; head groups of 1, 2, 3 and 8
CASES = [([1], 1, 1, 64, torch.float16), ([1, 1, 1], 8, 2, 128, torch.bfloat16), ([2, 31, 32, 33], 4, 4, 64, torch.bfloat16),
         ([63, 64, 65], 3, 1, 128, torch.float16), ([127, 128, 129], 2, 2, 128, torch.bfloat16),
         ([0, 5, 0, 0, 70, 0], 6, 2, 64, torch.float16), ([255, 256, 257, 1], 8, 1, 128, torch.float16),
         ([513], 4, 2, 64, torch.float16), ([1000, 3, 200], 2, 1, 128, torch.bfloat16),
         ([0], 2, 1, 64, torch.float16), ([1537], 2, 2, 128, torch.float16),
         # few blocks of many tiles: two groups of waves, the second with and without tiles of its own
         ([1024], 2, 1, 64, torch.bfloat16), ([1025], 4, 2, 128, torch.bfloat16), ([2047, 1], 2, 2, 64, torch.float16),
         ([1, 2047], 1, 1, 128, torch.float16), ([0, 2111, 33, 960], 3, 1, 128, torch.bfloat16), ([1900, 64, 0], 2, 1, 64, torch.float16),
         ([1023], 4, 2, 128, torch.bfloat16)]


@pytest.mark.parametrize("lens,Hq,Hkv,D,dtype", CASES)
def test_packed_prompts(lens, Hq, Hkv, D, dtype):
    q, k, v, cu = packed(lens, Hq, Hkv, D, dtype, seed=sum(lens) + D, pad=3)
    out = W4.attention_prompt(q, k, v, cu)
    torch.cuda.synchronize()
    check(out, q, k, v, lens)


@pytest.mark.parametrize("B", [63, 64, 65, 130, 4200])
def test_many_short_sequences(B):
    lens = [(7 * i) % 5 + (90 if i % 61 == 0 else 0) for i in range(B)]      # some of them empty
    q, k, v, cu = packed(lens, 2, 1, 64, torch.bfloat16, seed=B)
    out = W4.attention_prompt(q, k, v, cu)
    torch.cuda.synchronize()
    check(out, q, k, v, lens)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("D", [64, 128])
def test_rows_outside_are_neither_read_nor_written(D, dtype):
    """Rows before the first and behind the last sequence hold NaN and infinities, also the next
    sequence of a batch does not reach into its neighbour's tile."""
    lens, first, pad = [70, 40, 150], 9, 21
    T = first + sum(lens) + pad
    g = torch.Generator().manual_seed(11)
    x = torch.randn((T, 8 * D), generator=g).to(dtype)
    x[:first] = float("nan")
    x[first + sum(lens):] = float("inf")
    x = x.cuda()
    q, k, v = (t.unflatten(1, (-1, D)) for t in x.split([4 * D, 2 * D, 2 * D], dim=1))
    cu = torch.tensor(np.cumsum([first, *lens]), dtype=torch.int32, device="cuda")
    out = torch.full((T, 4, D), 7.0, dtype=dtype, device="cuda")
    got = W4.attention_prompt(q, k, v, cu, out=out)
    torch.cuda.synchronize()
    assert got.data_ptr() == out.data_ptr()
    check(out, q, k, v, lens, first)
    assert (out[:first] == 7.0).all() and (out[first + sum(lens):] == 7.0).all()


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_nan_in_one_sequence_stays_there(dtype):
    lens = [50, 30, 81]
    q, k, v, cu = packed(lens, 2, 1, 64, dtype, seed=5, fused=False)
    clean = W4.attention_prompt(q, k, v, cu)
    k2, v2 = k.clone(), v.clone()
    k2[50:80] = float("nan")
    v2[50:80] = float("inf")
    out = W4.attention_prompt(q, k2, v2, cu)
    torch.cuda.synchronize()
    assert torch.equal(out[:50], clean[:50]) and torch.equal(out[80:], clean[80:])


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n,at", [(200, 100), (200, 40), (129, 128), (64, 63), (33, 1), (700, 650), (1300, 1290), (1200, 1)])
def test_later_tokens_without_numbers_are_not_seen(n, at, D, dtype):
    """Infinities and NaN in the key and the value of one token: the rows before it as if it were not there,
    those from it on without numbers where they should be."""
    q, k, v, cu = packed([n], 2, 1, D, dtype, seed=n + at, fused=False)
    for what in ("value", "key", "both"):
        k2, v2 = k.clone(), v.clone()
        if what != "value":
            k2[at] = float("nan")
        if what != "key":
            v2[at, :, 3] = float("inf")
            v2[at, :, 9] = float("nan")
        out = W4.attention_prompt(q, k2, v2, cu)
        torch.cuda.synchronize()
        check(out[:at], q[:at], k[:at], v[:at], [at])
        if what == "value":
            assert torch.isinf(out[at:, :, 3]).all() and torch.isnan(out[at:, :, 9]).all()
            some = torch.ones(D, dtype=torch.bool)
            some[[3, 9]] = False
            ref, mag = (x[at:, :, some.numpy()] for x in reference(f64(q), f64(k), f64(v), [n]))
            u = U[dtype]                                   # the bound of check()
            tol = u * np.abs(ref) + (1 + u) * (u + E) * mag + n * 2.0 ** -25 * np.abs(f64(v)).max()
            assert (np.abs(f64(out)[at:, :, some.numpy()] - ref) <= tol).all()
        else:
            assert torch.isnan(out[at:]).all()


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("n", [700, 1400])
def test_peaked_scores_rising_along_the_row(dtype, n):
    """Scores that rise by far more than the kernel's rescaling threshold, tile after tile, and
    then fall: the running maximum moves often, and late tiles weigh nothing."""
    D = 64
    g = torch.Generator().manual_seed(3)
    q = torch.randn((n, 1, D), generator=g)
    k = torch.randn((n, 1, D), generator=g)
    q[..., 0] = 4.0
    k[..., 0] = torch.cat([torch.linspace(-30, 60, 400), torch.linspace(60, -30, n - 400)])[:, None]
    q, k = q.to(dtype).cuda(), k.to(dtype).cuda()
    v = torch.randn((n, 1, D), generator=g).to(dtype).cuda()
    cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    out = W4.attention_prompt(q, k, v, cu)
    torch.cuda.synchronize()
    # sum_d |q_d k_d| / 8 <= 4 * 60 / 8 + 24: e < 2 (72 * 54 + 64) 2^-24 < 4.8e-4
    check(out, q, k, v, [n], e=4.8e-4)


@pytest.mark.parametrize("n", [130, 1400])
def test_large_finite_scores_give_the_largest_key(n):
    """fp16 inputs near the type's largest value: scores of 1e10 and more, one key wins outright."""
    D = 64
    q = torch.full((n, 1, D), 60000.0, dtype=torch.float16, device="cuda")
    k = torch.full((n, 1, D), -60000.0, dtype=torch.float16, device="cuda")
    k[0] = 60000.0
    k[100] = 65504.0
    v = torch.arange(n, device="cuda", dtype=torch.float16)[:, None, None].expand(n, 1, D).contiguous()
    out = W4.attention_prompt(q, k, v, torch.tensor([0, n], dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    want = torch.where(torch.arange(n, device="cuda") < 100, 0.0, 100.0).half()
    assert torch.equal(out[:, 0, 0], want) and torch.equal(out[:, 0, D - 1], want)


def test_row_strides():
    """q, k and v with row strides of their own, larger than their rows."""
    lens, D = [90, 45], 128
    g = torch.Generator().manual_seed(17)
    T = sum(lens)
    big = [torch.randn((T, w), generator=g).to(torch.float16).cuda() for w in (3 * D + 8, 2 * D + 40, 5 * D)]
    q = big[0][:, 8:8 + 2 * D].unflatten(1, (2, D))
    k = big[1][:, :D].unflatten(1, (1, D))
    v = big[2][:, D:2 * D].unflatten(1, (1, D))
    cu = torch.tensor([0, 90, 135], dtype=torch.int32, device="cuda")
    out = W4.attention_prompt(q, k, v, cu)
    torch.cuda.synchronize()
    check(out, q, k, v, lens)


def test_bad_bounds_stay_inside():
    """Bounds outside [0, T] are clamped: the valid sequences of the batch come out right."""
    lens = [40, 60]
    q, k, v, _ = packed(lens, 2, 1, 64, torch.float16, seed=23)
    cu = torch.tensor([-5, 40, 1 << 30], dtype=torch.int32, device="cuda")
    out = W4.attention_prompt(q, k, v, cu)
    torch.cuda.synchronize()
    check(out, q, k, v, lens)


def test_refusals():
    q, k, v, cu = packed([40], 4, 2, 64, torch.float16, seed=1, fused=False)
    with pytest.raises(TypeError):
        W4.attention_prompt(q.float(), k, v, cu)
    with pytest.raises(TypeError):
        W4.attention_prompt(q, k.bfloat16(), v, cu)
    with pytest.raises(TypeError):
        W4.attention_prompt(q, k, v, cu.long())
    with pytest.raises(ValueError):
        W4.attention_prompt(q, k[:39], v[:39], cu)
    with pytest.raises(ValueError):
        W4.attention_prompt(q, k, v, cu[:1])
    with pytest.raises(ValueError):
        W4.attention_prompt(q, k, v, cu.cpu())
    with pytest.raises(ValueError):
        W4.attention_prompt(q, k.transpose(0, 1).contiguous().transpose(0, 1), v, cu)   # heads apart
    with pytest.raises(ValueError):
        W4.attention_prompt(q, k, v, cu, out=torch.empty((40, 4, 32), dtype=torch.float16, device="cuda"))
    with pytest.raises(W4.W4A16Error):
        W4.attention_prompt(q[:, :3], k, v, cu)                                         # 3 heads on 2
    with pytest.raises(W4.W4A16Error):
        W4.attention_prompt(q[..., :32].contiguous(), k[..., :32].contiguous(), v[..., :32].contiguous(), cu)


def test_other_stream_and_repeat_are_identical():
    q, k, v, cu = packed([300, 200], 4, 2, 128, torch.bfloat16, seed=2)
    a = W4.attention_prompt(q, k, v, cu)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        b = W4.attention_prompt(q, k, v, cu)
    st.synchronize()
    assert torch.equal(a.view(torch.int16), b.view(torch.int16))
