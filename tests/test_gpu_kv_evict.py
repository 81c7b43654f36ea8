"""GPU tests of the cache eviction: what is kept equals a stable sort of the weights on the host, and
the kept rows are the same bits; prompts, decode steps with accumulated weights, eviction and
further decoding run together."""

from __future__ import annotations

import numpy as np
import pytest
import torch

import w4a16_dequant_gemm_amd as W4
from tests.kv_util import attend, check_out, cmax, f64, make_cache, rows, weight_error

pytestmark = pytest.mark.gpu
H, BF = torch.float16, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _needs_gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    W4.lib()


def raw_cache(B, Hkv, T, D, bits, seed):
    g = torch.Generator().manual_seed(seed)
    shape = (B, Hkv, T)
    if bits == 8:
        codes = torch.randint(-128, 128, shape + (D,), generator=g).to(torch.int8)
    else:
        codes = torch.randint(-(1 << 31), 1 << 31, shape + (D // 8,), generator=g).to(torch.int32)
    scales = torch.rand(shape, generator=g).half()
    zeros = torch.randint(0, 16, shape, generator=g).half() if bits == 4 else None
    return tuple(None if t is None else t.cuda() for t in (codes, scales, zeros))


def expected(w, n, budget, recent):
    """Indices kept of the first ``n`` weights ``w`` (fp32, host)."""
    if n <= budget:
        return np.arange(n)
    old = n - recent
    key = np.where(np.isnan(w[:old]), np.inf, w[:old].astype(np.float64))
    # NaN above infinity: two keys, stable
    order = np.lexsort((np.arange(old), -key, ~np.isnan(w[:old])))
    return np.concatenate([np.sort(order[:budget - recent]), np.arange(old, n)])


def run_and_check(w, lens, D, bits, budget, recent, capacity=None, seed=0, into=False):
    B, Hkv, T = w.shape
    k, v = raw_cache(B, Hkv, T, D, bits, seed), raw_cache(B, Hkv, T, D, bits, seed + 1)
    wt = torch.from_numpy(w).cuda()
    lt = torch.tensor(lens, dtype=torch.int32, device="cuda")
    C = T if capacity is None else capacity
    out = None
    if into:
        new = lambda c: tuple(None if t is None else torch.full((B, Hkv, C) + t.shape[3:], 5, dtype=t.dtype, device="cuda")
                              for t in c)
        out = (new(k), new(v), torch.full((B, Hkv, C), 5.0, device="cuda"), torch.zeros(B, dtype=torch.int32, device="cuda"),
               torch.zeros((B, Hkv, budget), dtype=torch.int32, device="cuda"))
    ko, vo, wo, lo, kept = W4.kv_evict(k, v, wt, lt, budget, recent, bits, capacity=capacity, out=out)
    torch.cuda.synchronize()
    assert ko[1].shape == (B, Hkv, C)
    for b, n in enumerate(lens):
        n = min(max(n, 0), T)
        c = min(n, budget)
        assert int(lo[b]) == c
        for h in range(Hkv):
            want = expected(w[b, h], n, budget, recent)
            got = kept[b, h].cpu().numpy()
            np.testing.assert_array_equal(got[:c], want)
            assert (got[c:] == -1).all()
            at = torch.from_numpy(want).cuda()
            for src, dst in ((k, ko), (v, vo)):
                for s, d in zip(src, dst):
                    if s is not None:
                        assert torch.equal(d[b, h, :c], s[b, h][at])
                        if into:
                            assert (d[b, h, c:] == 5).all()
            assert torch.equal(wo[b, h, :c].view(torch.int32), wt[b, h][at].view(torch.int32))
            assert (wo[b, h, c:] == 0).all()


def heavy(shape, seed):
    return np.exp(np.random.default_rng(seed).normal(-3, 2, shape)).astype(np.float32)


# (B, Hkv, T, lens, budget, recent, D, bits): budgets of one, all recent, none recent, one above and
# below the length, sequences shorter than the budget and empty ones, lengths outside the room
CASES = [(1, 1, 1, [1], 1, 0, 64, 8), (1, 1, 2, [2], 1, 0, 64, 4), (1, 1, 2, [2], 1, 1, 128, 8),
         (3, 2, 65, [65, 64, 0], 64, 10, 64, 8), (2, 3, 130, [129, 3], 128, 128, 128, 4),
         (4, 1, 1000, [1000, 999, 500, -4], 500, 0, 128, 8), (2, 2, 1025, [1025, 5000], 17, 5, 64, 4),
         (1, 2, 5001, [5001], 2048, 100, 128, 4), (2, 1, 300, [300, 40], 400, 50, 64, 8),
         (1, 1, 20011, [20011], 20010, 1, 64, 8), (1, 2, 8192, [8192], 4000, 8, 64, 4), (2, 1, 8193, [8193, 100], 5000, 4500, 64, 8),
         (3, 2, 30000, [30000, 9000, 0], 9000, 20, 64, 8), (2, 1, 25000, [25000, 16385], 16384, 16384, 64, 4),
         (1, 1, 600001, [600001], 70000, 66000, 64, 4), (2, 1, 40000, [40000, 39999], 12000, 11990, 64, 8),
         # kept rows of 64 KB, the most that the selecting block copies, and one row more
         (3, 2, 3001, [3001, 512, 700], 512, 30, 128, 8), (3, 2, 3001, [3001, 513, 700], 513, 30, 128, 8),
         (1, 3, 4000, [4000], 2048, 0, 64, 4), (1, 3, 4000, [4000], 2049, 2049, 64, 4),
         (2, 1, 8192, [8192, 1], 1024, 1, 128, 4), (2, 1, 8192, [8192, 1025], 1025, 1, 64, 8)]


@pytest.mark.parametrize("B,Hkv,T,lens,budget,recent,D,bits", CASES)
def test_evict(B, Hkv, T, lens, budget, recent, D, bits):
    run_and_check(heavy((B, Hkv, T), T), lens, D, bits, budget, recent, seed=T)
    run_and_check(heavy((B, Hkv, T), T + 1), lens, D, bits, budget, recent, capacity=min(budget, T) + 3, seed=T, into=True)


@pytest.mark.parametrize("T", [700, 5000, 70001, 131100])
def test_ties_zeros_and_special_weights(T):
    """Few different values (ties everywhere, also between waves), all equal, all zero with both
    signs, negative values, infinities and NaN."""
    rng = np.random.default_rng(T)
    w = np.zeros((1, 6, T), np.float32)
    w[0, 0] = rng.integers(0, 3, T)
    w[0, 1] = 1.5
    w[0, 2] = np.where(rng.random(T) < 0.5, 0.0, -0.0)
    w[0, 3] = rng.normal(0, 1, T)
    w[0, 4] = heavy(T, T)
    w[0, 4, rng.integers(0, T, 9)] = np.inf
    w[0, 4, rng.integers(0, T, 9)] = np.nan
    w[0, 4, rng.integers(0, T, 9)] = -np.nan
    w[0, 4, rng.integers(0, T, 9)] = -np.inf
    w[0, 5] = rng.choice(np.array([1e-42, 2e-42, 3e-38, 1e-40], np.float32), T)      # subnormal weights
    for budget, recent in ((T // 2, 30), (9, 0), (T - 1, T // 3)):
        run_and_check(w, [T], 64, 8, budget, recent, seed=3)


def test_in_place_is_refused():
    k, v = raw_cache(1, 1, 64, 64, 8, 0), raw_cache(1, 1, 64, 64, 8, 1)
    w = torch.rand((1, 1, 64), device="cuda")
    n = torch.tensor([64], dtype=torch.int32, device="cuda")
    room = lambda c: tuple(None if t is None else torch.empty_like(t) for t in c)
    ok = (room(k), room(v), torch.empty_like(w), torch.empty_like(n), torch.empty((1, 1, 32), dtype=torch.int32, device="cuda"))
    W4.kv_evict(k, v, w, n, 32, 8, 8, out=ok)
    for i, own in enumerate((k, v, w, n)):
        bad = list(ok)
        bad[i] = own
        with pytest.raises(W4.W4A16Error):
            W4.kv_evict(k, v, w, n, 32, 8, 8, out=tuple(bad))
    with pytest.raises(W4.W4A16Error):
        W4.kv_evict(k, v, w, n, 32, 8, 8, out=(ok[0], ok[0], *ok[2:]))


def test_refusals():
    k, v = raw_cache(2, 1, 20, 64, 8, 0), raw_cache(2, 1, 20, 64, 8, 1)
    w = torch.rand((2, 1, 20), device="cuda")
    n = torch.tensor([20, 3], dtype=torch.int32, device="cuda")
    for budget, recent in ((0, 0), (5, 6), (5, -1), (-3, 0)):
        with pytest.raises(ValueError):
            W4.kv_evict(k, v, w, n, budget, recent, 8)
    with pytest.raises(ValueError):
        W4.kv_evict(k, v, w, n, 10, 2, 8, capacity=9)
    with pytest.raises(ValueError):
        W4.kv_evict(k, v, w[:, :, :19].contiguous(), n, 10, 2, 8)
    with pytest.raises(ValueError):
        W4.kv_evict(k, v, w, n[:1], 10, 2, 8)
    with pytest.raises(TypeError):
        W4.kv_evict(k, v, w.half(), n, 10, 2, 8)
    with pytest.raises(TypeError):
        W4.kv_evict(k, v, w, n, 10, 2, 4)
    with pytest.raises(ValueError):
        W4.kv_evict(k, v, w, n, 10, 2, 3)


@pytest.mark.parametrize("bits", [8, 4])
def test_prompt_decode_evict_decode(bits):
    """A serving loop of two sequences: prompt attention, quantized cache, decode steps that add up
    attention, eviction, a decode step over what is left; every output against fp64."""
    B, Hq, Hkv, D, dtype = 2, 4, 2, 64, H
    lens, steps, Tmax, budget, recent = [150, 90], 6, 160, 64, 16
    g = torch.Generator().manual_seed(bits)
    T = sum(lens)
    qkv = torch.randn((T, (Hq + 2 * Hkv) * D), generator=g).to(dtype).cuda()
    q, k, v = (t.unflatten(1, (-1, D)) for t in qkv.split([Hq * D, Hkv * D, Hkv * D], dim=1))
    cu = torch.tensor([0, 150, 240], dtype=torch.int32, device="cuda")
    out = W4.attention_prompt(q, k, v, cu)
    G = Hq // Hkv
    at = 0
    for n in lens:
        for h in range(Hq):
            for i in (0, 63, n - 1):
                ref, _, mag, qk = attend(f64(q)[at + i:at + i + 1, h], f64(k)[at:at + i + 1, h // G], f64(v)[at:at + i + 1, h // G])
                check_out(f64(out)[at + i:at + i + 1, h], ref, mag, dtype, weight_error(D, qk), n, 4.0, 1.0)
        at += n

    dense = [torch.zeros((B, Hkv, Tmax, D), dtype=dtype, device="cuda") for _ in range(2)]
    for b, (a, n) in enumerate(((0, 150), (150, 90))):
        for d, t in zip(dense, (k, v)):
            d[b, :, :n] = t[a:a + n].transpose(0, 1)
    caches = []
    for d in dense:
        c, s, z = W4.kv_quantize(d.view(B * Hkv, Tmax, D), bits)
        caches.append((c.view(B, Hkv, Tmax, -1), s.view(B, Hkv, Tmax), None if z is None else z.view(B, Hkv, Tmax)))
    kc, vc = caches
    lt = torch.tensor(lens, dtype=torch.int32, device="cuda")
    weights = torch.zeros((B, Hkv, Tmax), device="cuda")
    total = np.zeros((B, Hkv, Tmax))

    def step(kc, vc, lt, weights):
        qd = torch.randn((B, Hq, D), generator=g).to(dtype).cuda()
        o, w = W4.kv_attention_decode_weights(qd, kc, vc, lt, weights, bits)
        K, V = rows(kc, bits), rows(vc, bits)
        ps = []
        for b in range(B):
            n = int(lt[b])
            for hk in range(Hkv):
                hs = slice(hk * G, hk * G + G)
                ref, p, mag, qk = attend(f64(qd)[b, hs], K[b, hk, :n], V[b, hk, :n])
                check_out(f64(o)[b, hs], ref, mag, dtype, weight_error(D, qk), n, f64(vc[1])[b, :, :n].max(),
                          cmax((None, None, vc[2][b, :, :n] if vc[2] is not None else None), bits))
                ps.append((b, hk, n, p.sum(0)))
        return ps

    def append(kc, vc, lt, room):
        """A token's keys and values, quantized by a call on its rows, into slot lengths[b]."""
        for c in (kc, vc):
            x = torch.randn((B * Hkv, 1, D), generator=g).to(dtype).cuda()
            new = W4.kv_quantize(x, bits)
            for b in range(B):
                n = int(lt[b])
                assert n < room
                for dst, src in zip(c, new):
                    if dst is not None:
                        dst[b, :, n] = src.view(B, Hkv, 1, -1)[b, :, 0] if dst.dim() == 4 else src.view(B, Hkv)[b]
        return lt + 1

    for _ in range(steps):
        lt = append(kc, vc, lt, Tmax)
        for b, hk, n, p in step(kc, vc, lt, weights):
            total[b, hk, :n] += p
    np.testing.assert_allclose(f64(weights), total, rtol=steps * 4e-4, atol=1e-9)

    kc, vc, weights, lt, kept = W4.kv_evict(kc, vc, weights, lt, budget, recent, bits, capacity=budget + 8)
    assert lt.tolist() == [64, 64]
    carried = f64(weights).copy()
    for b in range(B):
        for hk in range(Hkv):
            np.testing.assert_allclose(carried[b, hk, :64], total[b, hk][kept[b, hk].cpu().numpy()], rtol=steps * 4e-4)
    lt = append(kc, vc, lt, budget + 8)
    for b, hk, n, p in step(kc, vc, lt, weights):
        carried[b, hk, :n] += p
    np.testing.assert_allclose(f64(weights), carried, rtol=7 * 4e-4, atol=1e-9)
