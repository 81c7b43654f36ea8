"""Keys whose addresses pass 32 bits: K caches of more than 4 GiB where a few far tokens of every kv head take
a known share of the weight (test_gpu_attention_limits has the values' side, over keys that are all alike).

A K read at a wrapped or truncated offset would find a token of another score.  Expected: with s the score
of the special tokens and T - 2 others of score 0, weights e^s / Z and 1 / Z, Z = T - 2 + 2 e^s.  Bound: the fp16
rounding of a weight and of the output (2^-11 each), the fp32 error of the score (2 (136 * 19 + 32) 2^-24
< 2^-11) and of Z, 2^24 terms summed over waves, splits and at most 4096 tiles each (2^-11): 2^-9.
"""

from __future__ import annotations

import math

import pytest
import torch

import w4a16_dequant_gemm_amd as W4
from tests.kv_util import make_cache

pytestmark = pytest.mark.gpu
H = torch.float16
T, HKV, D = 1 << 24, 3, 128
FAR = [T // 2 + 12345, T - 1]
BOUND = 2.0 ** -9


@pytest.fixture(scope="module", autouse=True)
def _needs_gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    W4.lib()


@pytest.fixture(scope="module")
def problem():
    def zero():
        return (torch.zeros((1, HKV, T, D), dtype=torch.int8, device="cuda"),
                torch.ones((1, HKV, T), dtype=H, device="cuda"), None)
    k, v = zero(), zero()
    for h in range(HKV):
        for i, t in enumerate(FAR):
            k[0][0, h, t, 0] = 100 + h
            k[1][0, h, t] = 0.25
            v[0][0, h, t] = 3 + 2 * h + i       # (their mean is not the head's before or behind)
    share = []
    for h in range(HKV):
        s = 8.0 * 0.25 * (100 + h) / math.sqrt(D)
        share.append(math.exp(s) / (T - 2 + 2 * math.exp(s)))
    return k, v, share


def query(B):
    q = torch.zeros((B, 2 * HKV, D), dtype=H, device="cuda")
    q[..., 0] = 8.0
    return q


def check(out, share):
    for h in range(2 * HKV):
        hk = h // 2
        want = share[hk] * (3 + 2 * hk + 4 + 2 * hk)
        assert (out[:, h].double() - want).abs().max() <= BOUND * want, h


def test_weights(problem):
    k, v, share = problem
    n = torch.tensor([T], dtype=torch.int32, device="cuda")
    out, sums = W4.kv_attention_decode_weights(query(1), k, v, n, None, 8)
    torch.cuda.synchronize()
    check(out, share)
    for h in range(HKV):
        far = sums[0, h, FAR].double()
        assert (far - 2 * share[h]).abs().max() <= BOUND * 2 * share[h]
        s = 8.0 * 0.25 * (100 + h) / math.sqrt(D)
        rest = sums[0, h].clone()
        rest[FAR] = 2 * share[h] / math.exp(s)
        assert (rest.double() * math.exp(s) / (2 * share[h]) - 1).abs().max() <= BOUND


@pytest.mark.parametrize("B", [1, 20, 40])      # rows streamed, and on two and four waves
def test_shared_prefix(problem, B):
    k, v, share = problem
    own = make_cache((B, HKV, 1, D), 8, H, 1)
    out = W4.kv_attention_decode_shared(query(B), (k[0][0], k[1][0], None), (v[0][0], v[1][0], None), T, own, own,
                                        torch.zeros(B, dtype=torch.int32, device="cuda"), 8)
    torch.cuda.synchronize()
    check(out, share)


def test_eviction(problem):
    k, v, _ = problem
    w = torch.rand((1, HKV, T), device="cuda", generator=torch.Generator(device="cuda").manual_seed(2))
    w[:, :, FAR[0]] = 2.0
    n = torch.tensor([T], dtype=torch.int32, device="cuda")
    budget, recent = 3000, 500
    ko, vo, _, _, kept = W4.kv_evict(k, v, w, n, budget, recent, 8, capacity=budget)
    torch.cuda.synchronize()
    for h in range(HKV):
        at = kept[0, h].long()
        assert int((at == FAR[0]).sum()) == 1 and int(at[-1]) == FAR[1]
        for src, dst in ((k, ko), (v, vo)):
            assert torch.equal(dst[0][0, h], src[0][0, h][at]) and torch.equal(dst[1][0, h], src[1][0, h][at])
        assert int(ko[0][0, h, :, 0].sum()) == 2 * (100 + h)
