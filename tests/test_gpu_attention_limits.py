"""The attention and eviction entry points where addresses pass 32 bits, on two streams at once and (where
there is one) on a second GPU."""

from __future__ import annotations

import numpy as np
import pytest
import torch

import w4a16_dequant_gemm_amd as W4
from tests.kv_util import make_cache

pytestmark = pytest.mark.gpu
H = torch.float16


@pytest.fixture(scope="module", autouse=True)
def _needs_gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    W4.lib()


def long_cache(T, Hkv, D=128):
    """KV8 caches ``[1, Hkv, T, D]`` of zero codes, more than 4 GiB each: every token scores the same."""
    codes = torch.zeros((1, Hkv, T, D), dtype=torch.int8, device="cuda")
    scales = torch.ones((1, Hkv, T), dtype=H, device="cuda")
    return codes, scales, None


def test_cache_offsets_past_32_bits():
    """2^24 tokens and three kv heads: weights of 1 / T each, the last token alone has a value, so each
    output is 127 scale / T; then an eviction that keeps tokens from both ends."""
    T, Hkv, D = 1 << 24, 3, 128
    k, v = long_cache(T, Hkv), long_cache(T, Hkv)
    for h in range(Hkv):
        v[0][0, h, T - 1] = 127
        v[1][0, h, T - 1] = 20000.0 * (h + 1)
    q = torch.randn((1, 2 * Hkv, D), device="cuda").to(H)
    n = torch.tensor([T], dtype=torch.int32, device="cuda")
    out, sums = W4.kv_attention_decode_weights(q, k, v, n, None, 8)
    torch.cuda.synchronize()
    for h in range(2 * Hkv):
        want = 127 * 20000.0 * (h // 2 + 1) / T
        # the rounding of the weight and of the output, and 2^24 equal terms summed in fp32 (pairwise over
        # waves, splits and 4096 tiles each: relative 2^-24 * 2 * 4096 at most)
        assert (out[0, h].double() - want).abs().max() <= want * (2.0 ** -10 + 2.0 ** -11)
    assert (sums.double() * T - 2.0).abs().max() <= 2 * 2.0 ** -10
    # the same tokens as a shared prefix, with nothing after it
    one = torch.zeros(1, dtype=torch.int32, device="cuda")
    small = make_cache((1, Hkv, 1, D), 8, H, 1)
    pre = W4.kv_attention_decode_shared(q, tuple(t[0] if t is not None else None for t in k),
                                        tuple(t[0] if t is not None else None for t in v), T, small, small, one, 8)
    torch.cuda.synchronize()
    assert (pre.double() - out.double()).abs().max() <= out.double().abs().max() * 2.0 ** -9
    del out, sums

    g = torch.Generator(device="cuda").manual_seed(3)
    w = torch.rand((1, Hkv, T), generator=g, device="cuda")
    budget, recent = 5000, 1000
    ko, vo, wo, lo, kept = W4.kv_evict(k, v, w, n, budget, recent, 8, capacity=budget)
    torch.cuda.synchronize()
    assert int(lo[0]) == budget
    for h in range(Hkv):
        order = torch.sort(w[0, h, :T - recent], descending=True, stable=True)[1][:budget - recent]
        want = torch.cat([order.sort()[0], torch.arange(T - recent, T, device="cuda")])
        assert torch.equal(kept[0, h].long(), want)
        assert torch.equal(wo[0, h], w[0, h][want])
        assert (vo[0][0, h, -1] == 127).all() and (vo[0][0, h, :-1] == 0).all()
        assert float(vo[1][0, h, -1]) == float(v[1][0, h, T - 1])


def test_prompt_offsets_past_32_bits():
    """Rows 2^23 elements apart: 600 of them span 10 GB."""
    n, D, stride = 600, 64, 1 << 23
    base = torch.empty((n, stride), dtype=H, device="cuda")
    g = torch.Generator().manual_seed(5)
    x = torch.randn((n, 4 * D), generator=g).to(H)
    base[:, stride - 4 * D:] = x.cuda()
    wide = base[:, stride - 4 * D:]
    q, k, v = (t.unflatten(1, (-1, D)) for t in wide.split([2 * D, D, D], dim=1))
    cu = torch.tensor([0, 70, n], dtype=torch.int32, device="cuda")
    out = W4.attention_prompt(q, k, v, cu)
    ref = W4.attention_prompt(q.contiguous(), k.contiguous(), v.contiguous(), cu)
    torch.cuda.synchronize()
    assert torch.equal(out, ref)


def test_two_streams_at_once():
    """The same calls on two streams without a wait between them, each with the workspace it allocates."""
    B, Hq, Hkv, D, P, T = 8, 8, 2, 128, 3000, 9000
    q = [torch.randn((B, Hq, D), device="cuda").to(H) for _ in range(2)]
    kp, vp = make_cache((Hkv, P, D), 8, H, 1), make_cache((Hkv, P, D), 8, H, 2)
    k, v = make_cache((B, Hkv, T, D), 8, H, 3), make_cache((B, Hkv, T, D), 8, H, 4)
    w = torch.rand((B, Hkv, T), device="cuda")
    n = torch.tensor([T - 7 * i for i in range(B)], dtype=torch.int32, device="cuda")

    def run(i):
        a = W4.kv_attention_decode_shared(q[i], kp, vp, P, k, v, n, 8)
        b, s = W4.kv_attention_decode_weights(q[i], k, v, n, w, 8, sums=torch.zeros_like(w))
        e = W4.kv_evict(k, v, s, n, 4000, 100, 8, capacity=4000)
        return [a, b, s, e[2], e[4], e[0][0], e[1][1]]
    want = [run(0), run(1)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(3):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i].append(run(i))
    torch.cuda.synchronize()
    for i in range(2):
        for r in got[i]:
            for a, b in zip(r, want[i]):
                assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


@pytest.mark.skipif(torch.cuda.device_count() < 2, reason="needs two GPUs")
def test_tensors_on_a_device_that_is_not_current():
    q = torch.randn((50, 2, 64), device="cuda:1").to(H)
    cu = torch.tensor([0, 50], dtype=torch.int32, device="cuda:1")
    with torch.cuda.device(0):
        out = W4.attention_prompt(q, q, q, cu)
    with torch.cuda.device(1):
        ref = W4.attention_prompt(q, q, q, cu)
    torch.cuda.synchronize(1)
    assert torch.equal(out, ref)
    with pytest.raises(ValueError):
        W4.attention_prompt(q, q.to("cuda:0"), q, cu)


def test_single_tokens_and_single_rows():
    """Batches of one-token prompts: the value row itself, at every head layout."""
    for Hq, Hkv, D in ((1, 1, 64), (8, 1, 128), (6, 3, 64)):
        n = 70
        q = torch.randn((n, Hq, D), device="cuda").to(H)
        k = torch.randn((n, Hkv, D), device="cuda").to(H)
        v = torch.randn((n, Hkv, D), device="cuda").to(H)
        out = W4.attention_prompt(q, k, v, torch.arange(n + 1, dtype=torch.int32, device="cuda"))
        torch.cuda.synchronize()
        want = v.repeat_interleave(Hq // Hkv, dim=1)
        assert torch.equal(out, want)
        assert np.isfinite(out.float().cpu().numpy()).all()
