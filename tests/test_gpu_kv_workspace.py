"""One workspace, of the size of a program's largest call, under smaller calls that split their work more
finely: nothing behind it is written, and the results are those of the calls' own workspaces."""

from __future__ import annotations

import pytest
import torch

import w4a16_dequant_gemm_amd as W4
from tests.kv_util import make_cache

pytestmark = pytest.mark.gpu
H = torch.float16
GUARD = 1 << 23         # more than any of the calls below uses in all


@pytest.fixture(scope="module", autouse=True)
def _needs_gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    W4.lib()


def guarded(need):
    return torch.full((need + GUARD,), 12345.0, device="cuda")


def same(a, b):
    return torch.equal(a.view(torch.uint8), b.view(torch.uint8))


@pytest.mark.parametrize("big,B,P,T", [((32, 16385, 40), 32, 16384, 40), ((64, 600, 400), 4, 600, 400),
                                       ((33, 5000, 300), 17, 2500, 300), ((40, 800, 220), 1, 790, 220)])
def test_shared(big, B, P, T):
    Hq, Hkv, D = 8, 2, 64
    q = torch.randn((B, Hq, D), device="cuda").to(H)
    kp, vp = make_cache((Hkv, P, D), 8, H, 1), make_cache((Hkv, P, D), 8, H, 2)
    k, v = make_cache((B, Hkv, T, D), 8, H, 3), make_cache((B, Hkv, T, D), 8, H, 4)
    n = torch.tensor([T - i % T for i in range(B)], dtype=torch.int32, device="cuda")
    need = W4.kv_attention_shared_workspace(big[0], Hq, Hkv, big[1], big[2], D)
    assert need >= W4.kv_attention_shared_workspace(B, Hq, Hkv, P, T, D)
    work = guarded(need)
    out = W4.kv_attention_decode_shared(q, kp, vp, P, k, v, n, 8, work=work)
    want = W4.kv_attention_decode_shared(q, kp, vp, P, k, v, n, 8)
    torch.cuda.synchronize()
    assert (work[need:] == 12345.0).all() and same(out, want)


@pytest.mark.parametrize("big,B,T", [((8, 8193), 8, 8192), ((8, 1100), 2, 1024), ((300, 600), 3, 590)])
def test_weights(big, B, T):
    Hq, Hkv, D = 8, 2, 64
    q = torch.randn((B, Hq, D), device="cuda").to(H)
    k, v = make_cache((B, Hkv, T, D), 8, H, 3), make_cache((B, Hkv, T, D), 8, H, 4)
    n = torch.tensor([T - 3 * i for i in range(B)], dtype=torch.int32, device="cuda")
    need = W4.kv_attention_weights_workspace(big[0], Hq, Hkv, big[1], D)
    assert need >= W4.kv_attention_weights_workspace(B, Hq, Hkv, T, D)
    work = guarded(need)
    got = W4.kv_attention_decode_weights(q, k, v, n, None, 8, work=work)
    want = W4.kv_attention_decode_weights(q, k, v, n, None, 8)
    torch.cuda.synchronize()
    assert (work[need:] == 12345.0).all() and all(same(a, b) for a, b in zip(got, want))


def test_evict():
    """524288 tokens are cut into more chunks than 524289."""
    T, D = 524288, 64
    need = W4.kv_evict_workspace(1, 1, T + 1)
    assert need >= W4.kv_evict_workspace(1, 1, T)
    c = torch.zeros((1, 1, T, D), dtype=torch.int8, device="cuda")
    cache = (c, torch.ones((1, 1, T), dtype=H, device="cuda"), None)
    w = torch.rand((1, 1, T), device="cuda")
    n = torch.tensor([T], dtype=torch.int32, device="cuda")
    work = guarded(need)
    got = W4.kv_evict(cache, cache, w, n, 1000, 10, 8, capacity=1000, work=work)
    torch.cuda.synchronize()
    assert (work[need:] == 12345.0).all()
    want = torch.cat([torch.sort(w[0, 0, :T - 10], descending=True, stable=True)[1][:990].sort()[0],
                      torch.arange(T - 10, T, device="cuda")])
    assert torch.equal(got[4][0, 0].long(), want)


def test_overlapping_outputs_are_refused():
    B, Hq, Hkv, D, T = 2, 8, 2, 64, 700
    q = torch.randn((B, Hq, D), device="cuda").to(H)
    k, v = make_cache((B, Hkv, T, D), 8, H, 3), make_cache((B, Hkv, T, D), 8, H, 4)
    kp, vp = make_cache((Hkv, 9, D), 8, H, 5), make_cache((Hkv, 9, D), 8, H, 6)
    n = torch.tensor([T, 3], dtype=torch.int32, device="cuda")
    w = torch.zeros((B, Hkv, T), device="cuda")
    with pytest.raises(W4.W4A16Error):
        W4.kv_attention_decode_shared(q, kp, vp, 9, k, v, n, 8, out=q)
    with pytest.raises(W4.W4A16Error):
        W4.kv_attention_decode_weights(q, k, v, n, w, 8, out=q)
    with pytest.raises(W4.W4A16Error):
        W4.kv_attention_decode_weights(q, k, v, n, w, 8, out=w.view(H).view(-1)[:q.numel()].view(q.shape))
    with pytest.raises(W4.W4A16Error):
        W4.kv_attention_decode_weights(q, k, v, n, w, 8, work=v[0].view(torch.float32).view(-1))
    out, sums = W4.kv_attention_decode_weights(q, k, v, n, w, 8)       # in place
    torch.cuda.synchronize()
    assert sums.data_ptr() == w.data_ptr() and abs(float(w.sum()) - B * Hq) < 1e-2
