"""GPU parity of the decode attention that adds up attention weights against fp64 (NumPy) on the
rows the caches stand for; the bounds are derived in kv_util."""

from __future__ import annotations

import numpy as np
import pytest
import torch

import w4a16_dequant_gemm_amd as W4
from tests.kv_util import attend, check_out, cmax, f64, make_cache, rows, spoil, weight_error

pytestmark = pytest.mark.gpu
H, BF = torch.float16, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _needs_gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    W4.lib()


def problem(B, Hq, Hkv, D, Tmax, bits, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    q = (torch.randn((B, Hq, D), generator=g) * 1.5).to(dtype).cuda()
    k = make_cache((B, Hkv, Tmax, D), bits, dtype, seed + 1)
    v = make_cache((B, Hkv, Tmax, D), bits, dtype, seed + 2, outliers=False)
    w = (torch.rand((B, Hkv, Tmax), generator=g) * 3).cuda()
    return q, k, v, w


def check(out, sums, q, k, v, before, lens, bits):
    B, Hq, D = q.shape
    Hkv = k[1].shape[1]
    G = Hq // Hkv
    K, V, got, qd, s, w0 = rows(k, bits), rows(v, bits), f64(out), f64(q), f64(sums), f64(before)
    for b, n in enumerate(lens):
        for hk in range(Hkv):
            hs = slice(hk * G, (hk + 1) * G)
            ref, p, mag, qk = attend(qd[b, hs], K[b, hk, :n], V[b, hk, :n])
            e = weight_error(D, qk)
            if n:
                check_out(got[b, hs], ref, mag, q.dtype, e, n, f64(v[1])[b, :, :n].max(),
                          cmax((None, None, v[2][b, :, :n] if v[2] is not None else None), bits))
            else:
                assert (got[b, hs] == 0).all()
            want = w0[b, hk, :n] + p.sum(0)
            tol = e * p.sum(0) + 4 * 2.0 ** -24 * (np.abs(want) + p.sum(0))
            assert (np.abs(s[b, hk, :n] - want) <= tol).all()
            np.testing.assert_array_equal(s[b, hk, n:], w0[b, hk, n:])     # behind the sequence: untouched


# groups of 1 .. 40 heads, lengths around the tiles and splits, odd room (unaligned weight rows)
CASES = [(1, 1, 1, 64, [1], 1, 8, H), (2, 4, 2, 128, [5, 0], 7, 4, BF), (3, 6, 2, 64, [127, 128, 129], 131, 8, BF),
         (2, 8, 1, 128, [255, 257], 261, 4, H), (1, 3, 1, 128, [1025], 1030, 8, H), (2, 40, 1, 64, [300, 33], 301, 8, H),
         (4, 4, 4, 128, [2049, 1, 700, 2050], 2051, 8, H), (1, 8, 2, 64, [5003], 5003, 4, BF),
         (1, 33, 1, 128, [70], 70, 4, H),
         # room for more tokens than one block's work, and the most and the least that is not
         (2, 4, 2, 128, [5, 0], 600, 4, BF), (3, 6, 2, 64, [127, 128, 129], 512, 8, BF), (3, 6, 2, 64, [127, 128, 513], 513, 8, BF),
         (1, 33, 1, 128, [70], 530, 4, H), (2, 8, 1, 128, [255, 257], 600, 4, H), (1, 16, 1, 128, [511], 512, 4, H),
         (2, 17, 1, 64, [300, 512], 512, 8, BF), (64, 4, 4, 64, [16 * i + 15 for i in range(64)], 1024, 8, H),
         (64, 4, 4, 64, [16 * i + 1 for i in range(64)], 1025, 4, H), (65, 4, 4, 64, [15 * i for i in range(65)], 1000, 4, BF),
         (2, 4, 2, 128, [5, 0], 1100, 4, BF), (3, 6, 2, 64, [127, 128, 769], 769, 8, BF), (1, 33, 1, 128, [70], 1100, 4, H),
         (2, 8, 1, 128, [255, 768], 768, 4, H), (2, 8, 1, 128, [255, 257], 1100, 4, H), (43, 3, 3, 128, [23 * i + 1 for i in range(43)], 1024, 8, BF)]


@pytest.mark.parametrize("B,Hq,Hkv,D,lens,Tmax,bits,dtype", CASES)
def test_weights(B, Hq, Hkv, D, lens, Tmax, bits, dtype):
    q, k, v, w = problem(B, Hq, Hkv, D, Tmax, bits, dtype, seed=Tmax)
    for c in (k, v):
        spoil(c, lens, bits)
    for b, n in enumerate(lens):
        w[b, :, n:] = 77.0
    lt = torch.tensor(lens, dtype=torch.int32, device="cuda")
    sums = torch.full_like(w, 77.0)
    out, got = W4.kv_attention_decode_weights(q, k, v, lt, w, bits, sums=sums)
    torch.cuda.synchronize()
    assert got.data_ptr() == sums.data_ptr()
    check(out, sums, q, k, v, w, lens, bits)
    # in place, and from nothing
    before = w.clone()
    out2, got2 = W4.kv_attention_decode_weights(q, k, v, lt, w, bits)
    out3, got3 = W4.kv_attention_decode_weights(q, k, v, lt, None, bits)
    torch.cuda.synchronize()
    assert got2.data_ptr() == w.data_ptr() and torch.equal(out2, out) and torch.equal(out3, out)
    check(out2, w, q, k, v, before, lens, bits)
    check(out3, got3, q, k, v, torch.zeros_like(w), lens, bits)


@pytest.mark.parametrize("room", [300, 700, 1100])
def test_a_query_that_is_no_number_gives_none(room):
    """NaN in one sequence's queries, an infinity in one head of another: NaN there, the rest as before."""
    q, k, v, w = problem(3, 8, 2, 64, room, 8, H, seed=13)
    lens = torch.tensor([300, 0, 77], dtype=torch.int32, device="cuda")
    clean, sums = W4.kv_attention_decode_weights(q, k, v, lens, w, 8, sums=torch.zeros_like(w))
    bad = q.clone()
    bad[:2] = float("nan")
    bad[2, 5, 9] = float("inf")
    out, got = W4.kv_attention_decode_weights(bad, k, v, lens, w, 8, sums=torch.zeros_like(w))
    torch.cuda.synchronize()
    assert torch.isnan(out[0]).all() and torch.isnan(out[2, 5]).all() and (out[1] == 0).all()
    keep = [i for i in range(8) if i != 5]
    assert torch.equal(out[2, keep], clean[2, keep])
    assert torch.isnan(got[0, :, :300]).all() and torch.isnan(got[2, 1, :77]).all()
    assert torch.equal(got[2, 0], sums[2, 0]) and (got[1] == 0).all() and (got[2, :, 77:] == 0).all()


def test_each_head_hands_out_one():
    """The weights of a kv head's G queries add up to G."""
    q, k, v, _ = problem(3, 12, 4, 128, 900, 8, H, seed=9)
    lens = torch.tensor([900, 17, 333], dtype=torch.int32, device="cuda")
    _, sums = W4.kv_attention_decode_weights(q, k, v, lens, None, 8)
    total = sums.double().sum(-1)
    assert (total - 3.0).abs().max() < 3 * 1e-4


def test_agrees_with_the_batched_decode():
    q, k, v, w = problem(4, 8, 2, 128, 700, 4, H, seed=10)
    lens = torch.tensor([700, 1, 350, 129], dtype=torch.int32, device="cuda")
    out, _ = W4.kv_attention_decode_weights(q, k, v, lens, w, 4)
    ref = W4.kv_attention_decode_batch(q, k, v, lens, 4)
    assert (out.float() - ref.float()).abs().max() <= 4 * 2.0 ** -11 * max(1.0, ref.float().abs().max().item())


@pytest.mark.parametrize("B,T", [(2, 333), (2, 700), (2, 1100), (140, 900)])
def test_work_buffer_and_repeat(B, T):
    """None, one for splits and one for the scores alone: nothing behind its end is written."""
    q, k, v, w = problem(B, 8, 2, 64, T, 8, BF, seed=11)
    lens = torch.tensor([T, 100] + [T - 3 * i for i in range(B - 2)], dtype=torch.int32, device="cuda")
    need = W4.kv_attention_weights_workspace(B, 8, 2, T, 64)
    work = torch.full((need + 4,), float("nan"), device="cuda")
    s1, s2 = torch.zeros_like(w), torch.zeros_like(w)
    a, _ = W4.kv_attention_decode_weights(q, k, v, lens, w, 8, sums=s1, work=work)
    b, _ = W4.kv_attention_decode_weights(q, k, v, lens, w, 8, sums=s2)
    torch.cuda.synchronize()
    assert torch.equal(a, b) and torch.equal(s1, s2) and torch.isnan(work[-4:]).all()


def test_refusals():
    q, k, v, w = problem(2, 4, 2, 64, 9, 8, H, seed=12)
    lt = torch.tensor([1, 2], dtype=torch.int32, device="cuda")
    run = W4.kv_attention_decode_weights
    with pytest.raises(TypeError):
        run(q, k, v, lt, w.double(), 8)
    with pytest.raises(ValueError):
        run(q, k, v, lt, w[:, :1].contiguous(), 8)
    with pytest.raises(ValueError):
        run(q, k, v, lt, w, 8, sums=w.cpu())
    with pytest.raises(ValueError):
        run(q, k, v, lt[:1], w, 8)
    with pytest.raises(ValueError):
        run(q, k, tuple(t[:, :, :5].contiguous() if t is not None else None for t in v), lt, w, 8)
    with pytest.raises(ValueError):
        run(q, k, v, lt, w, 8, work=torch.empty(1, device="cuda", dtype=H))
    with pytest.raises(ValueError):                          # (room for 600 tokens needs some)
        run(*problem(2, 4, 2, 64, 600, 8, H, seed=14)[:3], lt, None, 8, work=torch.empty(1, device="cuda"))
    big = torch.zeros(w.numel() + 3, device="cuda")
    with pytest.raises(W4.W4A16Error):                       # sums overlap weights, but are not they
        run(q, k, v, lt, big[:w.numel()].view_as(w), 8, sums=big[3:].view_as(w))
    with pytest.raises(W4.W4A16Error):
        run(q[:, :3].contiguous(), k, v, lt, w, 8)
