"""GPU parity of the decode attention over a shared prefix and own caches against fp64 (NumPy) on the
rows the caches stand for; the bound is derived in kv_util."""

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


def problem(B, Hq, Hkv, D, P, Tmax, bits, dtype, seed, Pmax=None, qscale=1.5, vscale=1.0):
    g = torch.Generator().manual_seed(seed)
    q = (torch.randn((B, Hq, D), generator=g) * qscale).to(dtype).cuda()
    Pmax = max(P, 1) if Pmax is None else Pmax
    kp, vp = (make_cache((Hkv, Pmax, D), bits, dtype, seed + i, scale=s, outliers=i == 1)
              for i, s in ((1, 1.0), (2, vscale)))
    k, v = (make_cache((B, Hkv, Tmax, D), bits, dtype, seed + i, scale=s, outliers=i == 3)
            for i, s in ((3, 1.0), (4, vscale)))
    return q, kp, vp, k, v


def check(out, q, kp, vp, P, k, v, lens, bits):
    B, Hq, D = q.shape
    Hkv = kp[1].shape[0]
    G = Hq // Hkv
    KP, VP, K, V = (rows(c, bits) for c in (kp, vp, k, v))
    got, qd = f64(out), f64(q)
    smax = max([float(vp[1][:, :P].float().max()) if P else 0.0] +
               [float(v[1][b, :, :n].float().max()) for b, n in enumerate(lens) if n])
    c = max(cmax((vp[0], vp[1], vp[2][:, :P] if P and vp[2] is not None else None), bits) if P or bits == 8 else 0.0,
            max([cmax((None, None, v[2][b, :, :n] if v[2] is not None else None), bits)
                 for b, n in enumerate(lens) if n], default=0.0))
    for b, n in enumerate(lens):
        for hk in range(Hkv):
            kk = np.concatenate([KP[hk, :P], K[b, hk, :n]])
            vv = np.concatenate([VP[hk, :P], V[b, hk, :n]])
            hs = slice(hk * G, (hk + 1) * G)
            ref, _, mag, qk = attend(qd[b, hs], kk, vv)
            check_out(got[b, hs], ref, mag, q.dtype, weight_error(D, qk), P + n, smax, c)


# rows per kv head of 1 .. 160 (every row arrangement and ragged tiles), prefixes and own lengths
# around the tiles of 64 and 128 tokens, heads in groups of 1 .. 40, several splits
CASES = [
    (1, 1, 1, 64, 1, [0], 1, 8, H), (3, 4, 4, 128, 63, [1, 0, 5], 8, 8, BF), (2, 6, 2, 64, 64, [64, 65], 70, 4, H),
    (4, 8, 1, 128, 65, [0, 127, 128, 129], 200, 4, BF), (5, 16, 2, 128, 300, [33, 0, 2, 300, 257], 300, 8, H),
    (9, 8, 1, 64, 1000, [7 * i for i in range(9)], 64, 8, BF), (33, 2, 2, 128, 129, [i % 5 for i in range(33)], 4, 4, H),
    (20, 8, 1, 128, 700, [i for i in range(20)], 32, 8, H), (2, 40, 1, 64, 90, [100, 3], 100, 8, H),
    (3, 40, 1, 128, 20, [0, 260, 40], 300, 4, BF), (65, 1, 1, 64, 2100, [1] * 65, 1, 4, H),
    (2, 2, 1, 128, 5000, [4000, 1], 4100, 8, H), (1, 3, 3, 128, 513, [600], 640, 4, H),
    (5, 8, 2, 64, 127, [3, 0, 65, 64, 1], 70, 4, BF), (12, 4, 1, 64, 191, [i for i in range(12)], 16, 8, H),
    (64, 1, 1, 64, 320, [0] * 64, 1, 4, H), (16, 1, 1, 128, 64, [5] * 16, 5, 8, BF), (17, 1, 1, 128, 192, [5] * 17, 5, 4, BF),
    # many rows and a prefix that is short beside the own caches (streamed), the next longer one (not)
    (40, 8, 2, 128, 75, [7 * i for i in range(40)], 300, 8, BF), (40, 8, 2, 128, 76, [7 * i for i in range(40)], 300, 8, BF),
    (33, 3, 1, 64, 33, [4 * i for i in range(33)], 132, 4, H), (33, 3, 1, 64, 34, [4 * i for i in range(33)], 132, 4, H),
    # the same sizes with more room for own tokens: one block of eight waves, or of four, a sequence ...
    (40, 8, 2, 128, 150, [7 * i for i in range(40)], 600, 8, BF), (40, 8, 2, 128, 151, [7 * i for i in range(40)], 873, 8, BF),
    (130, 8, 2, 64, 400, [i for i in range(130)], 200, 4, BF), (1, 1, 1, 64, 1, [0], 512, 8, H), (3, 4, 4, 128, 63, [1, 0, 5], 450, 8, BF), (2, 6, 2, 64, 64, [64, 65], 449, 4, H),
    (33, 2, 2, 128, 129, [i % 5 for i in range(33)], 400, 4, H), (12, 4, 1, 64, 191, [i for i in range(12)], 400, 8, H),
    (64, 1, 1, 64, 320, [0] * 64, 300, 4, H), (17, 1, 1, 128, 192, [5] * 17, 400, 4, BF), (3, 40, 1, 128, 130, [0, 260, 40], 500, 4, BF),
    (5, 8, 2, 64, 127, [3, 0, 65, 64, 1], 500, 4, BF), (2, 40, 1, 64, 256, [100, 256], 256, 8, H), (2, 40, 1, 64, 256, [100, 257], 257, 8, H),
    # ... or splits
    (40, 8, 2, 128, 250, [7 * i for i in range(40)], 1000, 8, BF), (40, 8, 2, 128, 251, [7 * i for i in range(40)], 1000, 8, BF),
    (1, 1, 1, 64, 1, [0], 1100, 8, H), (3, 4, 4, 128, 63, [1, 0, 5], 1100, 8, BF), (33, 2, 2, 128, 300, [i % 5 for i in range(33)], 1000, 4, H),
    (12, 4, 1, 64, 291, [i for i in range(12)], 900, 8, H), (64, 1, 1, 64, 320, [0] * 64, 900, 4, H), (17, 1, 1, 128, 292, [5] * 17, 900, 4, BF),
    (3, 40, 1, 128, 330, [0, 260, 40], 900, 4, BF), (5, 8, 2, 64, 127, [3, 0, 65, 64, 1], 1000, 4, BF), (2, 6, 2, 64, 64, [64, 65], 1000, 4, H),
    # many sequences behind a prefix that is too much to read for each
    (1100, 4, 4, 64, 240, [i % 12 for i in range(1100)], 12, 8, H)]


@pytest.mark.parametrize("B,Hq,Hkv,D,P,lens,Tmax,bits,dtype", CASES)
def test_shared_prefix(B, Hq, Hkv, D, P, lens, Tmax, bits, dtype):
    q, kp, vp, k, v = problem(B, Hq, Hkv, D, P, Tmax, bits, dtype, seed=B + P, Pmax=P + 3)
    for c in (kp, vp):
        spoil(c, P, bits)
    for c in (k, v):
        spoil(c, lens, bits)
    lt = torch.tensor(lens, dtype=torch.int32, device="cuda")
    out = W4.kv_attention_decode_shared(q, kp, vp, P, k, v, lt, bits)
    torch.cuda.synchronize()
    check(out, q, kp, vp, P, k, v, lens, bits)


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("room", [150, 700, 1100])
def test_no_prefix_and_no_tokens(bits, room):
    """P = 0 leaves the own tokens; a sequence with neither gets zeros."""
    lens = [0, 130, 1]
    q, kp, vp, k, v = problem(3, 4, 2, 128, 0, room, bits, H, seed=50)
    lt = torch.tensor(lens, dtype=torch.int32, device="cuda")
    out = torch.full_like(q, float("nan"))
    W4.kv_attention_decode_shared(q, kp, vp, 0, k, v, lt, bits, out=out)
    torch.cuda.synchronize()
    assert (out[0] == 0).all()
    check(out, q, kp, vp, 0, k, v, lens, bits)


def test_lengths_outside_are_clamped():
    q, kp, vp, k, v = problem(3, 2, 1, 64, 40, 20, 8, H, seed=51)
    lt = torch.tensor([-7, 1 << 30, 20], dtype=torch.int32, device="cuda")
    out = W4.kv_attention_decode_shared(q, kp, vp, 40, k, v, lt, 8)
    torch.cuda.synchronize()
    check(out, q, kp, vp, 40, k, v, [0, 20, 20], 8)


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("qscale", [1e-30, 1e4])
@pytest.mark.parametrize("room", [30, 500, 1000])
def test_bf16_queries_far_from_one(bits, qscale, room):
    """bf16 queries outside fp16's range: scaled by a power of two inside the kernel."""
    q, kp, vp, k, v = problem(4, 8, 2, 128, 150, room, bits, BF, seed=52, qscale=qscale)
    lens = [0, 30, 7, 1]
    out = W4.kv_attention_decode_shared(q, kp, vp, 150, k, v, torch.tensor(lens, dtype=torch.int32, device="cuda"), bits)
    torch.cuda.synchronize()
    if qscale < 1:
        check(out, q, kp, vp, 150, k, v, lens, bits)
    else:      # one token takes all the weight, up to scores closer than their fp32 error: 1e4 * 30 * 2^-16
        KP, VP, K, V = (rows(c, bits) for c in (kp, vp, k, v))
        for b, n in enumerate(lens):
            for h in range(8):
                kk = np.concatenate([KP[h // 4], K[b, h // 4, :n]])
                vv = np.concatenate([VP[h // 4], V[b, h // 4, :n]])
                s = kk @ f64(q)[b, h]
                top = np.sort(s)[-2:]
                if top[1] - top[0] > 1e4:
                    np.testing.assert_allclose(f64(out)[b, h], vv[s.argmax()], rtol=2.0 ** -7, atol=1e-6)


@pytest.mark.parametrize("B,Hq,Hkv", [(4, 8, 2), (12, 8, 2), (40, 8, 2)])
@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("P,room", [(150, 9), (150, 600), (300, 900)])
def test_bf16_queries_of_very_different_size(bits, B, Hq, Hkv, P, room):
    """Rows that share a block, from 1e-30 to 1e6 in size: each keeps its bits (16, 48 and 160 rows
    per kv head, one for each arrangement of the waves; a sequence as one block's work)."""
    q, kp, vp, k, v = problem(B, Hq, Hkv, 128, P, room, bits, BF, seed=60)
    size = torch.tensor([1e-30, 1.0, 1e-9, 1e6, 0.0, 1e-3, 3e4])[torch.arange(B * Hq) % 7].view(B, Hq, 1)
    q = (q.cpu().float() * size).to(BF).cuda()
    lens = [i % 10 for i in range(B)]
    out = W4.kv_attention_decode_shared(q, kp, vp, P, k, v, torch.tensor(lens, dtype=torch.int32, device="cuda"), bits)
    torch.cuda.synchronize()
    keep = (size.flatten() <= 1.0).view(B, Hq)                 # the large rows' scores differ by more than fp32 holds
    assert torch.isfinite(out).all()
    small = torch.where(keep[..., None].cuda(), q, torch.zeros_like(q))
    same = W4.kv_attention_decode_shared(small, kp, vp, P, k, v, torch.tensor(lens, dtype=torch.int32, device="cuda"), bits)
    torch.cuda.synchronize()
    check(same, small, kp, vp, P, k, v, lens, bits)
    # beside large rows a row's weights may differ by their fp16 roundings alone
    a, b = f64(out)[keep.numpy()], f64(same)[keep.numpy()]
    assert np.abs(a - b).max() <= 2.0 ** -7 * np.abs(b).max()


@pytest.mark.parametrize("B,Hq,Hkv", [(4, 8, 2), (12, 8, 2), (40, 8, 2)])
@pytest.mark.parametrize("dtype", [H, BF])
@pytest.mark.parametrize("P,room", [(140, 9), (140, 600), (290, 900)])
def test_rows_without_numbers_leave_the_others_alone(B, Hq, Hkv, dtype, P, room):
    """Unused places of a padded batch: NaN and infinities in some queries, the other rows as before."""
    q, kp, vp, k, v = problem(B, Hq, Hkv, 64, P, room, 8, dtype, seed=61)
    lt = torch.tensor([i % 10 for i in range(B)], dtype=torch.int32, device="cuda")
    clean = W4.kv_attention_decode_shared(q, kp, vp, P, k, v, lt, 8)
    bad = q.clone()
    bad[1] = float("nan")
    bad[2, 3, 5] = float("inf")
    bad[B - 1, 1] = -float("inf")
    out = W4.kv_attention_decode_shared(bad, kp, vp, P, k, v, lt, 8)
    torch.cuda.synchronize()
    ok = torch.ones((B, Hq), dtype=torch.bool)
    ok[1] = False
    ok[2, 3] = ok[B - 1, 1] = False
    a, b = f64(out)[ok.numpy()], f64(clean)[ok.numpy()]
    assert np.isfinite(a).all() and np.isnan(f64(out)[~ok.numpy()]).all()
    check(torch.where(ok[..., None].cuda(), out, clean), q, kp, vp, P, k, v, [i % 10 for i in range(B)], 8)
    if P > 256:         # rows of a wave move their references together: other roundings of the weights
        return
    # the common factor of the bf16 rows may be another one: the same values, up to a rounding
    assert np.abs(a - b).max() <= (0.0 if dtype == H else 2.0 ** -7 * np.abs(b).max())


@pytest.mark.parametrize("room", [10, 500, 1000])
def test_zero_value_rows_beside_small_ones(room):
    """A row of zeros is stored with scale 1 beside values of 1e-3: the small rows keep their bits."""
    q, kp, vp, k, v = problem(2, 4, 2, 64, 200, room, 8, BF, seed=53, vscale=1e-3)
    c, s, _ = vp
    c[:, 17] = 0
    s[:, 17] = 1.0
    out = W4.kv_attention_decode_shared(q, kp, vp, 200, k, v, torch.tensor([10, 0], dtype=torch.int32, device="cuda"), 8)
    torch.cuda.synchronize()
    check(out, q, kp, vp, 200, k, v, [10, 0], 8)


def test_prefix_equals_the_same_tokens_in_own_caches():
    """The shared form agrees with the batched decode over caches that each hold prefix and suffix."""
    B, Hq, Hkv, D, P, T, bits = 3, 8, 2, 128, 500, 77, 8
    q, kp, vp, k, v = problem(B, Hq, Hkv, D, P, T, bits, H, seed=54)
    full = [tuple(torch.cat([p[None].expand(B, *p.shape), t], 2).contiguous() if t is not None else None
                  for p, t in zip(cp, c)) for cp, c in ((kp, k), (vp, v))]
    lt = torch.tensor([77, 5, 40], dtype=torch.int32, device="cuda")
    a = W4.kv_attention_decode_shared(q, kp, vp, P, k, v, lt, bits)
    b = W4.kv_attention_decode_batch(q, full[0], full[1], lt + P, bits)
    torch.cuda.synchronize()
    # two fp16 roundings of outputs and the rounded weights between them
    assert (a.float() - b.float()).abs().max() <= 4 * 2.0 ** -11 * max(1.0, b.float().abs().max().item())


def test_repeat_and_other_stream_are_identical():
    q, kp, vp, k, v = problem(6, 8, 2, 128, 900, 50, 4, H, seed=55)
    lt = torch.tensor([50, 0, 3, 9, 50, 1], dtype=torch.int32, device="cuda")
    a = W4.kv_attention_decode_shared(q, kp, vp, 900, k, v, lt, 4)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    work = torch.full((W4.kv_attention_shared_workspace(6, 8, 2, 900, 50, 128) + 4,), float("nan"), device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        b = W4.kv_attention_decode_shared(q, kp, vp, 900, k, v, lt, 4, work=work)
    st.synchronize()
    assert torch.equal(a.view(torch.int16), b.view(torch.int16))
    assert torch.isnan(work[-4:]).all()


def test_refusals():
    q, kp, vp, k, v = problem(2, 4, 2, 64, 10, 8, 8, H, seed=56)
    lt = torch.tensor([1, 2], dtype=torch.int32, device="cuda")
    run = W4.kv_attention_decode_shared
    with pytest.raises(ValueError):
        run(q, kp, vp, 11, k, v, lt, 8)                     # P > Pmax
    with pytest.raises(ValueError):
        run(q, kp, vp, -1, k, v, lt, 8)
    with pytest.raises(ValueError):
        run(q, kp, vp, 10, k, v, lt, 5)
    with pytest.raises(TypeError):
        run(q, kp, vp, 10, k, v, lt, 4)                     # 8-bit codes as 4-bit ones
    with pytest.raises(TypeError):
        run(q, kp, vp, 10, k, v, lt.long(), 8)
    with pytest.raises(TypeError):
        run(q.float(), kp, vp, 10, k, v, lt, 8)
    with pytest.raises(ValueError):
        run(q, kp, vp, 10, k, v, lt[:1], 8)
    with pytest.raises(ValueError):
        run(q[:1], kp, vp, 10, k, v, lt[:1], 8)             # two cached sequences, one query
    with pytest.raises(ValueError):
        run(q, kp, tuple(t[:1] if t is not None else None for t in vp), 10, k, v, lt, 8)
    with pytest.raises(ValueError):
        run(q, kp, vp, 10, k, v, lt.cpu(), 8)
    with pytest.raises(ValueError):
        run(q, kp, vp, 10, k, v, lt, 8, work=torch.empty(3, device="cuda", dtype=H))
    with pytest.raises(ValueError):                         # (room for 1100 own tokens needs some)
        run(q, kp, vp, 10, *problem(2, 4, 2, 64, 10, 1100, 8, H, seed=57)[3:], lt, 8, work=torch.empty(3, device="cuda"))
    with pytest.raises(ValueError):
        run(q, kp, vp, 10, k, v, lt, 8, out=torch.empty((2, 4, 32), dtype=H, device="cuda"))
    with pytest.raises(W4.W4A16Error):
        run(q[:, :3].contiguous(), kp, vp, 10, k, v, lt, 8)
