"""Rotary positions against fp64 with whole-number angles: both pairings, part of the head, odd sizes, strides,
in place, positions of either sign up to the ends of 32 bits, the factor; the gradient against differences."""

import numpy as np
import pytest
import torch

import w4a16_dequant_gemm_amd as W4
from tests.paged_util import check_rotated, f64, rotate

pytestmark = pytest.mark.gpu


def words(freqs):
    return [int(w) % 2 ** 64 for w in freqs.cpu().tolist()]


def make(T, H, D, dtype, seed, pad=0):
    g = torch.Generator().manual_seed(seed)
    return torch.randn((T, (H + pad) * D), generator=g).to(dtype).cuda()[:, :H * D].unflatten(1, (H, D))


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,H,D,R", [(1, 1, 64, 64), (1, 40, 128, 128), (7, 3, 128, 64), (130, 5, 96, 96), (33, 2, 256, 48),
                                     (5, 9, 512, 512), (3, 2, 80, 80), (9, 4, 64, 18), (6, 1, 2, 2), (4, 3, 70, 34),
                                     (4100, 2, 64, 32), (2, 65, 128, 16), (3, 2, 512, 2)])
def test_values(T, H, D, R, interleaved, dtype):
    x = make(T, H, D, dtype, T + H, pad=2)
    g = torch.Generator().manual_seed(5)
    pos = torch.randint(0, 1 << 20, (T,), generator=g, dtype=torch.int64).to(torch.int32)
    freqs, _ = W4.rope_frequencies(R, 10000.0)
    got = W4.rope(x, pos.cuda(), freqs, interleaved=interleaved, mscale=1.25)
    ref, size = rotate(f64(x), pos.tolist(), words(freqs), R, interleaved, 1.25)
    check_rotated(f64(got), ref, size, dtype)
    assert torch.equal(got[..., R:], x[..., R:])


def test_far_positions():
    pos = torch.tensor([0, 1, -1, 2 ** 31 - 1, -2 ** 31, 123456789, -987654321], dtype=torch.int32)
    x = make(7, 3, 128, torch.float16, 1)
    freqs, _ = W4.rope_frequencies(128, 500000.0)
    got = W4.rope(x, pos.cuda(), freqs)
    ref, size = rotate(f64(x), pos.tolist(), words(freqs), 128, False)
    check_rotated(f64(got), ref, size, torch.float16)
    assert torch.equal(got[0], x[0])


def test_small_angles_keep_their_bits():
    """x0 = 0 leaves -x1 sin a alone, for angles down to 2^-60 of a turn."""
    D = 64
    freqs = torch.tensor([1 << max(62 - 2 * i, 4) for i in range(D // 2)], dtype=torch.int64).cuda()
    x = torch.zeros((3, 1, D), dtype=torch.bfloat16, device="cuda")
    x[..., D // 2:] = 3.0
    pos = torch.tensor([1, -1, 3], dtype=torch.int32)
    got = f64(W4.rope(x, pos.cuda(), freqs))
    ref, _ = rotate(f64(x), pos.tolist(), words(freqs), D, False)
    small = np.abs(ref[..., :D // 2]) < 0.5
    err = np.abs(got - ref)[..., :D // 2]
    # (the angle is a whole number of 2^-64 turns: relative 2^-22 and the output's rounding)
    assert (err[small] <= (2.0 ** -8 + 2.0 ** -20) * np.abs(ref[..., :D // 2])[small]).all()


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,R", [(128, 128), (128, 48), (64, 18)])
def test_in_place_and_strided(D, R, interleaved):
    T, H = 19, 5
    wide = torch.randn((T, (H + 3) * D + 8), generator=torch.Generator().manual_seed(2)).to(torch.bfloat16).cuda()
    before = wide.clone()
    x = wide[:, D:(H + 1) * D].unflatten(1, (H, D))
    pos = torch.arange(100, 100 + T, dtype=torch.int32).cuda()
    freqs, _ = W4.rope_frequencies(R)
    want = W4.rope(x.contiguous(), pos, freqs, interleaved=interleaved)
    other = torch.full((T, 2 * H * D), 7.0, dtype=torch.bfloat16, device="cuda")
    W4.rope(x, pos, freqs, interleaved=interleaved, out=other[:, H * D:].unflatten(1, (H, D)))
    assert torch.equal(other[:, H * D:].unflatten(1, (H, D)), want) and (other[:, :H * D] == 7).all()
    back = W4.rope(x, pos, freqs, interleaved=interleaved, out=x)
    assert back is x and torch.equal(x, want)
    wide[:, D:(H + 1) * D] = before[:, D:(H + 1) * D]
    assert torch.equal(wide, before)


def test_two_byte_alignment():
    """Rows that begin at odd elements take the pairs one by one, with the same results."""
    T, H, D = 11, 3, 64
    flat = torch.randn(T * (H * D + 5) + 1, generator=torch.Generator().manual_seed(3)).half().cuda()
    x = flat[1:].view(T, H * D + 5)[:, :H * D].unflatten(1, (H, D))
    pos = torch.arange(T, dtype=torch.int32).cuda()
    freqs, _ = W4.rope_frequencies(D)
    assert torch.equal(W4.rope(x, pos, freqs), W4.rope(x.contiguous(), pos, freqs))


@pytest.mark.parametrize("scaling,kw", [("linear", dict(factor=8.0)), ("base", dict(factor=4.0)),
                                        ("bands", dict(factor=8.0, original=8192)),
                                        ("ramp", dict(factor=16.0, original=4096, low=1.0, high=32.0))])
def test_scaled(scaling, kw):
    freqs, m = W4.rope_frequencies(128, 10000.0, scaling, **kw)
    x = make(9, 2, 128, torch.bfloat16, 8)
    pos = torch.arange(60000, 60009, dtype=torch.int32)
    got = W4.rope(x, pos.cuda(), freqs, mscale=m)
    ref, size = rotate(f64(x), pos.tolist(), words(freqs), 128, False, m)
    check_rotated(f64(got), ref, size, torch.bfloat16)


def test_gradient():
    """The gradient of sum(w * rope(x)) is rope(w, -positions): against differences in fp64 of the formula."""
    T, H, D, R = 3, 2, 64, 32
    freqs, _ = W4.rope_frequencies(R)
    pos = torch.tensor([3, 1000, 77777], dtype=torch.int32)
    w = make(T, H, D, torch.float16, 4)
    got = f64(W4.rope(w, (-pos).cuda(), freqs, mscale=1.5))
    rng = np.random.default_rng(1)
    x, d = rng.standard_normal((T, H, D)), rng.standard_normal((T, H, D))
    h = 2.0 ** -10
    f = lambda y: (f64(w) * rotate(y, pos.tolist(), words(freqs), R, False, 1.5)[0]).sum()
    slope = (f(x + h * d) - f(x - h * d)) / (2 * h)
    tol = (2.0 ** -11 * np.abs(got) + 2.0 ** -19).ravel() @ np.abs(d).ravel() + 1e-9
    assert abs((got * d).sum() - slope) <= tol


def test_no_numbers_stay_in_their_pair():
    x = make(2, 2, 64, torch.float16, 6)
    x[0, 0, 3] = float("nan")
    x[1, 1, 40] = float("inf")
    freqs, _ = W4.rope_frequencies(64)
    y = W4.rope(x, torch.tensor([5, 6], dtype=torch.int32).cuda(), freqs)
    odd = ~torch.isfinite(y)
    want = torch.zeros_like(odd)
    want[0, 0, [3, 35]] = True
    want[1, 1, [8, 40]] = True
    assert torch.equal(odd, want)
