"""The paged cache's entry points at their limits on sequences and rows."""

import pytest
import torch

import w4a16_dequant_gemm_amd as W4

pytestmark = pytest.mark.gpu


def test_most_sequences():
    """65535 sequences of one token each, with and without starts: attention gives back the value that was read."""
    B, D, page, Hq = 65535, 64, 16, 2
    g = torch.Generator(device="cuda").manual_seed(1)
    q, k, v = (torch.randn((B, h, D), generator=g, device="cuda").half() for h in (Hq, 1, 1))
    table = torch.arange(B, dtype=torch.int32, device="cuda").flip(0).view(B, 1).contiguous()
    lens = torch.ones(B, dtype=torch.int32, device="cuda")
    freqs, _ = W4.rope_frequencies(D)
    outcome = []
    for cu in (None, torch.arange(B + 1, dtype=torch.int32, device="cuda")):
        kp, vp = W4.kv_pages(B, 1, page, D)
        qo = W4.kv_append_paged(k, v, kp, vp, table, lens, cu, freqs=freqs, q=q)
        ko, vo = W4.kv_read_paged(kp, vp, table, lens, cu, T=B)
        outcome.append((*kp, *vp, qo, ko, vo, W4.kv_attention_paged(qo, kp, vp, table, lens, cu)))
    for a, b in zip(*outcome):
        assert torch.equal(a, b)
    *_, qo, ko, vo, out = outcome[0]
    assert torch.equal(qo, q)                              # (place 0)
    # half a step of the codes, and the rounding to fp16 of values below 8
    for got, want in ((ko, k), (vo, v)):
        tol = want.float().abs().amax(2, keepdim=True) / 127 / 2 + 8 * 2.0 ** -11
        assert ((got.float() - want.float()).abs() <= tol).all()
    # the one token's weight is 1: scale times code, rounded as in reading (and by fp32 sums besides)
    assert ((out.float() - vo.float()).abs() <= vo.float().abs() * 2.0 ** -10 + 2.0 ** -24).all()


def test_most_rows_of_a_rotation():
    T = 2 ** 24 - 1
    x = torch.randn((T, 1, 2), generator=torch.Generator(device="cuda").manual_seed(2), device="cuda").half()
    positions = torch.arange(T, dtype=torch.int32, device="cuda")
    freqs, _ = W4.rope_frequencies(2)                      # one radian a position
    y = W4.rope(x, positions, freqs)
    a, x = positions.double(), x[:, 0].double()
    # (the frequency is held to 2^-53: angles of 2^24 radians to 2^-29)
    ref = torch.stack([x[:, 0] * a.cos() - x[:, 1] * a.sin(), x[:, 1] * a.cos() + x[:, 0] * a.sin()], 1)
    size = x.abs().sum(1, keepdim=True)
    tol = 2.0 ** -11 * ref.abs() + (8 * 2.0 ** -24 + 2.0 ** -28) * size + 2.0 ** -25
    assert ((y[:, 0].double() - ref).abs() <= tol).all()
