"""Prompt attention where whole tiles of visible keys score -inf (infinities in the keys): weight 0, so the
rows are those of the other keys; rows that see nothing else are no numbers, as 0 / 0 is."""

from __future__ import annotations

import pytest
import torch

import w4a16_dequant_gemm_amd as W4
from tests.test_gpu_attention_prompt import check, packed

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _needs_gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    W4.lib()


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("D", [64, 128])
# a tile, part of the second, several; and all keys of the first of two groups of waves
@pytest.mark.parametrize("n,dead", [(200, 64), (200, 65), (400, 256), (1200, 64), (1200, 700), (100, 31)])
def test_first_keys_score_minus_infinity(n, dead, D, dtype):
    q, k, v, cu = packed([n], 2, 1, D, dtype, seed=n + dead, fused=False)
    q[..., 5] = q[..., 5].abs() + 1
    k[:dead, :, 5] = -float("inf")
    out = W4.attention_prompt(q, k, v, cu)
    torch.cuda.synchronize()
    assert torch.isnan(out[:dead]).all()
    # (q . k of the live keys: entries of q up to 5 at dimension 5, within the bound's sum |q k|)
    check(out[dead:], q[dead:], k[dead:], v[dead:], [n - dead])


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("n,dead", [(200, 64), (1200, 700)])
def test_rows_beside_others_with_finite_scores(n, dead, dtype):
    """Every second row does not meet the first keys' large entries (its query is 0 there): both kinds share
    tiles and the rescaling that the one of them causes."""
    D = 64
    q, k, v, cu = packed([n], 2, 1, D, dtype, seed=n, fused=False)
    q[..., 5] = 0
    k[:, :, 5] = 0
    k[:dead, :, 5] = -torch.finfo(dtype).max
    plain = q.clone()                           # rows that see every key
    q[::2, :, 5] = 4.0                          # rows of weight 0 there: scores of -inf (bf16) or -32000 (fp16)
    out = W4.attention_prompt(q, k, v, cu)
    both = W4.attention_prompt(plain, k, v, cu)
    live = W4.attention_prompt(plain[dead:], k[dead:], v[dead:], cu - torch.tensor([0, dead], dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    both[1::2] = out[1::2]
    check(both, plain, k, v, [n])
    live[::2] = out[dead::2]                    # (dead is even)
    check(live, plain[dead:], k[dead:], v[dead:], [n - dead])
