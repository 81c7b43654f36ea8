"""bf16 queries beside much larger ones in the same tile: entries down to 2^-21 of their row's largest reach the
products with all their bits (the bound of kv_util has no room for a lost one: a score here is 58 times the
small entry's relative error off)."""

from __future__ import annotations

import numpy as np
import pytest
import torch

import w4a16_dequant_gemm_amd as W4
from tests.kv_util import attend, check_out, f64, rows, weight_error

pytestmark = pytest.mark.gpu
H, BF = torch.float16, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _needs_gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    W4.lib()


def cache(shape, D, bits, keys, gen):
    """Keys that differ in element 2 alone; values of one to two."""
    n = int(np.prod(shape))
    if bits == 8:
        codes = torch.zeros((n, D), dtype=torch.int8)
        if keys:
            codes[:, 2] = 100 + torch.arange(n, dtype=torch.int8) % 28
        else:
            codes[:] = torch.randint(60, 127, (n, D), generator=gen, dtype=torch.int8)
        zeros = None
    else:
        words = torch.zeros((n, D // 8), dtype=torch.int64)
        if keys:
            words[:, 0] = (torch.arange(n) % 16) << 8
        else:
            words = torch.randint(0, 1 << 28, (n, D // 8), generator=gen)
        codes, zeros = words.to(torch.int32), torch.zeros(shape, dtype=H, device="cuda")
    scales = torch.full(shape, 60000.0 if keys else 1.0 / 64, dtype=H, device="cuda")
    return codes.view(*shape, -1).cuda(), scales, zeros


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("ratio", [9, 10, 11, 14, 17, 18, 30])
# a sequence whole, in splits, behind a prefix with two and with four waves of rows
@pytest.mark.parametrize("B,P,room", [(3, 0, 40), (3, 0, 1100), (6, 1500, 40), (40, 1500, 40)])
def test_small_entries_keep_their_bits(B, P, room, ratio, bits):
    Hq, D = 8, 64
    gen = torch.Generator().manual_seed(ratio)
    q = torch.zeros((B, Hq, D))
    q[:, 0::2, 1] = 2.0 ** ratio                # (element 1 of every key is 0)
    q[:, 1::2, 0] = 1.0
    for i, h in enumerate(range(1, Hq, 2)):     # 2^-14 (1 + 2^-7), 2^-15 (2 - 2^-7), ...
        q[:, h, 2] = 2.0 ** -14 * [1 + 2.0 ** -7, 1 - 2.0 ** -8, 1 + 3 * 2.0 ** -7, 1 + 5 * 2.0 ** -7][i]
    q = q.to(BF).cuda()
    kp, vp = cache((1, max(P, 1)), D, bits, True, gen), cache((1, max(P, 1)), D, bits, False, gen)
    k, v = cache((B, 1, room), D, bits, True, gen), cache((B, 1, room), D, bits, False, gen)
    lens = [room - 3 * (b % 10) for b in range(B)]
    out = W4.kv_attention_decode_shared(q, kp, vp, P, k, v, torch.tensor(lens, dtype=torch.int32, device="cuda"), bits)
    torch.cuda.synchronize()
    KP, VP, K, V = (rows(c, bits) for c in (kp, vp, k, v))
    got, qd = f64(out), f64(q)
    for b in range(0, B, max(1, B // 5)):
        kk, vv = np.concatenate([KP[0, :P], K[b, 0, :lens[b]]]), np.concatenate([VP[0, :P], V[b, 0, :lens[b]]])
        ref, _, mag, qk = attend(qd[b], kk, vv)
        check_out(got[b], ref, mag, BF, weight_error(D, qk), P + lens[b], 1.0 / 64, 127.0 if bits == 8 else 15.0)
