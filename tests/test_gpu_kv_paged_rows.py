"""Attention over the paged cache, row by row: what a row does not see must not reach it, and its error is bounded by
what it does see."""

import numpy as np
import pytest
import torch

import w4a16_dequant_gemm_amd as W4
from tests.paged_util import CODES, Pool

pytestmark = pytest.mark.gpu
NAMES = {torch.int8: "int8", torch.float8_e4m3fn: "e4m3"}
ids = lambda v: NAMES.get(v, None)


def starts(counts):
    return torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32).cuda()


def later_pages(dtype, codes, lengths, n, G, D, page, ratio):
    """V's scales of every sequence's pages from the middle of its last n tokens on, times `ratio`: the rows before the
    first of them come out in the same bits."""
    pool = Pool(lengths, 2, D, page, codes, 200 + page)
    q = torch.randn((sum(n), 2 * G, D), generator=torch.Generator().manual_seed(page), dtype=torch.float32).to(dtype).cuda()
    kp, vp, table, lens = pool.cuda()
    want = W4.kv_attention_paged(q, kp, vp, table, lens, starts(n))
    before = []
    for b, (length, count) in enumerate(zip(lengths, n)):
        first = -(-(length - count // 2) // page)                # the first page that is changed
        vp[1][table[b, first:-(-length // page)].long()] *= ratio
        kept = max(min(first * page - (length - count), count), 0)
        before += [True] * kept + [False] * (count - kept)
    before = torch.tensor(before, device="cuda")
    got = W4.kv_attention_paged(q, kp, vp, table, lens, starts(n))
    assert before.any() and not before.all() and torch.isfinite(want).all() and (want != 0).any(-1).all()
    assert torch.equal(got[before], want[before])


@pytest.mark.parametrize("ratio", [2.0 ** 12, 2.0 ** 40, 2.0 ** 100])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("codes", CODES, ids=ids)
@pytest.mark.parametrize("D,page", [(64, 16), (128, 16), (128, 32), (64, 64)])
def test_later_pages_of_few_rows(D, page, codes, dtype, ratio):
    """(scales up to 2^100 times as large: weights in proportion to them would round to 0)"""
    later_pages(dtype, codes, [70, 200, 69 + page, 1300], [12, 8, 14, 10], 2, D, page, ratio)


@pytest.mark.parametrize("ratio", [2.0 ** -20, 2.0 ** 12, 2.0 ** 30, 2.0 ** 100])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("codes", CODES, ids=ids)
@pytest.mark.parametrize("D,page", [(64, 16), (128, 16), (128, 32), (128, 64), (64, 128)])
def test_later_pages_of_chunks(D, page, codes, dtype, ratio):
    """Blocks of 128 rows, and of 256 for long sequences."""
    later_pages(dtype, codes, [150, 60, 69 + page, 350], [100, 40, 60, 200], 4, D, page, ratio)
    later_pages(dtype, codes, [1700, 1200], [333, 250], 4, D, page, ratio)
