"""Attention over the paged cache, row by row: what a row does not see must not reach it, and its error is bounded by
what it does see.

With p the row's weights, smax the largest scale of V among the pages that it sees and u the rounding of the output,

    |out - ref| <= u |ref| + (1 + u) ((2^-11 + e + (n / 16 + 40) 2^-24) sum p |v| + 2^-11 |ref|)
                   + n 2^-33 smax pmax cmax + 2^-25 [fp16]:

e is the fp32 error of a weight (scores, exponentials); weights times scales are rounded to fp16, relative 2^-11, where the
sum is of the rounded ones sum p d (v - out) with |d| <= 2^-11; below fp16's normal range by 2^-25 / 2^11 of 2 smax, twice
where they are rounded again before they are used, with the largest held between 1/2 and 16 times the maximum's.
"""

import numpy as np
import pytest
import torch

import w4a16_dequant_gemm_amd as W4
from tests.kv_util import U, weight_error
from tests.paged_util import CODES, Pool, TOP, f64

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


def check_rows(got, q, pool, b, n, Hq, dtype):
    """Rows ``got [n, Hq, D]`` of sequence b's last n tokens against the bound of what each sees."""
    k, v, live = pool.rows(b)
    D, G, L, u = pool.D, Hq // pool.Hkv, pool.lengths[b], U[dtype]
    assert live.all()
    scales = f64(pool.vs)[pool.table[b, :-(-L // pool.page)].numpy()]                  # [pages, Hkv]
    for h in range(Hq):
        hk = h // G
        s = q[:, h] @ k[:, hk].T / np.sqrt(D)                                           # [n, L]
        sizes = np.abs(q[:, h]) @ np.abs(k[:, hk]).T / np.sqrt(D)
        own = L - n + np.arange(n)
        s[np.arange(L) > own[:, None]] = -np.inf
        p = np.exp(s - s.max(1, keepdims=True))
        p /= p.sum(1, keepdims=True)
        ref, mag = p @ v[:, hk], p @ np.abs(v[:, hk])
        smax = np.maximum.accumulate(scales[:, hk])[own // pool.page]
        e = np.array([weight_error(D, float(sizes[i, :own[i] + 1].max())) for i in range(n)])
        m = (own + 1).astype(np.float64)
        tol = u * np.abs(ref) + (1 + u) * ((2.0 ** -11 + e + (m / 16 + 40) * 2.0 ** -24)[:, None] * mag + 2.0 ** -11 * np.abs(ref))
        tol += (m * 2.0 ** -33 * smax * p.max(1) * TOP[pool.codes])[:, None] + (2.0 ** -25 if dtype == torch.float16 else 0)
        err = np.abs(got[:, h] - ref)
        assert (err <= tol).all(), f"b {b} head {h}: worst {(err / tol).max():.2f} x"


@pytest.mark.parametrize("lean", [0.0, 12.0])
@pytest.mark.parametrize("ratio", [2.0 ** -9, 2.0 ** -20, 2.0 ** -40])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("codes", CODES, ids=ids)
@pytest.mark.parametrize("D,page,long", [(64, 16, False), (128, 16, True), (128, 32, False), (128, 64, True), (64, 64, False)])
def test_pages_of_small_scales(D, page, long, codes, dtype, ratio, lean):
    """Pages whose V is far smaller than that of others, ordinary and small ones in one tile: their weights count in
    full for the sum.  `lean`: scores of their tokens are that much higher (to nearly all of the weight)."""
    lengths, n, Hq = ([1400, 1100], [200, 130], 4) if long else ([220, 90, 40], [60, 90, 33], 4)
    pool = Pool(lengths, 1, D, page, codes, 300 + page, outliers=False)
    for b, length in enumerate(lengths):
        for i in range(-(-length // page)):
            at = pool.table[b, i]
            small = (i * page // 16 + b) % 3 != 0 if page < 64 else (i + b) % 2 == 1
            pool.kc[at, :, :, 0] = 64.0 if small else -64.0
            pool.ks[at] = 2.0 ** -6 if codes == torch.int8 else 2.0 ** -8
            pool.vs[at] *= ratio if small else 1.0
    q = torch.randn((sum(n), Hq, D), generator=torch.Generator().manual_seed(page), dtype=torch.float32)
    q[..., 0] = lean / 2 * D ** 0.5 / (64 * float(pool.ks[pool.table[0, 0], 0]))
    q = q.to(dtype).cuda()
    kp, vp, table, lens = pool.cuda()
    got = f64(W4.kv_attention_paged(q, kp, vp, table, lens, starts(n)))
    at = 0
    for b, count in enumerate(n):
        check_rows(got[at:at + count], f64(q[at:at + count]), pool, b, count, Hq, dtype)
        at += count


@pytest.mark.parametrize("lean", [0.0, 12.0])
@pytest.mark.parametrize("ratio", [2.0 ** -9, 2.0 ** -20])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_steps_on_pages_of_small_scales(dtype, ratio, lean):
    """The same for single tokens, and a few of one sequence."""
    lengths, Hq, D, page = [1300, 200, 70], 4, 128, 16
    pool = Pool(lengths, 2, D, page, torch.int8, 400, outliers=False)
    pool.ks[:] = 2.0 ** -6
    for b, length in enumerate(lengths):
        for i in range(-(-length // page)):
            at = pool.table[b, i]
            small = (i + b) % 3 != 0
            pool.kc[at, :, :, 0] = 64 if small else -64
            pool.vs[at] *= ratio if small else 1.0
    kp, vp, table, lens = pool.cuda()
    for n in ([1, 1, 1], [8, 3, 9]):
        q = torch.randn((sum(n), Hq, D), generator=torch.Generator().manual_seed(5), dtype=torch.float32)
        q[..., 0] = lean / 2 * D ** 0.5
        q = q.to(dtype).cuda()
        got = f64(W4.kv_attention_paged(q, kp, vp, table, lens, None if n[0] == 1 else starts(n)))
        at = 0
        for b, count in enumerate(n):
            check_rows(got[at:at + count], f64(q[at:at + count]), pool, b, count, Hq, dtype)
            at += count


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("codes", CODES, ids=ids)
@pytest.mark.parametrize("D,page", [(64, 16), (128, 64)])
def test_steps_round_once(D, page, codes, dtype):
    """Small scores, so that fp32 counts for little: outputs are the nearest 16-bit numbers but for that, so weights are
    held to more than 16 bits (their rests to 2^-22)."""
    lengths, Hq = [5, 20, 64, 13, 7], 8
    pool = Pool(lengths, 2, D, page, codes, 500, outliers=False)
    kp, vp, table, lens = pool.cuda()
    for n in ([1] * 5, [4, 3, 8, 2, 7]):
        q = (torch.randn((sum(n), Hq, D), generator=torch.Generator().manual_seed(7)) * 0.05).to(dtype).cuda()
        got = f64(W4.kv_attention_paged(q, kp, vp, table, lens, None if n[0] == 1 else starts(n)))
        q, at = f64(q), 0
        for b, count in enumerate(n):
            k, v, _ = pool.rows(b)
            for h in range(Hq):
                for i in range(count):
                    see = lengths[b] - count + i + 1
                    s = k[:see, h // 4] @ q[at + i, h] / np.sqrt(D)
                    p = np.exp(s - s.max())
                    p /= p.sum()
                    ref, mag = p @ v[:see, h // 4], p @ np.abs(v[:see, h // 4])
                    e = weight_error(D, float((np.abs(k[:see, h // 4]) @ np.abs(q[at + i, h])).max() / np.sqrt(D)))
                    out = got[at + i, h]
                    # half a step where the larger of the two lies: U is half of 2^0's
                    half = U[dtype] * np.exp2(np.floor(np.log2(np.maximum(np.maximum(np.abs(ref), np.abs(out)), 2.0 ** -14))))
                    assert (np.abs(out - ref) <= half + (2.0 ** -22 + e + (see / 16 + 40) * 2.0 ** -24) * mag).all()
            at += count


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("codes", CODES, ids=ids)
@pytest.mark.parametrize("n,G", [([1, 1, 1], 2), ([9, 3, 6], 2), ([90, 40, 75], 4)])
def test_lengths_past_the_table(n, G, codes, dtype):
    """Tokens behind the table have no page: the same as with a wider table whose further entries are none.  Rows keep
    their places (the first of a chunk that overruns the table see their own tokens)."""
    D, page = 64, 16
    pool = Pool([320, 300, 64], 2, D, page, codes, 600)
    kp, vp, _, _ = pool.cuda()
    narrow = pool.table[:, :10].contiguous()                # 160 tokens
    narrow[2, 4:] = -1
    wide = torch.full((3, 30), -1, dtype=torch.int32)
    wide[:, :10] = narrow
    lens = torch.tensor([165, 300, 64], dtype=torch.int32).cuda()
    q = torch.randn((sum(n), 2 * G, D), generator=torch.Generator().manual_seed(8)).to(dtype).cuda()
    cu = None if n[0] == 1 else starts(n)
    got = W4.kv_attention_paged(q, kp, vp, narrow.cuda(), lens, cu)
    want = W4.kv_attention_paged(q, kp, vp, wide.cuda(), lens, cu)
    assert torch.equal(got, want) and torch.isfinite(got).all()
    # (the last sequence may have more rows than tokens: its first rows have no place and see nothing)
    places = np.concatenate([np.arange(length - c, length) for length, c in zip(lens.tolist(), n)])
    assert np.array_equal((got != 0).any(-1).all(-1).cpu().numpy(), places >= 0)
    # and what the rows of the first sequence see, by the formula
    seen = Pool([160], 2, D, page, codes, 600)
    seen.kc, seen.ks, seen.vc, seen.vs, seen.table = pool.kc, pool.ks, pool.vc, pool.vs, narrow[:1]
    inside = n[0] - 5                                       # rows whose own tokens have a page
    if inside > 0:
        check_rows(f64(got[:inside]), f64(q[:inside]), seen, 0, inside, 2 * G, dtype)
