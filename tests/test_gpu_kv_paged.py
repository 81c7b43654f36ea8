"""The paged 8-bit cache: appending (bit for bit against the same fp32 steps on the host), rotation on the way,
reading back, attention of decode steps and chunks against fp64; pages that are none, empty sequences,
stale codes that are no numbers, strides, and the loop that a server runs."""

import numpy as np
import pytest
import torch

import w4a16_dequant_gemm_amd as W4
from tests.paged_util import CODES, HostCache, Pool, TOP, check_attention, check_rotated, f64, rotate

pytestmark = pytest.mark.gpu
NAMES = {torch.int8: "int8", torch.float8_e4m3fn: "e4m3"}
ids = lambda v: NAMES.get(v, None)


def starts(counts):
    return torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32).cuda()


def fused(T, heads, D, dtype, seed, scale=1.0):
    """Column blocks of one wide tensor, as a fused projection leaves them."""
    x = (torch.randn((T, sum(heads) * D), generator=torch.Generator().manual_seed(seed)) * scale).to(dtype).cuda()
    return [t.unflatten(1, (h, D)) for t, h in zip(x.split([h * D for h in heads], 1), heads)]


# --------------------------------------------------------------------------- append and read

@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("codes", CODES, ids=ids)
@pytest.mark.parametrize("page,D", [(16, 64), (32, 128), (64, 128), (128, 64)])
def test_append_steps_and_chunks(page, D, codes, dtype):
    """Several calls in a row on ragged sequences: codes and scales of K (not rotated) and V bit for bit."""
    Hkv, B, room = 3, 4, 5 * page
    P = room // page
    kp, vp = W4.kv_pages(B * P + 2, Hkv, page, D, codes)
    kp[0].view(torch.uint8).fill_(0x7F)                    # (a pool of torch.empty may hold anything)
    vp[0].view(torch.uint8).fill_(0x7F)
    kp[1].fill_(float("nan"))
    vp[1].fill_(float("nan"))
    table = torch.randperm(B * P + 2, generator=torch.Generator().manual_seed(1))[:B * P].view(B, P).to(torch.int32)
    host = [[[HostCache(page, codes) for _ in range(Hkv)] for _ in range(B)] for _ in range(2)]
    length = [0] * B
    plan = [[5, 0, page + 3, 1], "step", "step", [1, 2 * page, 0, 2], "step", [page, 1, page - 1, 2 * page + 1], "step"]
    for i, counts in enumerate(plan):
        n = [1] * B if counts == "step" else counts
        k, v = fused(sum(n), [Hkv, Hkv], D, dtype, 10 * i + page, 1.0 + i)
        length = [a + b for a, b in zip(length, n)]
        W4.kv_append_paged(k, v, kp, vp, table.cuda(), torch.tensor(length, dtype=torch.int32).cuda(),
                           None if counts == "step" else starts(n))
        at = 0
        for b in range(B):
            for h in range(Hkv):
                for x, c in ((k, host[0]), (v, host[1])):
                    c[b][h].write(x[at:at + n[b], h].float().cpu().numpy(), length[b] - n[b])
            at += n[b]
    for (c, s), cache, axis in ((kp, host[0], 0), (vp, host[1], 1)):
        c, s = f64(c.cpu().float()), s.cpu().numpy()
        for b in range(B):
            for h in range(Hkv):
                for i, (want, scale) in enumerate(cache[b][h].pages):
                    if len(want):
                        got = c[table[b, i], h] if axis == 0 else c[table[b, i], h].T
                        assert s[table[b, i], h] == scale
                        assert np.array_equal(got[:len(want)], want), (b, h, i)
    # pages of no sequence are as they were
    spare = sorted(set(range(B * P + 2)) - set(table.flatten().tolist()))
    assert (kp[0].view(torch.uint8)[spare] == 0x7F).all() and torch.isnan(vp[1][spare]).all()
    # and what reading gives is those codes times scales, rounded once
    lens = torch.tensor(length, dtype=torch.int32).cuda()
    for back in (length, [min(n, page + 5) for n in length], [1] * B):
        ko, vo = W4.kv_read_paged(kp, vp, table.cuda(), lens, starts(back), T=sum(back), dtype=dtype)
        at = 0
        for b in range(B):
            for out, cache in ((ko, host[0]), (vo, host[1])):
                for h in range(Hkv):
                    rows = np.concatenate([c.astype(np.float32) * s for c, s in cache[b][h].pages if len(c)])
                    want = torch.from_numpy(rows[length[b] - back[b]:length[b]]).to(dtype)
                    assert torch.equal(out[at:at + back[b], h].cpu(), want)
            at += back[b]


def grid_check(got, ref, size, scale, codes):
    """Values off a rotated row by half a step of the code at most (fp32 errors besides)."""
    half = 0.5 * scale if codes == torch.int8 else np.maximum(np.abs(ref) * 2.0 ** -4, scale * 2.0 ** -10)
    assert (np.abs(got - ref) <= half * (1 + 2.0 ** -20) + 16 * 2.0 ** -24 * (size + np.abs(ref)) + 2.0 ** -22 * scale * TOP[codes]).all()


@pytest.mark.parametrize("codes", CODES, ids=ids)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,R,page", [(64, 64, 16), (128, 128, 64), (128, 64, 32), (128, 34, 128), (64, 2, 16), (128, 126, 32)])
@pytest.mark.parametrize("explicit", [False, True])
def test_append_rotates(D, R, page, interleaved, codes, explicit):
    dtype, Hq, Hkv, n = torch.bfloat16, 6, 2, [page + 7, 1, 0, 3]
    before = [page // 2 + 1, 40, 7, 0]
    B, T = 4, sum(n)
    length = [a + b for a, b in zip(before, n)]
    P = max(-(-t // page) for t in length)
    kp, vp = W4.kv_pages(B * P, Hkv, page, D, codes)
    table = torch.arange(B * P, dtype=torch.int32).view(B, P).cuda()
    q, k, v = fused(T, [Hq, Hkv, Hkv], D, dtype, D + R)
    freqs, _ = W4.rope_frequencies(R, 10000.0)
    words = [int(w) % 2 ** 64 for w in freqs.cpu().tolist()]
    seq = np.repeat(np.arange(B), n)
    place = np.concatenate([np.arange(b, a) for a, b in zip(length, before)]).astype(np.int64)
    pos = np.arange(T) * 1000 - 7000 if explicit else place
    lens = torch.tensor(length, dtype=torch.int32).cuda()
    qo = W4.kv_append_paged(k, v, kp, vp, table, lens, starts(n), freqs=freqs, interleaved=interleaved, mscale=0.75, q=q,
                            positions=torch.from_numpy(pos).to(torch.int32).cuda() if explicit else None)
    ref, size = rotate(f64(q), pos, words, R, interleaved, 0.75)
    check_rotated(f64(qo), ref, size, dtype)
    ref, size = rotate(f64(k), pos, words, R, interleaved, 0.75)
    c, s = f64(kp[0].cpu().float()), f64(kp[1])
    for b in range(B):
        for i in range(P):
            mine = (seq == b) & (place // page == i)
            if not mine.any():
                continue
            page_id = int(table[b, i])
            got = c[page_id][:, place[mine] % page].swapaxes(0, 1)
            # (earlier slots of these pages hold nothing: the scale is the new rows' own, but for the old one's 0)
            want = np.abs(ref[mine]).max((0, 2)) / TOP[codes]
            assert np.allclose(s[page_id], want, rtol=2.0 ** -19, atol=0)
            sc = s[page_id][None, :, None]
            grid_check(got * sc, ref[mine], size[mine], sc, codes)


def test_append_without_positions_is_a_step():
    """cu_seqlens of one token each, and None, are the same call."""
    D, Hq, Hkv, page, B = 128, 8, 2, 16, 5
    q, k, v = fused(B, [Hq, Hkv, Hkv], D, torch.float16, 3)
    table = torch.arange(2 * B, dtype=torch.int32).view(B, 2).cuda()
    lens = torch.tensor([1, 16, 17, 32, 0], dtype=torch.int32).cuda()
    freqs, m = W4.rope_frequencies(D)
    got = []
    for cu in (None, starts([1] * B)):
        kp, vp = W4.kv_pages(2 * B, Hkv, page, D)
        qo = W4.kv_append_paged(k, v, kp, vp, table, lens, cu, freqs=freqs, q=q)
        got.append((*kp, *vp, qo))
    for a, b in zip(*got):
        assert torch.equal(a, b)
    assert (got[0][1][-2:] == 0).all()              # (the sequence of length 0 takes none)


def test_append_outside_the_table():
    """Tokens behind the table, at entries that are no pages and without a place are not written; rows of no
    sequence leave q_out as it was."""
    D, Hkv, page = 64, 2, 16
    n = [20, 20, 20, 6]
    T = sum(n) + 7
    q, k, v = fused(T, [4, Hkv, Hkv], D, torch.float16, 4)
    kp, vp = W4.kv_pages(8, Hkv, page, D)
    kp[0].fill_(-128), vp[0].fill_(-128), kp[1].fill_(5.0), vp[1].fill_(5.0)
    table = torch.tensor([[0, -1], [1, 8], [2 ** 31 - 1, 3], [4, 5]], dtype=torch.int32)
    lens = [36, 20, 20, 4]                          # the first overruns its table, the last has two rows too many
    cu = torch.tensor([3, 23, 43, 63, 69], dtype=torch.int32).cuda()
    qo = torch.full((T, 4, D), 9.0, dtype=torch.float16, device="cuda")
    freqs, _ = W4.rope_frequencies(D)
    W4.kv_append_paged(k, v, kp, vp, table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), cu, freqs=freqs, q=q, q_out=qo)
    written = torch.zeros((8, page), dtype=torch.bool)
    written[1, :] = True                            # tokens 0 .. 15 of the second sequence; its entry 8 is none
    written[3, :4] = True
    written[4, :4] = True
    assert torch.equal((kp[0].cpu() != -128).any(-1).all(1), written)
    assert torch.equal((vp[0].cpu() != -128).any(2).all(1), written)
    assert torch.equal((kp[1].cpu() != 5.0).all(1), written.any(1)) and torch.equal((vp[1].cpu() != 5.0).all(1), written.any(1))
    assert (qo[:3] == 9).all() and (qo[69:] == 9).all() and (qo[3:69] != 9).any(-1).all()
    # reading: zeros where there is no page, rows of no sequence untouched
    ko, vo = (torch.full((T, Hkv, D), 9.0, dtype=torch.float16, device="cuda") for _ in range(2))
    W4.kv_read_paged(kp, vp, table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), cu, out=(ko, vo))
    for out in (ko, vo):
        zero = (out == 0).all(-1).all(-1).cpu()
        assert (out[:3] == 9).all() and (out[69:] == 9).all()
        assert zero[3:23].all() and not zero[23:39].any() and zero[39:43].all()
        assert zero[43:59].all() and not zero[59:63].any() and zero[63:65].all() and not zero[65:69].any()


@pytest.mark.parametrize("codes", CODES, ids=ids)
def test_append_values_that_are_no_numbers(codes):
    D, page, nan, inf = 64, 16, float("nan"), float("inf")
    k, v = fused(5, [1, 1], D, torch.float16, 5)
    k, v = k.clone(), v.clone()
    k[2, 0, :4] = v[2, 0, :4] = torch.tensor([nan, inf, -inf, 0.5])
    kp, vp = W4.kv_pages(2, 1, page, D, codes)
    table = torch.tensor([[1]], dtype=torch.int32).cuda()
    W4.kv_append_paged(k, v, kp, vp, table, torch.tensor([5], dtype=torch.int32).cuda(), starts([5]))
    for x, (c, s), axis in ((k, kp, 0), (v, vp, 1)):
        host = HostCache(page, codes)
        host.write(x[:, 0].float().cpu().numpy(), 0)
        got = f64(c.cpu().float())[1, 0]
        got = got if axis == 0 else got.T
        assert float(s[1, 0]) == host.pages[0][1] and np.array_equal(got[:5], host.pages[0][0])
        assert got[2, 0] == 0 and got[2, 1] == TOP[codes] and got[2, 2] == -TOP[codes]


def test_append_zeros_and_subnormals():
    D, page = 64, 16
    kp, vp = W4.kv_pages(1, 1, page, D)
    table = torch.zeros((1, 1), dtype=torch.int32).cuda()
    z = torch.zeros((2, 1, D), dtype=torch.bfloat16, device="cuda")
    W4.kv_append_paged(z, z, kp, vp, table, torch.tensor([2], dtype=torch.int32).cuda(), starts([2]))
    assert (kp[1] == 0).all() and (kp[0][0, 0, :2] == 0).all() and (vp[0][0, 0, :, :2] == 0).all()
    z[:] = 2.0 ** -130
    W4.kv_append_paged(z[:1], z[:1], kp, vp, table, torch.tensor([3], dtype=torch.int32).cuda())
    host = HostCache(page, torch.int8)
    host.write(np.full((1, D), 2.0 ** -130, np.float32), 0)
    assert float(kp[1]) == host.pages[0][1] and (kp[0][0, 0, 2].cpu().numpy() == host.pages[0][0][0]).all()
    z[:] = 1.0
    W4.kv_append_paged(z[:1], z[:1], kp, vp, table, torch.tensor([4], dtype=torch.int32).cuda())
    assert (kp[0][0, 0, 3] == 127).all() and (kp[0][0, 0, :3] == 0).all() and (vp[0][0, 0, :, 3] == 127).all()


# --------------------------------------------------------------------------- attention

def attend(lengths, n, Hq, Hkv, D, page, codes, dtype, seed, decode=False, scale=1.0, qscale=1.0, change=None, room=0):
    pool = Pool(lengths, Hkv, D, page, codes, seed, scale, room)
    if change:
        change(pool)
    T = sum(n)
    q, _ = fused(T, [Hq, 1], D, dtype, seed + 1, qscale)
    out = torch.full((T, Hq, D), 9.0, dtype=dtype, device="cuda")
    kp, vp, table, lens = pool.cuda()
    got = W4.kv_attention_paged(q, kp, vp, table, lens, None if decode else starts(n), out=out)
    assert got is out
    at = 0
    for b in range(len(lengths)):
        check_attention(f64(out[at:at + n[b]]), f64(q[at:at + n[b]]), pool, b, n[b], Hq, dtype)
        at += n[b]
    return out


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("codes", CODES, ids=ids)
@pytest.mark.parametrize("Hq,Hkv,D,page", [(8, 2, 64, 16), (4, 4, 128, 32), (6, 1, 128, 64), (32, 1, 64, 128),
                                           (17, 1, 128, 16), (3, 3, 64, 64)])
def test_decode(Hq, Hkv, D, page, codes, dtype):
    lengths = [1, 0, 63, 64, 65, 2, 130, 700, 16, 17]
    attend(lengths, [1] * len(lengths), Hq, Hkv, D, page, codes, dtype, D + page, decode=True)


@pytest.mark.parametrize("codes", CODES, ids=ids)
@pytest.mark.parametrize("Hq,Hkv,D,page", [(8, 2, 128, 64), (2, 2, 64, 16)])
def test_decode_long(Hq, Hkv, D, page, codes):
    """Sequences that are split over blocks, next to short and empty ones."""
    attend([5000, 3, 0, 1025, 20000], [1] * 5, Hq, Hkv, D, page, codes, torch.float16, 7, decode=True, qscale=1.5)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("codes", CODES, ids=ids)
@pytest.mark.parametrize("Hq,Hkv,D,page", [(4, 1, 128, 64), (2, 2, 64, 16), (3, 1, 128, 32), (5, 1, 64, 128)])
def test_chunks(Hq, Hkv, D, page, codes, dtype):
    """Chunks behind cached tokens, whole prompts, empty ones, single tokens and more rows than tokens."""
    lengths, n = [150, 77, 5, 40, 300, 3, 129], [33, 77, 0, 1, 130, 5, 64]
    attend(lengths, n, Hq, Hkv, D, page, codes, dtype, D + page)


@pytest.mark.parametrize("codes", CODES, ids=ids)
def test_chunks_long(codes):
    attend([2500, 40, 1200], [20, 40, 3], 4, 2, 128, 64, codes, torch.bfloat16, 11)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("codes", CODES, ids=ids)
@pytest.mark.parametrize("page", [16, 64, 128])
def test_chunks_of_many_rows(page, codes, dtype):
    """Hundreds of rows a sequence (256 to a block), split over blocks, beside a short, an empty and one with more
    rows than tokens; pages that are none and of scale 0 in between."""
    def change(pool):
        pool.table[0, 2] = -1
        pool.table[0, 600 // page] = 1 << 30
        pool.vs[pool.table[1, 1]] = 0.0
        pool.ks[pool.table[1, 3]] = 0.0
    attend([2100, 1200, 30, 0], [301, 220, 33, 0], 4, 1, 128, page, codes, dtype, 13 + page, change=change)


@pytest.mark.parametrize("codes", CODES, ids=ids)
@pytest.mark.parametrize("decode", [True, False])
def test_entries_that_are_no_pages(codes, decode):
    """Tokens there are not attended to: in the middle, the last page, a whole sequence."""
    def change(pool):
        pool.table[0, 1] = -1
        pool.table[1, 2] = pool.kc.shape[0]
        pool.table[2, :] = -5
        pool.table[3, 0] = 2 ** 31 - 1
    n = [1] * 4 if decode else [20, 3, 5, 40]
    attend([100, 70, 50, 1300], n, 4, 2, 64, 32, codes, torch.float16, 21, decode=decode, change=change)


@pytest.mark.parametrize("codes", CODES, ids=ids)
@pytest.mark.parametrize("spread", [1e-3, 1e4, 1e8])
def test_scales_far_apart(codes, spread):
    """V's scales grow and fall along a sequence by large factors."""
    def change(pool):
        for b, row in enumerate(pool.table.tolist()):
            for i, p in enumerate(row):
                if p >= 0:
                    pool.vs[p] *= spread ** (((i + b) % 3) / 2) * (1e-4 if spread > 1e6 else 1.0)
    attend([400, 131, 1500], [1, 1, 1], 4, 1, 128, 16, codes, torch.bfloat16, 31, decode=True, change=change)
    attend([400, 131], [17, 90], 2, 1, 64, 16, codes, torch.bfloat16, 32, change=change)


def test_one_page_outweighs_all():
    """A key that takes nearly all the weight, late and early, in a long sequence."""
    def change(pool):
        pool.ks[pool.table[0, 3]] *= 60
        pool.ks[pool.table[1, 200]] *= 60
    attend([5000, 5000], [1, 1], 4, 2, 64, 16, torch.int8, torch.float16, 41, decode=True, qscale=3.0, change=change)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("n,page", [(1, 64), (1, 16), (40, 64), (40, 16), (300, 64)])
def test_many_faint_tokens(n, page, dtype):
    """One token of score 26 (base 2) whose V is 0 before 32768 of score 0 and V 1: all weights are powers of two, and
    each output is L / (L + 2^26) for the L of them that its row sees, which 16 bits hold to half a step (the rest:
    fp32 scores and sums)."""
    L = 1 << 15
    P = (L + 1 + n) // page + 1
    (kc, ks), (vc, vs) = kp, vp = W4.kv_pages(P, 1, page, 128, torch.int8)
    kc.zero_(), vc.fill_(127), ks.fill_(1.0), vs.fill_(1.0 / 127)
    kc[0, 0, 0, 0], vc[0, 0, :, 0] = 127, 0
    ks[0] = 26.0 * 128 ** 0.5 / (1.4426950408889634 * 127)
    table = torch.arange(P, dtype=torch.int32, device="cuda")[None]
    lengths = torch.tensor([L + 1], dtype=torch.int32, device="cuda")
    q = torch.zeros((n, 1, 128), dtype=dtype, device="cuda")
    q[:, :, 0] = 1.0
    got = W4.kv_attention_paged(q, kp, vp, table, lengths, starts([n]) if n > 1 else None).double()
    faint = (L - n + 1 + torch.arange(n, device="cuda").double())[:, None, None]
    ref = faint / (faint + 2.0 ** 26)
    assert ((got - ref).abs() <= (torch.finfo(dtype).eps / 2 + 2.0 ** -14) * ref).all()


@pytest.mark.parametrize("decode", [True, False])
def test_queries_that_are_no_numbers(decode):
    D, Hq, Hkv, page = 128, 8, 2, 32
    pool = Pool([900, 80, 2000], Hkv, D, page, torch.int8, 51)
    n = [1, 1, 1] if decode else [9, 80, 5]
    T = sum(n)
    q, = fused(T, [Hq], D, torch.float16, 52)
    kp, vp, table, lens = pool.cuda()
    cu = None if decode else starts(n)
    want = W4.kv_attention_paged(q, kp, vp, table, lens, cu)
    bad = q.clone()
    bad[0, 1, 5], bad[1, 6, 0], bad[T - 1, 7] = float("nan"), float("inf"), float("-inf")
    got = W4.kv_attention_paged(bad, kp, vp, table, lens, cu)
    odd = torch.zeros((T, Hq), dtype=torch.bool, device="cuda")
    odd[0, 1] = odd[1, 6] = odd[T - 1, 7] = True
    assert torch.isnan(got[odd]).any(-1).all()
    assert torch.equal(got[~odd], want[~odd])


def test_shared_pages():
    """Two sequences that begin with the same pages."""
    def change(pool):
        pool.table[1, :4] = pool.table[0, :4]
    attend([100, 90, 200], [1, 1, 1], 4, 2, 128, 16, torch.int8, torch.float16, 61, decode=True, change=change)
    attend([100, 90, 200], [30, 20, 5], 4, 2, 128, 16, torch.int8, torch.float16, 62, change=change)


def test_rows_of_no_sequence_are_left():
    D, Hq, Hkv, page, T = 64, 4, 2, 16, 60
    pool = Pool([30, 50], Hkv, D, page, torch.float8_e4m3fn, 71)
    q, = fused(T, [Hq], D, torch.bfloat16, 72)
    q[:4] = float("nan")
    kp, vp, table, lens = pool.cuda()
    out = torch.full((T, Hq, D), 9.0, dtype=q.dtype, device="cuda")
    cu = torch.tensor([4, 24, 50], dtype=torch.int32).cuda()
    W4.kv_attention_paged(q, kp, vp, table, lens, cu, out=out)
    assert (out[:4] == 9).all() and (out[50:] == 9).all()
    check_attention(f64(out[4:24]), f64(q[4:24]), pool, 0, 20, Hq, q.dtype)
    check_attention(f64(out[24:50]), f64(q[24:50]), pool, 1, 26, Hq, q.dtype)


@pytest.mark.parametrize("B", [63, 64, 65, 200])
def test_many_sequences(B):
    """More sequences than a wave has lanes, some far longer than others."""
    rng = np.random.default_rng(B)
    lengths = [int(x) for x in rng.integers(0, 60, B)]
    lengths[B // 3], lengths[B - 1] = 3000, 1500
    attend(lengths, [1] * B, 2, 1, 64, 16, torch.int8, torch.float16, B, decode=True)
    n = [min(x, int(y)) for x, y in zip(lengths, rng.integers(0, 12, B))]
    attend(lengths, n, 2, 1, 64, 16, torch.int8, torch.float16, B + 1)


def test_tables_wider_than_the_sequences():
    attend([40, 1, 300], [1, 1, 1], 8, 2, 128, 64, torch.int8, torch.float16, 81, decode=True, room=500)
    attend([40, 1, 300], [7, 1, 200], 8, 2, 128, 64, torch.int8, torch.float16, 82, room=500)


# --------------------------------------------------------------------------- together

@pytest.mark.parametrize("codes", CODES, ids=ids)
def test_serving_loop(codes):
    """Prompts, then steps, with page allocation as a server does it: every output against attention in fp64 over
    what reading back gives, and the rows that were read within the codes' steps of the rotated ones."""
    D, Hq, Hkv, page, dtype, B = 128, 8, 2, 16, torch.bfloat16, 3
    kp, vp = W4.kv_pages(64, Hkv, page, D, codes)
    free = torch.randperm(64, generator=torch.Generator().manual_seed(1)).tolist()
    table = torch.full((B, 20), -1, dtype=torch.int32)
    freqs, m = W4.rope_frequencies(D, 10000.0, "ramp", factor=4.0, original=128, low=1.0, high=32.0)
    length = [0] * B
    for step, n in enumerate([[40, 7, 65], [1, 1, 1], [1, 1, 1], [20, 1, 3], [1, 1, 1]]):
        length = [a + b for a, b in zip(length, n)]
        for b in range(B):
            for i in range(-(-length[b] // page)):
                if table[b, i] < 0:
                    table[b, i] = free.pop()
        q, k, v = fused(sum(n), [Hq, Hkv, Hkv], D, dtype, step)
        cu = None if n == [1] * B else starts(n)
        args = (kp, vp, table.cuda(), torch.tensor(length, dtype=torch.int32).cuda())
        qr = W4.kv_append_paged(k, v, *args, cu, freqs=freqs, mscale=m, q=q)
        out = f64(W4.kv_attention_paged(qr, *args, cu))
        kk, vv = W4.kv_read_paged(*args, starts(length), T=sum(length), dtype=dtype)
        at = first = 0
        for b in range(B):
            K, V = f64(kk[first:first + length[b]]), f64(vv[first:first + length[b]])
            for i in range(n[b]):
                see = length[b] - n[b] + i + 1
                for h in range(Hq):
                    s = K[:see, h // 4] @ f64(qr[at + i, h]) / np.sqrt(D)
                    p = np.exp(s - s.max())
                    p /= p.sum()
                    # the rows were rounded to bf16 on reading: K's moves a weight by up to 2^-8 of sum |q k| / sqrt(D)
                    # twice, V's an output by 2^-8
                    move = 2.0 ** -8 * (np.abs(K[:see, h // 4]) @ np.abs(f64(qr[at + i, h]))).max() / np.sqrt(D)
                    tol = (2.0 ** -7 + 2.0 ** -10 + np.expm1(2 * move)) * (p @ np.abs(V[:see, h // 4])) + 1e-6
                    assert (np.abs(out[at + i, h] - p @ V[:see, h // 4]) <= tol).all()
            at += n[b]
            first += length[b]


def graph_of(fn):
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        fn()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=side):
            fn()
    torch.cuda.synchronize()
    return graph


def test_captured_steps():
    """A decode step in a captured graph, replayed on lengths and inputs that change in place, against eager
    calls on a copy of the cache."""
    D, Hq, Hkv, page, B, dtype = 128, 8, 2, 16, 3, torch.float16
    lengths = [1500, 5, 200]
    pool = Pool(lengths, Hkv, D, page, torch.int8, 91, room=2)
    used = set(pool.table[pool.table >= 0].tolist())
    free = [i for i in range(pool.kc.shape[0]) if i not in used]
    for b in range(B):
        pool.table[b, -(-lengths[b] // page)] = free[b]         # the next page of each
    kp, vp, table, lens = pool.cuda()
    copy = tuple(tuple(t.clone() for t in c) for c in (kp, vp))
    q, k, v = fused(B, [Hq, Hkv, Hkv], D, dtype, 92)
    freqs, _ = W4.rope_frequencies(D)
    qo, out = torch.empty((B, Hq, D), dtype=dtype, device="cuda"), torch.empty((B, Hq, D), dtype=dtype, device="cuda")
    work = torch.empty(W4.kv_attention_paged_workspace(Hq, Hkv, D, table.shape[1] * page), device="cuda")
    start = lens.clone()

    def step():
        W4.kv_append_paged(k, v, kp, vp, table, lens, freqs=freqs, q=q, q_out=qo)
        W4.kv_attention_paged(qo, kp, vp, table, lens, out=out, work=work)
    graph = graph_of(step)
    for a, c in ((kp, copy[0]), (vp, copy[1])):
        for x, y in zip(a, c):
            x.copy_(y)
    for rep in range(6):
        lens.copy_(start + rep)
        for t in (q, k, v):
            t.copy_(torch.randn(t.shape, generator=torch.Generator().manual_seed(rep)))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        q2 = W4.kv_append_paged(k, v, *copy, table, lens, freqs=freqs, q=q)
        want = W4.kv_attention_paged(q2, *copy, table, lens)
        assert torch.equal(out, want) and torch.equal(qo, q2)
        for a, c in ((kp, copy[0]), (vp, copy[1])):
            for x, y in zip(a, c):
                assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


def test_two_streams():
    """Calls on two streams with workspaces of their own."""
    D, Hq, Hkv, page = 128, 8, 2, 16
    a, b = (Pool([4000, 900], Hkv, D, page, torch.int8, 100 + i) for i in range(2))
    qs = [fused(2, [Hq], D, torch.float16, 110 + i)[0] for i in range(2)]
    data = [p.cuda() for p in (a, b)]
    want = [W4.kv_attention_paged(q, *d) for q, d in zip(qs, data)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [[torch.empty_like(q) for _ in range(20)] for q in qs]
    works = [torch.empty(W4.kv_attention_paged_workspace(Hq, Hkv, D, 4096), device="cuda") for _ in range(2)]
    for i in range(20):
        for s, q, d, o, w in zip(streams, qs, data, outs, works):
            with torch.cuda.stream(s):
                W4.kv_attention_paged(q, *d, out=o[i], work=w)
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        for x in o:
            assert torch.equal(x, w)


# --------------------------------------------------------------------------- what calls may meet

@pytest.mark.parametrize("codes", CODES, ids=ids)
@pytest.mark.parametrize("counts", [[1, 1, 1], [70, 3, 200]])
def test_pools_past_four_gib(counts, codes):
    """The same sequences at the end of a pool of 4.5 GiB a cache and in a small one: the same bits."""
    Hkv, D, page, dtype = 8, 128, 128, torch.bfloat16
    lengths, T = [700, 130, 1500], sum(counts)
    cu = None if counts == [1, 1, 1] else starts(counts)
    outcome = []
    for N in (32, 36864):                                  # pages of 128 KiB
        kp, vp = W4.kv_pages(N, Hkv, page, D, codes)
        pages = list(range(N - 1, N - 21, -1))
        table = torch.full((3, 12), -1, dtype=torch.int32)
        for b in range(3):
            for j in range(-(-lengths[b] // page)):
                table[b, j] = pages.pop()
        table, lens = table.cuda(), torch.tensor(lengths, dtype=torch.int32).cuda()
        k, v = fused(sum(lengths), [Hkv, Hkv], D, dtype, 1)
        freqs, _ = W4.rope_frequencies(D)
        W4.kv_append_paged(k, v, kp, vp, table, lens, starts(lengths), freqs=freqs)
        q, k, v = fused(T, [4 * Hkv, Hkv, Hkv], D, dtype, 2, 3.0)
        qo = W4.kv_append_paged(k, v, kp, vp, table, lens, cu, freqs=freqs, q=q)
        outcome.append((W4.kv_attention_paged(qo, kp, vp, table, lens, cu),
                        *W4.kv_read_paged(kp, vp, table, lens, starts(lengths), T=sum(lengths), dtype=dtype)))
        del kp, vp
    for a, b in zip(*outcome):
        assert torch.equal(a, b)
    assert outcome[0][0].float().abs().max() > 0


def test_chunks_of_hundreds_of_sequences():
    """Appending, reading and attending for 150 sequences of a call against a call for each."""
    Hkv, Hq, D, page, B, dtype = 2, 4, 64, 16, 150, torch.float16
    rng = np.random.default_rng(5)
    counts = [int(c) for c in rng.integers(0, 40, B)]
    lengths = [c + int(x) for c, x in zip(counts, rng.integers(0, 90, B))]
    P = 9
    table = torch.randperm(B * P, generator=torch.Generator().manual_seed(1)).view(B, P).to(torch.int32).cuda()
    lens = torch.tensor(lengths, dtype=torch.int32).cuda()
    T = sum(counts)
    q, k, v = fused(T, [Hq, Hkv, Hkv], D, dtype, 6)
    freqs, _ = W4.rope_frequencies(D)
    kp, vp = W4.kv_pages(B * P, Hkv, page, D)
    copy = tuple(tuple(t.clone() for t in c) for c in (kp, vp))
    cu = starts(counts)
    qo = W4.kv_append_paged(k, v, kp, vp, table, lens, cu, freqs=freqs, q=q)
    got = (qo, W4.kv_attention_paged(qo, kp, vp, table, lens, cu), *W4.kv_read_paged(kp, vp, table, lens, cu, T=T))
    at = 0
    for b, n in enumerate(counts):
        if n:
            one = (table[b:b + 1], lens[b:b + 1], starts([n]))
            rows = slice(at, at + n)
            q1 = W4.kv_append_paged(k[rows], v[rows], *copy, *one, freqs=freqs, q=q[rows])
            kv1 = W4.kv_read_paged(*copy, *one, T=n)
            assert torch.equal(got[0][rows], q1)
            assert torch.equal(got[2][rows], kv1[0]) and torch.equal(got[3][rows], kv1[1])
            # (another kernel may serve the one sequence: the same up to roundings of weights and output)
            o1 = W4.kv_attention_paged(q1, *copy, *one)
            assert (got[1][rows].float() - o1.float()).abs().max() <= 4 * 2.0 ** -11 * max(1.0, float(kv1[1].abs().max()))
        at += n
    for a, c in zip((*kp, *vp), (*copy[0], *copy[1])):
        assert torch.equal(a.view(torch.uint8), c.view(torch.uint8))


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_rows_that_are_no_numbers_in_long_chunks(dtype):
    """Blocks of 256 rows: only the rows whose query is no number differ."""
    D, Hq, Hkv, page = 128, 4, 1, 64
    pool = Pool([2500], Hkv, D, page, torch.int8, 53)
    n = 400
    q, = fused(n, [Hq], D, dtype, 54)
    kp, vp, table, lens = pool.cuda()
    want = W4.kv_attention_paged(q, kp, vp, table, lens, starts([n]))
    bad = q.clone()
    bad[3, 1, 5], bad[200, 3, 0], bad[n - 1, 0] = float("nan"), float("inf"), float("-inf")
    got = W4.kv_attention_paged(bad, kp, vp, table, lens, starts([n]))
    odd = torch.zeros((n, Hq), dtype=torch.bool, device="cuda")
    odd[3, 1] = odd[200, 3] = odd[n - 1, 0] = True
    assert torch.isnan(got[odd]).any(-1).all()
    assert torch.equal(got[~odd], want[~odd])


@pytest.mark.parametrize("n", [1, 40, 400])
@pytest.mark.parametrize("size", [1.0e5, 3.0e34])
def test_scores_past_the_whole_numbers_of_fp32(n, size):
    """Scores of 10^7 and of 10^36: one key takes all the weight and its V comes out exactly (V's codes and scale
    are whole)."""
    D, page, L = 128, 32, 1200
    P = -(-L // page)
    (kc, ks), (vc, vs) = kp, vp = W4.kv_pages(P, 1, page, D)
    best = 500
    kc[:, :, :, 0] = 3
    kc[best // page, 0, best % page, 0] = 100
    vc.copy_(torch.randint(-100, 101, vc.shape, dtype=torch.int8, generator=torch.Generator().manual_seed(3)))
    ks.fill_(size)
    vs.fill_(2.0)
    q = torch.zeros((n, 1, D), dtype=torch.bfloat16, device="cuda")
    q[:, :, 0] = 16.0
    table = torch.arange(P, dtype=torch.int32, device="cuda")[None]
    lens = torch.tensor([L], dtype=torch.int32, device="cuda")
    got = W4.kv_attention_paged(q, kp, vp, table, lens, None if n == 1 else starts([n]))
    want = 2.0 * vc[best // page, 0, :, best % page].to(torch.bfloat16)
    assert torch.equal(got, want.expand(n, 1, D))


def test_whatever_stands_in_the_tables():
    """The largest and smallest whole numbers, and starts that decrease: outputs of sound sequences beside
    them are as ever where starts are sound, and nothing outside is written where they are not."""
    Hkv, Hq, D, page, dtype = 2, 8, 64, 16, torch.float16
    lo, hi = -2 ** 31, 2 ** 31 - 1
    pool = Pool([1500, 40, 900], Hkv, D, page, torch.int8, 61)
    kp, vp, table, lens = pool.cuda()
    q, = fused(3, [Hq], D, dtype, 62)
    want = W4.kv_attention_paged(q, kp, vp, table, lens)
    for place, value in ((0, lo), (0, hi), (1, lo)):
        l2 = lens.clone()
        l2[1] = value
        t2 = table.clone()
        t2[1, place] = value
        got = W4.kv_attention_paged(q, kp, vp, t2, l2)
        assert torch.equal(got[[0, 2]], want[[0, 2]])
        W4.kv_read_paged(kp, vp, t2, l2)
    before = [t.clone() for t in (*kp, *vp)]
    k, v = fused(3, [Hkv, Hkv], D, dtype, 63)
    none = torch.full_like(table, lo)
    W4.kv_append_paged(k, v, kp, vp, none, torch.tensor([lo, hi, 0], dtype=torch.int32).cuda())
    W4.kv_append_paged(k, v, kp, vp, none, torch.tensor([hi, lo, 5], dtype=torch.int32).cuda(), starts([1, 1, 1]))
    for t, b in zip((*kp, *vp), before):
        assert torch.equal(t.view(torch.uint8), b.view(torch.uint8))
    for T in (3, 300):
        big = torch.full((T + 2, Hq, D), 7.0, dtype=dtype, device="cuda")
        q, = fused(T, [Hq], D, dtype, 64)
        for cu in ([T, 0, T, 0], [lo, hi, lo, hi], [hi, hi, lo, lo], [2, 1, 0, hi]):
            cu = torch.tensor(cu, dtype=torch.int32).cuda()
            W4.kv_attention_paged(q, kp, vp, table, lens, cu, out=big[1:T + 1])
            W4.kv_read_paged(kp, vp, table, lens, cu, T=T)
        assert (big[0] == 7).all() and (big[T + 1] == 7).all()


def test_two_graphs():
    """A captured decode step and a captured chunk, scratch of their own captures, replayed in turn."""
    D, Hq, Hkv, page = 128, 8, 2, 16
    pools = [Pool(lengths, Hkv, D, page, torch.int8, 71 + i) for i, lengths in enumerate(([3000, 800], [2500]))]
    data = [p.cuda() for p in pools]
    qs = [fused(n, [Hq], D, torch.bfloat16, 73 + n)[0] for n in (2, 300)]
    cus = [None, starts([300])]
    outs = [torch.empty(q.shape, dtype=q.dtype, device="cuda") for q in qs]
    graphs = [graph_of(lambda i=i: W4.kv_attention_paged(qs[i], *data[i], cus[i], out=outs[i])) for i in range(2)]
    for rep in range(4):
        for i in (0, 1, 0):
            qs[i].copy_(torch.randn(qs[i].shape, generator=torch.Generator().manual_seed(10 * rep + i)))
            data[i][3][0] -= 17
            outs[i].zero_()
            graphs[i].replay()
            want = W4.kv_attention_paged(qs[i], *data[i], cus[i])
            assert torch.equal(outs[i], want)


def test_single_rows_of_wide_tensors():
    """One token: rows of whatever distance, heads in the middle of a wider row."""
    D, Hkv, page = 64, 2, 16
    kp, vp = W4.kv_pages(4, Hkv, page, D)
    wide = torch.randn((1, 5 * Hkv * D), generator=torch.Generator().manual_seed(1)).half().cuda()
    part = lambda i: wide[:, i * Hkv * D:(i + 1) * Hkv * D].unflatten(1, (Hkv, D))
    table = torch.tensor([[2, 1]], dtype=torch.int32).cuda()
    one = torch.tensor([1], dtype=torch.int32).cuda()
    freqs, _ = W4.rope_frequencies(D)
    qo = W4.kv_append_paged(part(1), part(3), kp, vp, table, one, freqs=freqs, q=part(4))
    got = W4.kv_attention_paged(qo, kp, vp, table, one)
    assert torch.equal(qo, part(4))                        # (place 0)
    # (half a step of the codes; fp16 roundings of the weight and of the output, of values below 8)
    tol = part(3).float().abs().amax(2, keepdim=True) / 127 / 2 + 2 * 8 * 2.0 ** -11
    assert ((got.float() - part(3).float()).abs() <= tol).all()


@pytest.mark.parametrize("n,counts", [(5, 200), (3, 300), (6, 90), (2, 700)])
def test_cuts_that_fit_the_gpu(n, counts):
    """Chunks of several sequences whose even cut would not fit into one round of blocks, against a call for each
    sequence (cut otherwise): the same up to the roundings of weights and outputs."""
    D, Hkv, page, L = 128, 8, 64, 6000
    pool = Pool([L] * n, Hkv, D, page, torch.int8, 121, outliers=False)
    kp, vp, table, lens = pool.cuda()
    q, = fused(n * counts, [Hkv], D, torch.float16, 122)
    got = W4.kv_attention_paged(q, kp, vp, table, lens, starts([counts] * n)).float()
    vmax = float(np.nanmax(f64(pool.vs))) * 127
    for b in range(n):
        rows = slice(b * counts, (b + 1) * counts)
        want = W4.kv_attention_paged(q[rows], kp, vp, table[b:b + 1], lens[b:b + 1], starts([counts])).float()
        # (each side: 2^-11 sum p (|v| + |out|) of the weights, 2^-11 |out| of the output, fp32 sums)
        assert (got[rows] - want).abs().max() <= 2 * 3.1 * 2.0 ** -11 * vmax
        # (over a row of uncorrelated values each of the two sides' two roundings has at most 2^-11 of the norm)
        assert (got[rows] - want).norm() <= 4 * 2.0 ** -11 * want.norm()


def test_descriptions_that_are_wrong():
    """The binding names what is wrong with a cache's description, whichever way it is wrong."""
    kp, vp = W4.kv_pages(4, 2, 16, 64)
    table = torch.zeros((3, 2), dtype=torch.int32, device="cuda")
    lens = torch.ones(3, dtype=torch.int32, device="cuda")
    q = torch.zeros((3, 4, 64), dtype=torch.float16, device="cuda")
    cu = starts([1, 1, 1])
    good = dict(kpages=kp, vpages=vp, table=table, lengths=lens, cu_seqlens=None)
    W4.kv_attention_paged(q, **good)
    for error, change in ((TypeError, dict(kpages=(None, kp[1]))), (TypeError, dict(vpages=(vp[0], 3.0))),
                          (TypeError, dict(kpages=(kp[0].cpu().numpy(), kp[1]))),
                          (TypeError, dict(vpages=(vp[0].view(torch.uint8), vp[1]))),
                          (TypeError, dict(kpages=(kp[0], kp[1].double()))), (TypeError, dict(table=None)),
                          (TypeError, dict(table=table.long())), (TypeError, dict(lengths=[1, 1, 1])),
                          (TypeError, dict(lengths=lens.float())), (TypeError, dict(cu_seqlens=cu.long())),
                          (ValueError, dict(kpages=(kp[0][0], kp[1]))), (ValueError, dict(kpages=(kp[0][:, :1], kp[1]))),
                          (ValueError, dict(kpages=vp)), (ValueError, dict(kpages=(kp[0], kp[1][:2]))),
                          (ValueError, dict(table=table[0])), (ValueError, dict(table=table[:2])),
                          (ValueError, dict(table=table.t().contiguous().t())), (ValueError, dict(lengths=lens[:, None])),
                          (ValueError, dict(lengths=lens.cpu())), (ValueError, dict(cu_seqlens=cu[1:])),
                          (ValueError, dict(kpages=(kp[0].cpu(), kp[1].cpu()))),
                          (ValueError, dict(table=table[:2], lengths=lens[:2]))):
        with pytest.raises(error):
            W4.kv_attention_paged(q, **{**good, **change})
        with pytest.raises(error):
            W4.kv_append_paged(q[:, :2].contiguous(), q[:, :2].contiguous(), **{**good, **change})
    for error, T in ((ValueError, None), (TypeError, 3.0), (ValueError, 2 ** 70), (W4.W4A16Error, 0)):
        with pytest.raises(error):
            W4.kv_read_paged(kp, vp, table, lens, cu, T=T)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("step", [True, False])
def test_queries_without_rotation_are_copied(D, step):
    """Without frequencies q comes out as it went in, and K as without q."""
    Hkv, Hq, page = 2, 6, 16
    n = [1, 1, 1] if step else [5, 0, 33]
    T = sum(n)
    q, k, v = fused(T, [Hq, Hkv, Hkv], D, torch.bfloat16, 131)
    table = torch.arange(9, dtype=torch.int32, device="cuda").view(3, 3)
    lens = torch.tensor([max(c, 1) for c in n], dtype=torch.int32, device="cuda")
    cu = None if step else starts(n)
    pools = [W4.kv_pages(9, Hkv, page, D) for _ in range(2)]
    qo = W4.kv_append_paged(k, v, *pools[0], table, lens, cu, q=q)
    assert W4.kv_append_paged(k, v, *pools[1], table, lens, cu) is None
    assert torch.equal(qo, q)
    for a, b in zip(*pools):
        for x, y in zip(a, b):
            assert torch.equal(x, y)
    assert pools[0][0][0].any()
