"""Appending chunks of so many sequences that a block takes several heads, one after the other: bit for bit against a
call for each sequence (a head a block), V's codes and scales against the same fp32 steps on the host."""

import numpy as np
import pytest
import torch

import w4a16_dequant_gemm_amd as W4
from tests.paged_util import CODES, HostCache, f64

pytestmark = pytest.mark.gpu
NAMES = {torch.int8: "int8", torch.float8_e4m3fn: "e4m3"}


def starts(counts):
    return torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32).cuda()


@pytest.mark.parametrize("codes", CODES, ids=NAMES.get)
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("page,D,Hkv,B", [(16, 64, 8, 150), (32, 128, 7, 80), (64, 128, 8, 70), (128, 64, 5, 110), (128, 128, 3, 200)])
def test_several_heads_a_block(page, D, Hkv, B, dtype, codes):
    rng = np.random.default_rng(page + D)
    freqs, _ = W4.rope_frequencies(D, 10000.0)
    P = 4
    table = torch.randperm(B * P, generator=torch.Generator().manual_seed(1)).view(B, P).to(torch.int32)
    kp, vp = W4.kv_pages(B * P, Hkv, page, D, codes)
    copy = tuple(tuple(t.clone() for t in c) for c in (kp, vp))
    host = [[HostCache(page, codes) for _ in range(Hkv)] for _ in range(B)]
    length = [0] * B
    grown = kept = 0
    for call in range(3):
        counts = [int(c) for c in rng.integers(0, page + page // 4, B)]
        T = sum(counts)
        # (blocks aimed at: 1024, of pages of 16 2048, K and V apart)
        assert 1024 * (2 if page == 16 else 1) // (2 * (T // page + 2 * B)) < Hkv
        # every (sequence, head) of a size of its own, so that some of the pages begun before grow
        size = np.exp2(rng.uniform(-3, 3, (B, Hkv)))
        seq = np.repeat(np.arange(B), counts)
        x = torch.from_numpy(rng.standard_normal((T, 2 * Hkv, D)) * np.concatenate([size, size[:, ::-1]], 1)[seq][:, :, None])
        k, v = (t.to(dtype).cuda() for t in x.float().split(Hkv, 1))
        wide = torch.cat([k, v], 1)
        k, v = wide[:, :Hkv], wide[:, Hkv:]
        length = [a + b for a, b in zip(length, counts)]
        lens, tab = torch.tensor(length, dtype=torch.int32).cuda(), table.cuda()
        before = vp[1].cpu()
        W4.kv_append_paged(k, v, kp, vp, tab, lens, starts(counts), freqs=freqs)
        at = 0
        for b, n in enumerate(counts):
            if n:
                W4.kv_append_paged(k[at:at + n], v[at:at + n], *copy, tab[b:b + 1], lens[b:b + 1], starts([n]), freqs=freqs)
                rows = v[at:at + n].float().cpu().numpy()
                old = length[b] - n
                for h in range(Hkv):
                    if old % page:
                        s = host[b][h].pages[old // page][1]
                    host[b][h].write(rows[:, h], old)
                    if old % page:
                        more = host[b][h].pages[old // page][1] > s
                        grown, kept = grown + more, kept + (not more)
            at += n
        for x, y in zip((*kp, *vp), (*copy[0], *copy[1])):
            assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
    assert grown > B and kept > B
    c, s = f64(vp[0].cpu().float()), vp[1].cpu().numpy()
    for b in range(B):
        for h in range(Hkv):
            for i, (want, scale) in enumerate(host[b][h].pages):
                if len(want):
                    assert s[table[b, i], h] == scale
                    assert np.array_equal(c[table[b, i], h].T[:len(want)], want), (b, h, i)
