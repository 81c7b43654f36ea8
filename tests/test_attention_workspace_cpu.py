"""The workspace sizes of the attention and eviction calls (host only): a buffer for the largest batch,
prefix and cache of a program holds every smaller call of the same heads, so the sizes never grow where
B, P or Tmax shrink.  A call knows no size of its buffer: one that asked for more than a larger call
would write behind it."""

import os
import random

import pytest

from w4a16_dequant_gemm_amd import _lib as L

HEADS = [(8, 2, 64), (32, 8, 128), (32, 32, 128), (8, 1, 64), (40, 1, 128), (1, 1, 64), (34, 2, 128)]


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(L.LIB_PATH):
        from w4a16_dequant_gemm_amd.build import build
        build()
    return L.lib()


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(2.0 ** rng.uniform(lo.bit_length() - 1, hi.bit_length())))))


@pytest.mark.parametrize("big,small", [((32, 16385, 512), (32, 16384, 512)), ((33, 32768, 1024), (32, 32768, 1024)),
                                       ((64, 600, 400), (4, 600, 400)), ((32, 4096, 513), (32, 4096, 512))])
def test_shared_need_shrinks_with_the_problem(lib, big, small):
    need = lambda s: lib.w4a16_kv_attention_shared_workspace(s[0], 32, 8, s[1], s[2], 128)
    assert need(big) >= need(small) >= 0


@pytest.mark.parametrize("T,less", [(8193, 8192), (1025, 1024), (513, 512), (65537, 65536)])
def test_weights_need_shrinks_with_the_problem(lib, T, less):
    need = lambda n: lib.w4a16_kv_attention_weights_workspace(8, 32, 8, n, 128)
    assert need(T) >= need(less) >= 0


@pytest.mark.parametrize("T,less", [(524289, 524288), (524288, 8193), (8193, 8192), (1 << 24, 1 << 20)])
def test_evict_need_shrinks_with_the_problem(lib, T, less):
    need = lambda n: lib.w4a16_kv_evict_workspace(2, 8, n)
    assert need(T) >= need(less) >= 0


@pytest.mark.parametrize("Hq,Hkv,D", HEADS)
def test_sizes_grow_with_every_dimension(lib, Hq, Hkv, D):
    rng = random.Random(Hq * Hkv * D)
    shared, weights = lib.w4a16_kv_attention_shared_workspace, lib.w4a16_kv_attention_weights_workspace
    evict = lib.w4a16_kv_evict_workspace
    for _ in range(20000):
        B, P, T = _log(rng, 1, 512), rng.choice([0, _log(rng, 1, 1 << 16)]), _log(rng, 1, 1 << 17)
        b, p, t = rng.randint(1, B), rng.randint(0, P), rng.randint(1, T)
        if rng.random() < 0.5:                      # one step below in one of them
            b, p, t = rng.choice([(max(B - 1, 1), P, T), (B, max(P - 1, 0), T), (B, P, max(T - 1, 1))])
        big, small = shared(B, Hq, Hkv, P, T, D), shared(b, Hq, Hkv, p, t, D)
        assert big >= small >= 0, f"shared {(B, P, T)}: {big}, {(b, p, t)}: {small}"
        big, small = weights(B, Hq, Hkv, T, D), weights(b, Hq, Hkv, t, D)
        assert big >= small >= 0, f"weights {(B, T)}: {big}, {(b, t)}: {small}"
        T2 = _log(rng, 1, min(1 << 21, (1 << 33) // (B * Hkv)))     # (a cache has 2^33 rows at most)
        t2 = rng.choice([max(T2 - 1, 1), rng.randint(1, T2)])
        big, small = evict(B, Hkv, T2), evict(b, Hkv, t2)
        assert big >= small >= 0, f"evict {(B, T2)}: {big}, {(b, t2)}: {small}"


def test_a_call_uses_at_most_what_its_size_says(lib):
    """Also within the sizes that need none: the call's own use, over all smaller calls."""
    rng = random.Random(2)
    zero = 0
    for Hq, Hkv, D in HEADS:
        for _ in range(10000):
            B, P, T = _log(rng, 1, 512), rng.choice([0, _log(rng, 1, 1 << 15)]), _log(rng, 1, 1 << 12)
            b, p, t = rng.randint(1, B), rng.randint(0, P), rng.randint(1, T)
            size = lib.w4a16_kv_attention_shared_workspace(B, Hq, Hkv, P, T, D)
            for s in ((B, P, T), (b, p, t)):
                use = lib.w4a16_kv_attention_shared_call_workspace(s[0], Hq, Hkv, s[1], s[2], D)
                assert 0 <= use <= size, f"{(B, P, T)}: {size}, {s} uses {use}"
                zero += use == 0 and size > 0
    assert zero > 0
    assert lib.w4a16_kv_attention_shared_call_workspace(2, 8, 3, 10, 8, 64) == L.ERR_SHAPE


def test_short_sequences_need_none_at_any_smaller_size(lib):
    """Where the size is 0 no buffer is passed at all: no smaller call may want one."""
    rng = random.Random(1)
    for Hq, Hkv, D in HEADS:
        for _ in range(4000):
            B, P, T = _log(rng, 1, 400), rng.randint(0, 1100), rng.randint(1, 1100)
            if lib.w4a16_kv_attention_shared_workspace(B, Hq, Hkv, P, T, D) == 0:
                b, p, t = rng.randint(1, B), rng.randint(0, P), rng.randint(1, T)
                assert lib.w4a16_kv_attention_shared_workspace(b, Hq, Hkv, p, t, D) == 0, (B, P, T, b, p, t)
