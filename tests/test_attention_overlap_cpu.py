"""Outputs and workspaces of the cache attention and eviction calls that overlap an input, or one another, are
refused before anything is enqueued (host only, made-up device addresses that nothing reads): the kernels
read and write at times of their own and are told that their pointers differ."""

import os

import pytest

import w4a16_dequant_gemm_amd._lib as L

MB = 1 << 20
B, Hq, Hkv, D, T, P, PMAX = 2, 8, 4, 64, 1100, 700, 900
ROWS, PROWS = B * Hkv * T, (Hkv - 1) * PMAX + P
NAMES = ["kcodes", "kscales", "kzeros", "vcodes", "vscales", "vzeros"]


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(L.LIB_PATH):
        from w4a16_dequant_gemm_amd.build import build
        build()
    return L.lib()


def cache(at, bits):
    return {n: None if bits == 8 and "zeros" in n else at + i * 16 * MB for i, n in enumerate(NAMES)}


def size(name, rows, bits):
    return rows * D * bits // 8 if "codes" in name else 2 * rows


def struct(c):
    return L.KvCache(*(c[n] for n in NAMES))


Q, LENS, WORK, OUT, W, SUMS = (0x10000000 + i * 16 * MB for i in range(6))
QBYTES = 2 * B * Hq * D


def shared(lib, bits, **kw):
    a = dict(q=Q, own=cache(0x20000000, bits), prefix=cache(0x30000000, bits), lens=LENS, work=WORK, out=OUT, P=P)
    a.update(kw)
    return lib.w4a16_kv_attention_decode_shared(a["q"], 0, B, Hq, Hkv, D, bits, struct(a["prefix"]), a["P"], PMAX,
                                                struct(a["own"]), a["lens"], T, a["work"], a["out"], None)


def weights(lib, bits, **kw):
    a = dict(q=Q, own=cache(0x20000000, bits), lens=LENS, w=W, sums=SUMS, work=WORK, out=OUT)
    a.update(kw)
    return lib.w4a16_kv_attention_decode_weights(a["q"], 0, B, Hq, Hkv, D, bits, struct(a["own"]), a["lens"], T, a["w"],
                                                 a["sums"], a["work"], a["out"], None)


def touching(lo, n, own, step):
    """Addresses from which `own` bytes just reach into the n bytes from lo, at either end."""
    return [(lo - own) // step * step + step, (lo + n - 1) // step * step]


@pytest.mark.parametrize("bits", [8, 4])
def test_shared(lib, bits):
    work = 4 * (D + 2) * B * Hq             # (at least one split of every row)
    own, pre = cache(0x20000000, bits), cache(0x30000000, bits)
    spans = [(Q, QBYTES), (LENS, 4 * B)]
    spans += [(own[n], size(n, ROWS, bits)) for n in NAMES if own[n]]
    spans += [(pre[n], size(n, PROWS, bits)) for n in NAMES if pre[n]]
    for lo, n in spans:
        for at in touching(lo, n, QBYTES, 2):
            assert shared(lib, bits, out=at) == L.ERR_OVERLAP, hex(at)
        for at in touching(lo, n, work, 16):
            assert shared(lib, bits, work=at) == L.ERR_OVERLAP, hex(at)
    assert shared(lib, bits, out=WORK) == L.ERR_OVERLAP
    assert shared(lib, bits, work=OUT + QBYTES - 16) == L.ERR_OVERLAP


@pytest.mark.parametrize("bits", [8, 4])
def test_weights(lib, bits):
    work, n = 4 * (T + D + 2) * B * Hq, 4 * B * Hkv * T
    own = cache(0x20000000, bits)
    spans = [(Q, QBYTES), (LENS, 4 * B)] + [(own[m], size(m, ROWS, bits)) for m in NAMES if own[m]]
    for lo, m in spans + [(W, n)]:
        for at in touching(lo, m, QBYTES, 2):
            assert weights(lib, bits, out=at) == L.ERR_OVERLAP, hex(at)
        for at in touching(lo, m, n, 4):
            assert weights(lib, bits, sums=at) == L.ERR_OVERLAP, hex(at)
        for at in touching(lo, m, work, 16):
            assert weights(lib, bits, work=at) == L.ERR_OVERLAP, hex(at)
    assert weights(lib, bits, out=SUMS) == L.ERR_OVERLAP
    assert weights(lib, bits, w=SUMS, out=SUMS + n - 2) == L.ERR_OVERLAP      # (accumulation in place)
    assert weights(lib, bits, work=SUMS + n - 8 & -16) == L.ERR_OVERLAP
    assert weights(lib, bits, work=OUT) == L.ERR_OVERLAP
    assert weights(lib, bits, w=SUMS + 4) == L.ERR_OVERLAP


@pytest.mark.parametrize("bits", [8, 4])
def test_evict_workspace(lib, bits):
    tokens, budget, tout = 9000, 50, 60
    src, dst = cache(0x20000000, bits), cache(0x30000000, bits)
    lo, kept = 0x18000000, 0x19000000
    rows = {True: B * Hkv * tokens, False: B * Hkv * tout}

    def call(work):
        return lib.w4a16_kv_evict(struct(src), W, LENS, B, Hkv, tokens, D, bits, budget, 10, struct(dst), tout, SUMS,
                                  lo, kept, work, None)
    used = 4 * B * Hkv * 2 * 6148           # two chunks of a histogram of each digit and a state
    spans = [(W, 4 * rows[True]), (LENS, 4 * B), (SUMS, 4 * rows[False]), (lo, 4 * B), (kept, 4 * B * Hkv * budget)]
    spans += [(c[m], size(m, rows[c is src], bits)) for c in (src, dst) for m in NAMES if c[m]]
    for at, n in spans:
        for w in touching(at, n, used, 16):
            assert call(w) == L.ERR_OVERLAP, hex(w)
