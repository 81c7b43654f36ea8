"""Host-only checks of the attention and eviction entry points (no GPU): every documented refusal
comes back as a status before anything is enqueued (fake device pointers are never dereferenced),
and the workspace sizes cover what they have to."""

import ctypes
import os

import pytest

from w4a16_dequant_gemm_amd import _lib as L

A, B, C, D, E = 0x1000000, 0x2000000, 0x3000000, 0x4000000, 0x5000000


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(L.LIB_PATH):
        from w4a16_dequant_gemm_amd.build import build
        build()
    return L.lib()


def prompt(lib, **kw):
    a = dict(q=A, k=B, v=C, dt=0, T=100, B=2, cu=D, Hq=8, Hkv=4, D=64, qs=1024, ks=1024, vs=1024, out=E)
    a.update(kw)
    return lib.w4a16_attention_prompt(a["q"], a["k"], a["v"], a["dt"], a["T"], a["B"], a["cu"], a["Hq"], a["Hkv"],
                                      a["D"], a["qs"], a["ks"], a["vs"], a["out"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), L.ERR_NULL), (dict(k=None), L.ERR_NULL), (dict(v=None), L.ERR_NULL), (dict(cu=None), L.ERR_NULL),
    (dict(out=None), L.ERR_NULL), (dict(dt=2), L.ERR_DTYPE), (dict(T=0), L.ERR_SHAPE), (dict(B=0), L.ERR_SHAPE),
    (dict(Hkv=3), L.ERR_SHAPE), (dict(Hq=0), L.ERR_SHAPE), (dict(D=96), L.ERR_SHAPE), (dict(qs=504), L.ERR_SHAPE),
    (dict(ks=248), L.ERR_SHAPE), (dict(vs=248), L.ERR_SHAPE), (dict(qs=(1 << 24) + 8), L.ERR_SHAPE),
    (dict(T=(1 << 30) + 1), L.ERR_SHAPE), (dict(T=1 << 30, Hq=64), L.ERR_SHAPE), (dict(B=(1 << 20) + 1), L.ERR_SHAPE),
    (dict(B=1 << 18, Hq=64, qs=4096), L.ERR_SHAPE), (dict(T=1 << 29, Hq=4, qs=1024), L.ERR_SHAPE),
    (dict(qs=1028), L.ERR_ALIGN), (dict(ks=1026), L.ERR_ALIGN), (dict(q=A + 8), L.ERR_ALIGN),
    (dict(k=B + 2), L.ERR_ALIGN), (dict(v=C + 4), L.ERR_ALIGN), (dict(cu=D + 2), L.ERR_ALIGN),
    (dict(out=E + 8), L.ERR_ALIGN), (dict(out=A), L.ERR_OVERLAP), (dict(out=C + 2 * 1024), L.ERR_OVERLAP),
    (dict(out=B + 2 * (99 * 1024 + 4 * 64) - 16), L.ERR_OVERLAP), (dict(out=D - 16), L.ERR_OVERLAP)])
def test_prompt_refusals(lib, kw, status):
    assert prompt(lib, **kw) == status


def cache(bits=8, **kw):
    p = dict(kcodes=A, kscales=A + 0x100000, kzeros=A + 0x200000 if bits == 4 else None, vcodes=A + 0x300000,
             vscales=A + 0x400000, vzeros=A + 0x500000 if bits == 4 else None)
    p.update(kw)
    return L.KvCache(p["kcodes"], p["kscales"], p["kzeros"], p["vcodes"], p["vscales"], p["vzeros"])


BAD_CACHES = [(8, dict(kcodes=None), L.ERR_NULL), (8, dict(kscales=None), L.ERR_NULL), (8, dict(vcodes=None), L.ERR_NULL),
              (8, dict(vscales=None), L.ERR_NULL), (4, dict(kzeros=None), L.ERR_NULL), (4, dict(vzeros=None), L.ERR_NULL),
              (8, dict(kcodes=A + 8), L.ERR_ALIGN), (8, dict(vcodes=A + 4), L.ERR_ALIGN), (8, dict(kscales=A + 1), L.ERR_ALIGN),
              (4, dict(vzeros=A + 1), L.ERR_ALIGN)]
SIZES = [(dict(Hkv=3), L.ERR_SHAPE), (dict(B=0), L.ERR_SHAPE), (dict(B=65536), L.ERR_SHAPE), (dict(D=32), L.ERR_SHAPE),
         (dict(Tmax=0), L.ERR_SHAPE), (dict(Tmax=(1 << 24) + 1), L.ERR_SHAPE), (dict(B=4096, Hq=65532), L.ERR_SHAPE),
         (dict(B=1 << 15, Hq=128), L.ERR_SHAPE), (dict(bits=6), L.ERR_SCHEME), (dict(dt=3), L.ERR_DTYPE), (dict(q=None), L.ERR_NULL), (dict(own=None), L.ERR_NULL),
         (dict(lens=None), L.ERR_NULL), (dict(work=None, Tmax=1100), L.ERR_NULL), (dict(out=None), L.ERR_NULL),
         (dict(q=B + 8), L.ERR_ALIGN), (dict(lens=C + 2), L.ERR_ALIGN), (dict(work=D + 8), L.ERR_ALIGN),
         (dict(out=E + 1), L.ERR_ALIGN)]


def shared(lib, **kw):
    a = dict(q=B, dt=0, B=2, Hq=8, Hkv=4, D=64, bits=8, P=10, Pmax=10, lens=C, Tmax=8, work=D, out=E)
    a.update(kw)
    own = a["own"] if "own" in a else cache(a["bits"])
    prefix = a["prefix"] if "prefix" in a else cache(a["bits"])
    return lib.w4a16_kv_attention_decode_shared(a["q"], a["dt"], a["B"], a["Hq"], a["Hkv"], a["D"], a["bits"], prefix,
                                                a["P"], a["Pmax"], own, a["lens"], a["Tmax"], a["work"], a["out"], None)


def weights(lib, **kw):
    a = dict(q=B, dt=0, B=2, Hq=8, Hkv=4, D=64, bits=8, lens=C, Tmax=8, work=D, out=E, w=E + 0x100000, sums=E + 0x200000)
    a.update(kw)
    own = a["own"] if "own" in a else cache(a["bits"])
    return lib.w4a16_kv_attention_decode_weights(a["q"], a["dt"], a["B"], a["Hq"], a["Hkv"], a["D"], a["bits"], own,
                                                 a["lens"], a["Tmax"], a["w"], a["sums"], a["work"], a["out"], None)


@pytest.mark.parametrize("call", [shared, weights])
@pytest.mark.parametrize("kw,status", SIZES)
def test_decode_refusals(lib, call, kw, status):
    assert call(lib, **kw) == status


@pytest.mark.parametrize("call", [shared, weights])
@pytest.mark.parametrize("bits,kw,status", BAD_CACHES)
def test_decode_cache_refusals(lib, call, bits, kw, status):
    assert call(lib, bits=bits, own=cache(bits, **kw)) == status


def test_shared_prefix_refusals(lib):
    assert shared(lib, P=11) == L.ERR_SHAPE
    assert shared(lib, P=1100, Pmax=1100, work=None) == L.ERR_NULL
    assert shared(lib, P=-1) == L.ERR_SHAPE
    assert shared(lib, Pmax=(1 << 24) + 1) == L.ERR_SHAPE
    assert shared(lib, prefix=None) == L.ERR_NULL
    assert shared(lib, prefix=cache(8, vscales=None)) == L.ERR_NULL
    assert shared(lib, B=60000, Tmax=1 << 24) == L.ERR_SHAPE


def test_weights_refusals(lib):
    assert weights(lib, sums=None) == L.ERR_NULL
    assert weights(lib, w=E + 2) == L.ERR_ALIGN
    assert weights(lib, sums=E + 0x100001) == L.ERR_ALIGN
    assert weights(lib, sums=E + 0x100000 + 4) == L.ERR_OVERLAP      # 2 * 4 * 8 floats from E + 0x100000


def evict(lib, **kw):
    a = dict(bits=8, w=B, lens=C, B=2, Hkv=4, Tmax=100, D=64, budget=50, recent=10, Tout=60, wo=D, lo=D + 0x10000,
             kept=D + 0x20000, work=None)
    a.update(kw)
    shift = E - A
    src = a["src"] if "src" in a else cache(a["bits"])
    dst = a["dst"] if "dst" in a else L.KvCache(*(None if p is None else p + shift for p in (
        getattr(cache(a["bits"]), f) for f, _ in L.KvCache._fields_)))
    return lib.w4a16_kv_evict(src, a["w"], a["lens"], a["B"], a["Hkv"], a["Tmax"], a["D"], a["bits"], a["budget"],
                              a["recent"], dst, a["Tout"], a["wo"], a["lo"], a["kept"], a["work"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(src=None), L.ERR_NULL), (dict(dst=None), L.ERR_NULL), (dict(w=None), L.ERR_NULL), (dict(lens=None), L.ERR_NULL),
    (dict(wo=None), L.ERR_NULL), (dict(lo=None), L.ERR_NULL), (dict(kept=None), L.ERR_NULL), (dict(bits=3), L.ERR_SCHEME),
    (dict(B=0), L.ERR_SHAPE), (dict(D=100), L.ERR_SHAPE), (dict(budget=0), L.ERR_SHAPE), (dict(recent=-1), L.ERR_SHAPE),
    (dict(recent=51), L.ERR_SHAPE), (dict(Tout=49), L.ERR_SHAPE), (dict(Tout=(1 << 24) + 1), L.ERR_SHAPE),
    (dict(Tmax=0), L.ERR_SHAPE), (dict(B=1 << 14, Hkv=256, Tmax=1, Tout=1), L.ERR_SHAPE), (dict(w=B + 2), L.ERR_ALIGN), (dict(wo=D + 1), L.ERR_ALIGN), (dict(lens=C + 1), L.ERR_ALIGN),
    (dict(lo=D + 0x10002), L.ERR_ALIGN), (dict(kept=D + 0x20001), L.ERR_ALIGN),
    (dict(Tmax=8193), L.ERR_NULL), (dict(Tmax=8193, work=D + 0x30008), L.ERR_ALIGN),
    (dict(dst="src"), L.ERR_OVERLAP), (dict(wo=B + 4), L.ERR_OVERLAP), (dict(lo=C), L.ERR_OVERLAP),
    (dict(lo=D), L.ERR_OVERLAP), (dict(kept=A), L.ERR_OVERLAP)])
def test_evict_refusals(lib, kw, status):
    if kw.get("dst") == "src":
        kw = dict(dst=cache(8))
    assert evict(lib, **kw) == status


@pytest.mark.parametrize("bits,kw,status", BAD_CACHES)
def test_evict_cache_refusals(lib, bits, kw, status):
    assert evict(lib, bits=bits, src=cache(bits, **kw)) == status
    assert evict(lib, bits=bits, dst=cache(bits, **kw)) == status


def test_workspaces(lib):
    need = lib.w4a16_kv_attention_shared_workspace
    assert need(2, 8, 4, 1100, 8, 64) >= 2 * 8 * (64 + 2) * 2
    assert need(2, 8, 4, 0, 1100, 64) >= 2 * 8 * (64 + 2)
    assert need(2, 8, 4, 10, 8, 64) == 0 and need(2, 8, 4, 0, 512, 64) == 0
    assert need(2, 8, 3, 10, 8, 64) == L.ERR_SHAPE and need(2, 8, 4, -1, 8, 64) == L.ERR_SHAPE
    assert need(2, 8, 4, 10, 0, 64) == L.ERR_SHAPE and need(2, 8, 4, 10, 8, 65) == L.ERR_SHAPE
    need = lib.w4a16_kv_attention_weights_workspace
    assert need(2, 8, 4, 1100, 64) >= 2 * 8 * (1100 + 64 + 2) and need(2, 34, 2, 9, 64) >= 2 * 34 * (9 + 64 + 2)
    assert need(2, 8, 4, 512, 64) == 0 and need(200, 8, 4, 1000, 64) >= 200 * 8 * 1000
    assert need(2, 8, 3, 9, 64) == L.ERR_SHAPE and need(0, 8, 4, 9, 64) == L.ERR_SHAPE
    assert need(65535, 256, 4, 1 << 13, 64) == L.ERR_SHAPE
    need = lib.w4a16_kv_evict_workspace
    assert need(4, 8, 8192) == 0 and need(4, 8, 8193) > 4 * 8 * 2 * 5120 and need(1, 1, 1 << 24) > 64 * 5120
    assert need(0, 8, 8193) == L.ERR_SHAPE and need(1, 1, (1 << 24) + 1) == L.ERR_SHAPE


def test_overlap_status_has_a_text(lib):
    assert b"overlap" in lib.w4a16_strerror(L.ERR_OVERLAP)
    assert ctypes.sizeof(L.KvCache) == 6 * ctypes.sizeof(ctypes.c_void_p)
