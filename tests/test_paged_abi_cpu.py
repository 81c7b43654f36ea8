"""Host-only checks of the rotary and paged-cache entry points (no GPU): every documented refusal comes back as a
status before anything is enqueued (made-up device addresses that nothing reads), and the frequencies."""

import math
import os

import pytest
import torch

import w4a16_dequant_gemm_amd as W4
from w4a16_dequant_gemm_amd import _lib as L

MB = 1 << 20
POOL = 0x40000000


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(L.LIB_PATH):
        from w4a16_dequant_gemm_amd.build import build
        build()
    return L.lib()


BASE = dict(kcodes=POOL, kscales=POOL + 64 * MB, vcodes=POOL + 128 * MB, vscales=POOL + 192 * MB, table=0x10000000,
            lengths=0x11000000, cu_seqlens=0x12000000, pages=100, page=16, table_pages=8, B=2, T=30, Hkv=4, D=64, format=0)
CODE_BYTES, SCALE_BYTES = 100 * 4 * 16 * 64, 4 * 100 * 4


def cache(**kw):
    a = {**BASE, **kw}
    return L.KvPaged(*(a[n] for n, _ in L.KvPaged._fields_))


def split(kw):
    return {k: v for k, v in kw.items() if k in BASE}, {k: v for k, v in kw.items() if k not in BASE}


def append(lib, **kw):
    mine, kw = split(kw)
    a = dict(cache=cache(**mine), k=0x20000000, v=0x21000000, dt=0, ks=256, vs=256, pos=0x22000000, freqs=0x23000000, R=64,
             m=1.0, q=0x24000000, Hq=8, qs=512, qo=0x25000000)
    a.update(kw)
    return lib.w4a16_kv_append_paged(a["cache"], a["k"], a["v"], a["dt"], a["ks"], a["vs"], a["pos"], a["freqs"], a["R"], 0,
                                     a["m"], a["q"], a["Hq"], a["qs"], a["qo"], None)


def read(lib, **kw):
    mine, kw = split(kw)
    a = dict(cache=cache(**mine), dt=0, ko=0x26000000, vo=0x27000000)
    a.update(kw)
    return lib.w4a16_kv_read_paged(a["cache"], a["dt"], a["ko"], a["vo"], None)


def attend(lib, **kw):
    mine, kw = split(kw)
    a = dict(cache=cache(**mine), q=0x24000000, dt=0, Hq=8, qs=512, work=None, out=0x25000000)
    a.update(kw)
    return lib.w4a16_kv_attention_paged(a["cache"], a["q"], a["dt"], a["Hq"], a["qs"], a["work"], a["out"], None)


COMMON = [(dict(cache=None), L.ERR_NULL), (dict(kcodes=None), L.ERR_NULL), (dict(kscales=None), L.ERR_NULL),
          (dict(vcodes=None), L.ERR_NULL), (dict(vscales=None), L.ERR_NULL), (dict(table=None), L.ERR_NULL),
          (dict(lengths=None), L.ERR_NULL), (dict(format=2), L.ERR_SCHEME), (dict(format=-1), L.ERR_SCHEME),
          (dict(page=8), L.ERR_SHAPE), (dict(page=48), L.ERR_SHAPE), (dict(page=256), L.ERR_SHAPE),
          (dict(D=96), L.ERR_SHAPE), (dict(B=0), L.ERR_SHAPE), (dict(B=65536), L.ERR_SHAPE), (dict(T=0), L.ERR_SHAPE),
          (dict(T=(1 << 24) + 1), L.ERR_SHAPE), (dict(Hkv=0), L.ERR_SHAPE), (dict(Hkv=65536), L.ERR_SHAPE),
          (dict(pages=0), L.ERR_SHAPE), (dict(pages=1 << 31), L.ERR_SHAPE), (dict(table_pages=0), L.ERR_SHAPE),
          (dict(table_pages=(1 << 20) + 1), L.ERR_SHAPE), (dict(cu_seqlens=None), L.ERR_SHAPE),
          (dict(T=1 << 23, Hkv=64), L.ERR_SHAPE), (dict(B=65535, Hkv=65), L.ERR_SHAPE),
          (dict(kcodes=POOL + 8), L.ERR_ALIGN), (dict(vcodes=POOL + 4), L.ERR_ALIGN), (dict(kscales=POOL + 2), L.ERR_ALIGN),
          (dict(vscales=POOL + 1), L.ERR_ALIGN), (dict(table=0x10000002), L.ERR_ALIGN),
          (dict(lengths=0x11000001), L.ERR_ALIGN), (dict(cu_seqlens=0x12000002), L.ERR_ALIGN), (dict(dt=2), L.ERR_DTYPE)]


@pytest.mark.parametrize("call", [append, read, attend])
@pytest.mark.parametrize("kw,status", COMMON)
def test_common_refusals(lib, call, kw, status):
    assert call(lib, **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(k=None), L.ERR_NULL), (dict(v=None), L.ERR_NULL), (dict(freqs=None), L.ERR_NULL), (dict(q=None), L.ERR_NULL),
    (dict(qo=None), L.ERR_NULL), (dict(R=63), L.ERR_SHAPE), (dict(R=66), L.ERR_SHAPE), (dict(R=-2), L.ERR_SHAPE),
    (dict(ks=248), L.ERR_SHAPE), (dict(vs=0), L.ERR_SHAPE), (dict(vs=(1 << 24) + 8), L.ERR_SHAPE), (dict(qs=504), L.ERR_SHAPE),
    (dict(Hq=0), L.ERR_SHAPE), (dict(Hq=65536, qs=1 << 24), L.ERR_SHAPE), (dict(k=0x20000008), L.ERR_ALIGN),
    (dict(v=0x21000002), L.ERR_ALIGN), (dict(ks=260), L.ERR_ALIGN), (dict(vs=257), L.ERR_ALIGN), (dict(pos=0x22000002), L.ERR_ALIGN),
    (dict(freqs=0x23000004), L.ERR_ALIGN), (dict(q=0x24000008), L.ERR_ALIGN), (dict(qo=0x25000008), L.ERR_ALIGN),
    (dict(qs=516), L.ERR_ALIGN), (dict(qo=0x24000000), L.ERR_OVERLAP)])
def test_append_refusals(lib, kw, status):
    assert append(lib, **kw) == status


def touching(lo, n, own, step):
    """Addresses from which `own` bytes just reach into the n bytes from lo, at either end."""
    return [(lo - own) // step * step + step, (lo + n - 1) // step * step]


SEQUENCES = [(0x10000000, 4 * 2 * 8), (0x11000000, 8), (0x12000000, 12)]
POOLS = [("kcodes", CODE_BYTES, 16), ("vcodes", CODE_BYTES, 16), ("kscales", SCALE_BYTES, 4), ("vscales", SCALE_BYTES, 4)]


def test_append_overlaps(lib):
    row = 2 * (29 * 256 + 4 * 64)
    spans = SEQUENCES + [(0x20000000, row), (0x21000000, row), (0x22000000, 4 * 30), (0x23000000, 4 * 64),
                         (0x24000000, 2 * 30 * 512)]
    for lo, n in spans:
        for at in touching(lo, n, 2 * 30 * 512, 16):
            assert append(lib, qo=at) == L.ERR_OVERLAP, hex(at)
        for name, size, step in POOLS:
            for at in touching(lo, n, size, step):
                assert append(lib, **{name: at}) == L.ERR_OVERLAP, (name, hex(at))
    for name, size, step in POOLS:
        for at in touching(BASE[name], size, 2 * 30 * 512, 16):
            assert append(lib, qo=at) == L.ERR_OVERLAP
    assert append(lib, vcodes=POOL + CODE_BYTES - 16) == L.ERR_OVERLAP
    assert append(lib, kscales=POOL + CODE_BYTES - 4) == L.ERR_OVERLAP


@pytest.mark.parametrize("kw,status", [(dict(ko=None), L.ERR_NULL), (dict(vo=None), L.ERR_NULL),
                                       (dict(ko=0x26000008), L.ERR_ALIGN), (dict(vo=0x27000002), L.ERR_ALIGN),
                                       (dict(vo=0x26000000), L.ERR_OVERLAP)])
def test_read_refusals(lib, kw, status):
    assert read(lib, **kw) == status


def test_read_overlaps(lib):
    own = 2 * 30 * 4 * 64
    for lo, n in SEQUENCES + [(BASE[name], size) for name, size, _ in POOLS]:
        for at in touching(lo, n, own, 16):
            assert read(lib, ko=at) == L.ERR_OVERLAP and read(lib, vo=at) == L.ERR_OVERLAP


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), L.ERR_NULL), (dict(out=None), L.ERR_NULL), (dict(Hq=6), L.ERR_SHAPE), (dict(Hq=0), L.ERR_SHAPE),
    (dict(Hq=65536, qs=1 << 24), L.ERR_SHAPE), (dict(qs=504), L.ERR_SHAPE), (dict(qs=(1 << 24) + 8), L.ERR_SHAPE),
    (dict(T=1 << 22, Hq=1024, qs=1 << 16), L.ERR_SHAPE),
    (dict(table_pages=1000), L.ERR_NULL), (dict(table_pages=1000, work=0x30000008), L.ERR_ALIGN), (dict(q=0x24000008), L.ERR_ALIGN),
    (dict(out=0x25000004), L.ERR_ALIGN), (dict(qs=516), L.ERR_ALIGN), (dict(out=0x24000000), L.ERR_OVERLAP)])
def test_attention_refusals(lib, kw, status):
    assert attend(lib, **kw) == status


def test_attention_overlaps(lib):
    own = 2 * 30 * 512
    for lo, n in SEQUENCES + [(0x24000000, own)] + [(BASE[name], size) for name, size, _ in POOLS]:
        for at in touching(lo, n, own, 16):
            assert attend(lib, out=at) == L.ERR_OVERLAP
    need = 4 * lib.w4a16_kv_attention_paged_workspace(8, 4, 64, 16000, 1)
    wide = dict(table_pages=1000)
    for lo, n in SEQUENCES[1:] + [(0x10000000, 8000), (0x24000000, own), (0x25000000, own)] + [
            (BASE[name], size) for name, size, _ in POOLS]:
        for at in touching(lo, n, need, 16):
            assert attend(lib, work=at, **wide) == L.ERR_OVERLAP


def test_attention_workspace(lib):
    need = lib.w4a16_kv_attention_paged_workspace
    for chunks in (0, 1):
        assert need(8, 2, 64, 1024, chunks) == 0 and need(8, 2, 64, 1025, chunks) > 0
    assert need(8, 2, 64, 5000, 0) <= need(8, 2, 64, 5000, 1)
    for bad in ((8, 3, 64, 99), (0, 1, 64, 99), (8, 2, 96, 99), (8, 2, 64, 0), (8, 2, 64, (1 << 24) + 1), (65536, 1, 64, 9)):
        assert need(*bad, 1) == L.ERR_SHAPE
    sizes = [need(8, 2, 64, t, 1) for t in range(1, 20000, 37)]
    assert sizes == sorted(sizes)


def rope(lib, **kw):
    a = dict(x=0x20000000, dt=0, T=30, H=4, D=64, xs=512, pos=0x22000000, freqs=0x23000000, R=64, m=1.0, out=0x24000000, os=256)
    a.update(kw)
    return lib.w4a16_rope(a["x"], a["dt"], a["T"], a["H"], a["D"], a["xs"], a["pos"], a["freqs"], a["R"], 0, a["m"], a["out"],
                          a["os"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), L.ERR_NULL), (dict(pos=None), L.ERR_NULL), (dict(freqs=None), L.ERR_NULL), (dict(out=None), L.ERR_NULL),
    (dict(dt=2), L.ERR_DTYPE), (dict(T=0), L.ERR_SHAPE), (dict(T=1 << 24), L.ERR_SHAPE), (dict(H=0), L.ERR_SHAPE),
    (dict(H=65536, xs=1 << 24, os=1 << 24), L.ERR_SHAPE), (dict(D=63, R=62), L.ERR_SHAPE), (dict(D=514, xs=4096, os=4096), L.ERR_SHAPE),
    (dict(R=0), L.ERR_SHAPE), (dict(R=66), L.ERR_SHAPE), (dict(R=31), L.ERR_SHAPE), (dict(xs=255), L.ERR_SHAPE),
    (dict(os=255), L.ERR_SHAPE), (dict(out=0x20000000), L.ERR_SHAPE), (dict(x=0x20000001), L.ERR_ALIGN),
    (dict(out=0x24000001), L.ERR_ALIGN), (dict(pos=0x22000002), L.ERR_ALIGN), (dict(freqs=0x23000004), L.ERR_ALIGN),
    (dict(out=0x20000002), L.ERR_OVERLAP), (dict(out=0x20000000 + 2 * 512 * 29 + 510), L.ERR_OVERLAP),
    (dict(out=0x22000000), L.ERR_OVERLAP), (dict(out=0x23000000 - 2 * 30 * 256 + 2), L.ERR_OVERLAP)])
def test_rope_refusals(lib, kw, status):
    assert rope(lib, **kw) == status


def turns(freqs):
    return [int(w) % 2 ** 64 / 2.0 ** 64 for w in freqs.tolist()]


def test_frequencies():
    f, m = W4.rope_frequencies(64, 10000.0, device="cpu")
    assert f.shape == (32,) and m == 1.0
    assert all(abs(t * 2 * math.pi - 10000.0 ** (-i / 32)) < 1e-15 for i, t in enumerate(turns(f)))
    g, m = W4.rope_frequencies(64, 10000.0, "linear", factor=8.0, device="cpu")
    assert m == 1.0 and all(abs(8 * a - b) < 1e-15 for a, b in zip(turns(g), turns(f)))
    g, _ = W4.rope_frequencies(64, 10000.0, "base", factor=4.0, device="cpu")
    assert turns(g)[0] == turns(f)[0] and abs(4 * turns(g)[-1] / turns(f)[-1] - 1) < 1e-9
    # bands: 1024 positions turn the first pairs more than 4 times, the last less than once
    g, _ = W4.rope_frequencies(64, 10000.0, "bands", factor=8.0, original=1024, device="cpu")
    for a, b in zip(turns(g), turns(f)):
        n = 1024 * b
        keep = min(max((n - 1) / 3, 0), 1)
        assert abs(a - b * (keep + (1 - keep) / 8)) < 1e-15
    assert turns(g)[0] == turns(f)[0] and abs(8 * turns(g)[-1] / turns(f)[-1] - 1) < 1e-9
    # ramp: 32 turns in 4096 positions at index 9.86 of 32, one at 22.5
    g, m = W4.rope_frequencies(64, 10000.0, "ramp", factor=16.0, original=4096, low=1.0, high=32.0, device="cpu")
    lo, hi = (32 * math.log(4096 / (n * 2 * math.pi)) / math.log(10000.0) for n in (32, 1))
    lo, hi = math.floor(lo), math.ceil(hi)
    for i, (a, b) in enumerate(zip(turns(g), turns(f))):
        keep = 1 - min(max((i - lo) / (hi - lo), 0), 1)
        assert abs(a - b * (keep + (1 - keep) / 16)) < 1e-15
    assert abs(m - (0.1 * math.log(16.0) + 1)) < 1e-15
    for bad in (dict(rotary_dim=3), dict(rotary_dim=0), dict(rotary_dim=8, factor=0.0), dict(rotary_dim=8, base=-1.0),
                dict(rotary_dim=8, scaling="other"), dict(rotary_dim=8, scaling="bands"),
                dict(rotary_dim=8, scaling="ramp", original=100, low=2.0, high=1.0)):
        with pytest.raises(ValueError):
            W4.rope_frequencies(device="cpu", **bad)


def test_binding_refuses_host_tensors():
    x, pos = torch.zeros((2, 1, 64), dtype=torch.float16), torch.zeros(2, dtype=torch.int32)
    f, _ = W4.rope_frequencies(64, device="cpu")
    kp, vp = W4.kv_pages(2, 1, 16, 64, device="cpu")
    table, lens = torch.zeros((2, 1), dtype=torch.int32), torch.ones(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        W4.rope(x, pos, f)
    with pytest.raises(ValueError):
        W4.kv_append_paged(x, x, kp, vp, table, lens)
    with pytest.raises(ValueError):
        W4.kv_read_paged(kp, vp, table, lens)
    with pytest.raises(ValueError):
        W4.kv_attention_paged(x, kp, vp, table, lens)
    with pytest.raises(TypeError):
        W4.kv_pages(2, 1, 16, 64, torch.uint8, device="cpu")
    with pytest.raises(ValueError):
        W4.kv_pages(2, 1, 24, 64, device="cpu")
