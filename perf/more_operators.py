"""Cases of the paged 8-bit KV cache's operators, for timing and comparison.

What a serving loop does with a cache whose tokens lie in pages, between the fused projection of
queries, keys and values and the output projection:

``rope``    rotation of heads by their tokens' positions (16 bits in and out);
``append``  new tokens' keys, rotated on the way, and values into the pages, in 8 bits with one scale
            for each page and head, which grows as the page fills; the queries are rotated in the same
            call.  What comes back is the rotated queries and every token of the pages that were
            touched, as the values that the cache then stands for;
``read``    tokens of the pages as 16-bit rows;
``attend``  causal attention of the sequences' last tokens over the pages: one token each in a decode
            step, several in a chunk of a prompt.

A case is a dict of plain values.  ``prepare`` makes its inputs on the GPU, ``run`` is one pass:
with ``own`` false in elementary torch operations in 32 bits (angles in 64), with ``own`` true
through the package's entry points.  ``exact`` computes the same outputs in 64 bits.
"""

import math
import random

import torch

own = False

DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}
CODES = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}
TOP = {"int8": 127.0, "e4m3": 448.0}


# --------------------------------------------------------------------------- cases

def listed():
    return [
        # the queries and keys of a decode step of 16 sequences of a small model: launch latency
        dict(name="rope_step", op="rope", T=16, H=10, D=64, R=64, inter=False, far=4096, base=10000.0, factor=1.0,
             dtype="fp16", mix=1),
        # the prompt of one long document, grouped heads: 32 query and 8 key heads
        dict(name="rope_prompt", op="rope", T=16384, H=40, D=128, R=128, inter=False, far=16384, base=500000.0,
             factor=1.0, dtype="bf16", mix=2),
        # interleaved pairs in part of the head, positions stretched over a long context
        dict(name="rope_part", op="rope", T=5001, H=64, D=128, R=48, inter=True, far=1000000, base=10000.0, factor=8.0,
             dtype="fp16", mix=3),
        # the decode step of a few users of a small model
        dict(name="append_small", op="append", B=4, n=1, past=500, Hq=8, Hkv=2, D=64, page=16, codes="int8", R=64,
             inter=False, dtype="fp16", mix=4),
        # the decode step of a large batch with grouped heads
        dict(name="append_step", op="append", B=128, n=1, past=2048, Hq=32, Hkv=8, D=128, page=64, codes="e4m3", R=128,
             inter=False, dtype="bf16", mix=5),
        # prompts of up to 1024 tokens that arrive together, some behind earlier turns
        dict(name="append_prompts", op="append", B=12, n=1024, past=700, Hq=32, Hkv=32, D=128, page=32, codes="int8",
             R=128, inter=False, dtype="fp16", mix=6),
        # cached conversations taken out of the pages, to be kept elsewhere
        dict(name="read_turns", op="read", B=5, n=100, past=300, Hkv=2, D=64, page=16, codes="int8", dtype="fp16", mix=7),
        # a cached document as 16-bit rows
        dict(name="read_documents", op="read", B=2, n=30001, past=0, Hkv=8, D=128, page=64, codes="e4m3", dtype="bf16",
             mix=8),
        # a decode step of a few users of a small model
        dict(name="attend_small", op="attend", B=4, n=1, past=500, Hq=8, Hkv=2, D=64, page=16, codes="int8",
             dtype="fp16", mix=9),
        # the batched decode step of the 7B-like model, 16 sequences of up to 4096 tokens
        dict(name="attend_batch", op="attend", B=16, n=1, past=4095, Hq=32, Hkv=32, D=128, page=16, codes="int8",
             dtype="fp16", mix=10),
        # long contexts with grouped heads
        dict(name="attend_long", op="attend", B=8, n=1, past=65535, Hq=32, Hkv=8, D=128, page=64, codes="e4m3",
             dtype="bf16", mix=11),
        # a chunk of a long prompt behind what is cached already
        dict(name="attend_chunk", op="attend", B=1, n=2048, past=30000, Hq=32, Hkv=8, D=128, page=64, codes="int8",
             dtype="bf16", mix=12),
    ]


def _log(rng, lo, hi):
    """An integer of [lo, hi], uniform in its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "append", "read", "attend", "attend"])
    mix, dtype = rng.randrange(1 << 30), rng.choice(["fp16", "bf16"])
    Hkv = rng.choice([1, 2, 3, 4, 8])
    Hq = Hkv * rng.choice([1, 2, 3, 4, 6, 8])
    if Hq > 40:
        Hq = Hkv
    if op == "rope":
        D = rng.choice([64, 96, 128, 256])
        T = _log(rng, 1, min(16384, (1 << 26) // (D * (Hq + Hkv))))
        return dict(op=op, T=T, H=Hq + Hkv, D=D, R=rng.choice([D, D, D // 2, D // 4 + 2]), inter=rng.random() < 0.4,
                    far=_log(rng, 100, 1000000), base=rng.choice([10000.0, 500000.0]), factor=rng.choice([1.0, 1.0, 4.0]),
                    dtype=dtype, mix=mix)
    D = rng.choice([64, 128])
    case = dict(op=op, Hkv=Hkv, D=D, page=rng.choice([16, 32, 64, 128]), codes=rng.choice(["int8", "e4m3"]), dtype=dtype,
                mix=mix)
    if op == "read":
        B = _log(rng, 1, 32)
        return dict(case, B=B, n=_log(rng, 1, 32768 // B), past=_log(rng, 1, 1000))
    if op == "append":
        B = _log(rng, 1, 128)
        n = 1 if rng.random() < 0.5 else _log(rng, 2, 8192 // B)
        return dict(case, B=B, n=n, past=_log(rng, 1, 2048), Hq=Hq, R=rng.choice([D, D, D // 2, 0]),
                    inter=rng.random() < 0.3)
    B = _log(rng, 1, 32)
    n = 1 if rng.random() < 0.6 else _log(rng, 2, 1024)
    past = _log(rng, 1, 32768)
    while B > 1 and (B * n * Hq * (past + n) > 1 << 30 or B * (past + n) * Hkv > 1 << 21):
        B //= 2
    return dict(case, B=B, n=n, past=min(past, max(1, (1 << 30) // (n * Hq))), Hq=Hq)


def _lengths(case):
    """Host lists ``(new, total)``: every sequence's new (or last) tokens and all that the pages then
    hold of it.  One sequence takes the whole room, the others are spread below it."""
    rng = random.Random(case["mix"])
    B, n, past = case["B"], case["n"], case["past"]
    low = (past + 3) // 4 if n == 1 else 0
    new = [1 if n == 1 else _log(rng, 1, n) for _ in range(B)]
    old = [rng.randint(low, past) for _ in range(B)]
    top = rng.randrange(B)
    new[top], old[top] = n, past
    return new, [a + b for a, b in zip(new, old)]


def _read_counts(case):
    """How many of each sequence's last tokens a pass reads back: behind an append those of every page
    that it touched."""
    new, total = _lengths(case)
    if case["op"] == "read":
        return new
    return [t - (t - n) // case["page"] * case["page"] for n, t in zip(new, total)]


def work(case):
    D = case["D"]
    if case["op"] == "rope":
        rows = case["T"] * case["H"]
        return {"bytes": 4 * rows * D + 4 * case["T"], "flops": 3 * rows * case["R"]}
    Hkv, page = case["Hkv"], case["page"]
    new, total = _lengths(case)
    if case["op"] == "attend":
        pairs = sum(n * t - n * (n - 1) // 2 for n, t in zip(new, total))
        pages = sum(-(-t // page) for t in total)
        return {"bytes": 2 * Hkv * D * sum(total) + pages * (8 * Hkv + 4) + 4 * sum(new) * case["Hq"] * D,
                "flops": 4 * case["Hq"] * D * pairs}
    back = sum(_read_counts(case))
    moved = 2 * Hkv * D * back * 3                  # a code read, a 16-bit value written, K and V
    if case["op"] == "append":
        T = sum(new)
        moved += 2 * Hkv * D * T * 3 + 4 * T * case["Hq"] * D
        return {"bytes": moved, "flops": T * D * (6 * Hkv + 3 * case["Hq"]) + 2 * Hkv * D * back}
    return {"bytes": moved, "flops": 2 * Hkv * D * back}


# --------------------------------------------------------------------------- inputs

def _frequencies(R, base, factor=1.0):
    """Angle per position of each of R / 2 pairs, 64 bits, positions divided by ``factor``."""
    return [base ** (-2.0 * i / R) / factor for i in range(R // 2)]


def _phases(freqs):
    """The same as 64-bit fractions of a turn, what the package's rotations take."""
    words = [round(f / (2 * math.pi) * 2 ** 64) % 2 ** 64 for f in freqs]
    return [w - 2 ** 64 if w >= 2 ** 63 else w for w in words]


def _pool(g, case, total):
    """Pages of normal rows in 8 bits, one scale a page and head, and every sequence's table of them in
    random order (-1 behind a sequence's pages).  The last page belongs to no sequence."""
    Hkv, D, page = case["Hkv"], case["D"], case["page"]
    counts = [-(-t // page) for t in total]
    N = sum(counts) + 3
    order = torch.randperm(N - 1, generator=g, device="cuda").to(torch.int32).cpu()
    table = torch.full((len(total), max(counts) + 2), -1, dtype=torch.int32)
    at = 0
    for b, c in enumerate(counts):
        table[b, :c] = order[at:at + c]
        at += c

    def pages(shape, outliers):
        x = torch.randn(shape, generator=g, device="cuda")
        if outliers:
            x = torch.where(torch.rand(shape, generator=g, device="cuda") < 0.02, x * 8.0, x)
        x = x.to(DTYPES[case["dtype"]]).float()
        s = x.abs().amax((2, 3)) / TOP[case["codes"]]
        x /= s[..., None, None]
        return x.round_().to(torch.int8) if case["codes"] == "int8" else x.clamp_(-448, 448).to(CODES["e4m3"]), s
    k, v = pages((N, Hkv, page, D), True), pages((N, Hkv, D, page), False)
    return k, v, table.cuda()


def _starts(counts):
    cu = [0]
    for n in counts:
        cu.append(cu[-1] + n)
    return torch.tensor(cu, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op, D, dt = case["op"], case["D"], DTYPES[case["dtype"]]
    st = dict(case=case)
    if op == "rope":
        # the heads to rotate are a column block of one fused projection's output
        T, H = case["T"], case["H"]
        wide = torch.randn((T, (H + 8) * D), generator=g, device="cuda").to(dt)
        st["x"] = wide[:, :H * D].unflatten(1, (H, D))
        st["positions"] = torch.randint(0, case["far"], (T,), generator=g, device="cuda").to(torch.int32)
        freqs = _frequencies(case["R"], case["base"], case["factor"])
        st["freqs"] = torch.tensor(freqs, dtype=torch.float64, device="cuda")
        st["phases"] = torch.tensor(_phases(freqs), dtype=torch.int64, device="cuda")
        st["scale"] = 1.0 if case["factor"] == 1.0 else 0.1 * math.log(case["factor"]) + 1.0
        st["out"] = torch.empty((T, H, D), dtype=dt, device="cuda")
        return st
    new, total = _lengths(case)
    st["new"], st["total"] = new, total
    st["k"], st["v"], st["table"] = _pool(g, case, total)
    st["lengths"] = torch.tensor(total, dtype=torch.int32, device="cuda")
    T, Hkv = sum(new), case["Hkv"]
    st["cu"] = None if op != "read" and case["n"] == 1 else _starts(new)
    if op == "read":
        st["kout"], st["vout"] = (torch.empty((T, Hkv, D), dtype=dt, device="cuda") for _ in range(2))
        return st
    Hq = case["Hq"]
    if op == "attend":
        st["q"] = (torch.randn((T, Hq, D), generator=g, device="cuda") * 1.2).to(dt)
        st["out"] = torch.empty((T, Hq, D), dtype=dt, device="cuda")
        return st
    qkv = torch.randn((T, (Hq + 2 * Hkv) * D), generator=g, device="cuda").to(dt)
    st["q_new"] = qkv[:, :Hq * D].unflatten(1, (Hq, D))
    st["k_new"] = qkv[:, Hq * D:(Hq + Hkv) * D].unflatten(1, (Hkv, D))
    st["v_new"] = qkv[:, (Hq + Hkv) * D:].unflatten(1, (Hkv, D))
    if case["R"]:
        freqs = _frequencies(case["R"], 10000.0)
        st["freqs"] = torch.tensor(freqs, dtype=torch.float64, device="cuda")
        st["phases"] = torch.tensor(_phases(freqs), dtype=torch.int64, device="cuda")
    st["scale"] = 1.0
    back = _read_counts(case)
    st["back"], st["cu_back"] = back, _starts(back)
    st["q_out"] = torch.empty((T, Hq, D), dtype=dt, device="cuda")
    st["kout"], st["vout"] = (torch.empty((sum(back), Hkv, D), dtype=dt, device="cuda") for _ in range(2))
    return st


# --------------------------------------------------------------------------- the passes

def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(st):
    import w4a16_dequant_gemm_amd as W4
    case = st["case"]
    op = case["op"]
    if op == "rope":
        return W4.rope(st["x"], st["positions"], st["phases"], interleaved=case["inter"], mscale=st["scale"], out=st["out"])
    if op == "attend":
        return W4.kv_attention_paged(st["q"], st["k"], st["v"], st["table"], st["lengths"], st["cu"], out=st["out"])
    if op == "read":
        return W4.kv_read_paged(st["k"], st["v"], st["table"], st["lengths"], st["cu"], out=(st["kout"], st["vout"]))
    if case["R"]:
        q = W4.kv_append_paged(st["k_new"], st["v_new"], st["k"], st["v"], st["table"], st["lengths"], st["cu"],
                               freqs=st["phases"], interleaved=case["inter"], q=st["q_new"], q_out=st["q_out"])
    else:
        W4.kv_append_paged(st["k_new"], st["v_new"], st["k"], st["v"], st["table"], st["lengths"], st["cu"])
        q = st["q_new"]
    k, v = W4.kv_read_paged(st["k"], st["v"], st["table"], st["lengths"], st["cu_back"], out=(st["kout"], st["vout"]))
    return q, k, v


def _rotate(x, positions, st):
    """``x [T, H, D]`` in 32 bits with its first R values rotated in pairs by position times frequency."""
    case = st["case"]
    R = case["R"]
    if not R:
        return x
    a = positions.double()[:, None, None] * st["freqs"]
    c, s = (torch.cos(a) * st["scale"]).float(), (torch.sin(a) * st["scale"]).float()
    if case["inter"]:
        x0, x1 = x[..., 0:R:2], x[..., 1:R:2]
        turned = torch.stack([x0 * c - x1 * s, x1 * c + x0 * s], -1).flatten(-2)
    else:
        x0, x1 = x[..., :R // 2], x[..., R // 2:R]
        turned = torch.cat([x0 * c - x1 * s, x1 * c + x0 * s], -1)
    return torch.cat([turned, x[..., R:]], -1)


def _floats(codes, index):
    """Pages of a pool as 32-bit values of their codes (8-bit floats are indexed as bytes)."""
    return codes.view(torch.uint8)[index].view(codes.dtype).float()


def _places(cu, lengths, T):
    """Of T packed tokens, the sequence and the place in it of each: the last ones of every sequence."""
    if cu is None:
        seq = torch.arange(T, device="cuda")
        return seq, lengths.long() - 1
    i = torch.arange(T, device="cuda")
    seq = torch.searchsorted(cu[1:].contiguous(), i, right=True)
    return seq, lengths[seq].long() - cu[seq + 1] + i


def _run_plain(st):
    case = st["case"]
    op, page, dt = case["op"], case.get("page"), DTYPES[case["dtype"]]
    if op == "rope":
        return _rotate(st["x"].float(), st["positions"], st).to(dt)
    if op == "attend":
        return _plain_attend(st)
    if op == "read":
        return _plain_read(st, st["cu"], st["kout"].shape[0])
    T = st["k_new"].shape[0]
    seq, pos = _places(st["cu"], st["lengths"], T)
    q = _rotate(st["q_new"].float(), pos, st).to(dt)
    _plain_append(st, st["k"], _rotate(st["k_new"].float(), pos, st), False)
    _plain_append(st, st["v"], st["v_new"].float(), True)
    return (q,) + _plain_read(st, st["cu_back"], st["kout"].shape[0])


def _plain_append(st, cache, x, across):
    """New rows ``x [T, Hkv, D]`` into the pages, which hold rows (K) or, ``across``, columns (V)."""
    case, (codes, scales) = st["case"], cache
    page, top, whole = case["page"], TOP[case["codes"]], case["codes"] == "int8"
    lengths = st["lengths"].long()
    B = lengths.shape[0]
    new = torch.ones_like(lengths) if st["cu"] is None else (st["cu"][1:] - st["cu"][:-1]).long()
    first = torch.arange(B, device="cuda") if st["cu"] is None else st["cu"][:-1].long()
    before = lengths - new
    M = max((t - 1) // page - (t - n) // page + 1 for n, t in zip(st["new"], st["total"]))
    m = before[:, None] // page + torch.arange(M, device="cuda")             # touched pages of each sequence
    live = m * page < lengths[:, None]
    spare = codes.shape[0] - 1
    ids = torch.where(live, torch.gather(st["table"].long(), 1, torch.where(live, m, 0)), spare)
    pos = m[..., None] * page + torch.arange(page, device="cuda")            # [B, M, page]
    fresh = (pos >= before[:, None, None]) & (pos < lengths[:, None, None])
    token = torch.where(fresh, first[:, None, None] + pos - before[:, None, None], 0)
    rows = torch.where(fresh[..., None, None], x[token], torch.zeros((), device="cuda"))    # [B, M, page, Hkv, D]
    rows = rows.permute(0, 1, 3, 4, 2) if across else rows.permute(0, 1, 3, 2, 4)
    kept = (m * page < before[:, None])[..., None]                           # pages with earlier tokens
    old = scales[ids]
    s = torch.maximum(torch.where(kept, old, torch.zeros_like(old)), rows.abs().amax((-1, -2)) / top)
    c = _floats(codes, ids)
    again = c * (old / torch.where(s > 0, s, torch.ones_like(s)))[..., None, None]
    u = rows / torch.where(s > 0, s, torch.ones_like(s))[..., None, None]
    if whole:
        again, u = again.round(), u.round()
    again = torch.where((s > old)[..., None, None], again, c)
    fresh, kept = fresh[:, :, None, :], (kept & (pos < before[:, None, None]))[:, :, None, :]
    fresh, kept = (t[..., None, :] if across else t[..., None] for t in (fresh, kept))
    c = torch.where(fresh, u.clamp(-top, top), torch.where(kept, again.clamp(-top, top), c))
    codes.view(torch.uint8)[ids] = c.to(codes.dtype).view(torch.uint8)
    scales[ids] = s


def _plain_read(st, cu, T):
    page, dt = st["case"]["page"], DTYPES[st["case"]["dtype"]]
    seq, pos = _places(cu, st["lengths"], T)
    ids, slot = st["table"][seq, pos // page].long(), pos % page
    (kc, ks), (vc, vs) = st["k"], st["v"]
    k = kc.view(torch.uint8)[ids, :, slot].view(kc.dtype).float() * ks[ids][..., None]
    v = vc.view(torch.uint8)[ids, :, :, slot].view(vc.dtype).float() * vs[ids][..., None]
    return k.to(dt), v.to(dt)


def _plain_attend(st):
    case = st["case"]
    B, Hq, Hkv, D, n = case["B"], case["Hq"], case["Hkv"], case["D"], case["n"]
    G = Hq // Hkv
    ids = st["table"].long().clamp(min=0)
    (kc, ks), (vc, vs) = st["k"], st["v"]
    K = (_floats(kc, ids) * ks[ids][..., None, None]).transpose(1, 2).reshape(B, Hkv, -1, D)
    V = (_floats(vc, ids) * vs[ids][..., None, None]).permute(0, 2, 1, 4, 3).reshape(B, Hkv, -1, D)
    i = torch.arange(n, device="cuda")
    first = torch.arange(B, device="cuda") if st["cu"] is None else st["cu"][:-1].long()
    new = torch.ones_like(first) if st["cu"] is None else (st["cu"][1:] - st["cu"][:-1]).long()
    row = torch.where(i < new[:, None], first[:, None] + i, 0)                               # [B, n]
    q = (st["q"][row].float() / math.sqrt(D)).view(B, n, Hkv, G, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * n, D)
    sc = torch.matmul(q, K.transpose(2, 3)).view(B, Hkv, G, n, -1)
    last = (st["lengths"].long() - new)[:, None] + i                                         # a row's own token
    hidden = torch.arange(K.shape[2], device="cuda") > last[..., None]
    sc = sc.masked_fill_(hidden[:, None, None], -math.inf)
    m = sc.amax(-1, keepdim=True)
    e = sc.sub_(torch.where(m == -math.inf, torch.zeros_like(m), m)).exp_()
    o = torch.matmul(e.view(B, Hkv, G * n, -1), V).view(B, Hkv, G, n, D) / e.sum(-1, keepdim=True)
    o = o.permute(0, 3, 1, 2, 4).reshape(B * n, Hq, D)
    seq, pos = _places(st["cu"], st["lengths"], st["q"].shape[0])
    return o[seq * n + pos - (st["lengths"].long() - new)[seq]].to(st["q"].dtype)


# --------------------------------------------------------------------------- 64 bits

def _turned(x, place, case, freqs, scale):
    """Rotation of ``x [n, H, D]`` (64 bits) by complex multiplication."""
    R = case["R"]
    if not R:
        return x
    part = x[..., :R].unflatten(-1, (R // 2, 2)) if case["inter"] else x[..., :R].unflatten(-1, (2, R // 2)).transpose(-1, -2)
    angle = (place.double().unsqueeze(-1) * torch.tensor(freqs, dtype=torch.float64, device="cuda")).unsqueeze(1)
    z = torch.complex(part[..., 0].contiguous(), part[..., 1].contiguous()) * torch.polar(torch.full_like(angle, scale), angle)
    y = torch.view_as_real(z)
    y = y if case["inter"] else y.transpose(-1, -2)
    return torch.cat([y.flatten(-2), x[..., R:]], -1)


def _nearest_code(x, codes):
    """The codes nearest to 64-bit values, ties to even: whole numbers, or three bits behind the
    leading one down to 2^-9."""
    if codes == "int8":
        return torch.round(x).clamp(-127, 127)
    e = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6)))
    step = torch.exp2(e - 3)
    return (torch.round(x / step) * step).clamp(-448, 448)


def exact(case, seed):
    st = prepare(case, seed)
    op, D = case["op"], case["D"]
    if op == "rope":
        freqs = _frequencies(case["R"], case["base"], case["factor"])
        return _turned(st["x"].double(), st["positions"], case, freqs, st["scale"])
    page, Hkv = case["page"], case["Hkv"]
    table = st["table"].cpu().tolist()
    (kc, ks), (vc, vs) = st["k"], st["v"]

    def held(b, first, last):
        """Tokens first .. last - 1 of sequence b, K and V [tokens, Hkv, D]."""
        at = torch.tensor(table[b][first // page:(last + page - 1) // page], device="cuda")
        kk = kc.view(torch.int8)[at].view(kc.dtype).to(torch.float32).double() * ks[at].double()[:, :, None, None]
        vv = vc.view(torch.int8)[at].view(vc.dtype).to(torch.float32).double() * vs[at].double()[:, :, None, None]
        kk, vv = kk.transpose(1, 2).reshape(-1, Hkv, D), vv.permute(0, 3, 1, 2).reshape(-1, Hkv, D)
        cut = first // page * page
        return kk[first - cut:last - cut], vv[first - cut:last - cut]
    if op == "read":
        parts = [held(b, t - n, t) for b, (n, t) in enumerate(zip(st["new"], st["total"]))]
        return torch.cat([p[0] for p in parts]), torch.cat([p[1] for p in parts])
    at = 0
    if op == "attend":
        G = case["Hq"] // Hkv
        out = torch.zeros(st["out"].shape, dtype=torch.float64, device="cuda")
        for b, (n, t) in enumerate(zip(st["new"], st["total"])):
            kk, vv = held(b, 0, t)
            for h in range(case["Hq"]):
                s = (st["q"][at:at + n, h].double() @ kk[:, h // G].t()) * D ** -0.5
                own_place = torch.arange(t - n, t, device="cuda").unsqueeze(1)
                s[torch.arange(t, device="cuda") > own_place] = -math.inf
                out[at:at + n, h] = torch.softmax(s, 1) @ vv[:, h // G]
            at += n
        return out
    top = TOP[case["codes"]]
    freqs = _frequencies(case["R"], 10000.0)
    qs, krows, vrows = [], [], []
    for b, (n, t) in enumerate(zip(st["new"], st["total"])):
        place = torch.arange(t - n, t, device="cuda")
        take = slice(at, at + n)
        qs.append(_turned(st["q_new"][take].double(), place, case, freqs, 1.0))
        fresh = (_turned(st["k_new"][take].double(), place, case, freqs, 1.0), st["v_new"][take].double())
        for p in range((t - n) // page, (t - 1) // page + 1):
            lo, hi = max(p * page, t - n), min((p + 1) * page, t)
            for rows, into, (codes, scales), axis in ((fresh[0], krows, st["k"], 1), (fresh[1], vrows, st["v"], 2)):
                x = rows[lo - (t - n):hi - (t - n)]                         # [tokens, Hkv, D]
                s = x.abs().amax((0, 2)) / top
                kept = None
                if lo > p * page:
                    before = scales[table[b][p]].double()
                    kept = codes[table[b][p]].to(torch.float32).double().narrow(axis, 0, lo - p * page)
                    kept = kept.transpose(0, 1) if axis == 1 else kept.permute(2, 0, 1)
                    s = torch.maximum(s, before)
                    grown = (s > before).unsqueeze(-1)
                    kept = torch.where(grown, _nearest_code(kept * (before / s).unsqueeze(-1), case["codes"]), kept)
                c = _nearest_code(x / s.unsqueeze(-1), case["codes"])
                into.append((c if kept is None else torch.cat([kept, c])) * s.unsqueeze(-1))
        at += n
    return torch.cat(qs), torch.cat(krows), torch.cat(vrows)
