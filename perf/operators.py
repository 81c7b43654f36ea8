"""Cases of the attention operators around the quantized KV cache, for timing and comparison.

Four operators that one serving loop calls in turn:

``prompt``   causal attention over packed prompts (16-bit keys and values, before they are
             quantized into the cache);
``shared``   decode attention of a batch whose sequences share one quantized prefix and own a
             quantized suffix each;
``weights``  decode attention over the quantized cache that also adds up the attention weight
             every cached token receives;
``evict``    compaction of a quantized cache to a budget: the most recent tokens and those with
             the largest accumulated weight.

A case is a dict of plain values.  ``prepare`` makes its inputs on the GPU, ``run`` is one pass:
with ``own`` false in elementary torch operations in 32 bits, with ``own`` true through the
package's entry points.  ``exact`` computes the same outputs in 64 bits.
"""

import math
import random

import torch

own = False

DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}


# --------------------------------------------------------------------------- cases

def listed():
    return [
        # a handful of short chat turns of a small model arriving together: launch latency
        dict(name="prompt_turns", op="prompt", B=6, longest=96, Hq=8, Hkv=2, D=64, dtype="fp16", pad=5, mix=1),
        # packed prompts of the 7B-like model, lengths from a few tokens to 1024
        dict(name="prompt_packed", op="prompt", B=12, longest=1024, Hq=32, Hkv=32, D=128, dtype="fp16", pad=0, mix=2),
        # one long document with grouped heads
        dict(name="prompt_long", op="prompt", B=1, longest=16384, Hq=32, Hkv=8, D=128, dtype="bf16", pad=0, mix=3),
        # a few users of a small model behind a short system prompt
        dict(name="shared_small", op="shared", B=4, Hq=8, Hkv=2, D=64, P=333, Tmax=64, bits=8, dtype="fp16", mix=4),
        # a batch behind a system prompt with tools and examples
        dict(name="shared_batch", op="shared", B=32, Hq=32, Hkv=8, D=128, P=4096, Tmax=512, bits=8, dtype="bf16",
             mix=5),
        # many questions on one long document, 4-bit cache
        dict(name="shared_document", op="shared", B=128, Hq=32, Hkv=8, D=128, P=32768, Tmax=1024, bits=4,
             dtype="fp16", mix=6),
        # one conversation of a few hundred tokens
        dict(name="weights_single", op="weights", B=1, Hq=8, Hkv=2, D=64, Tmax=500, bits=8, dtype="bf16", mix=7),
        # the batched decode step of the 7B-like model, 16 sequences up to 4096 tokens
        dict(name="weights_batch", op="weights", B=16, Hq=32, Hkv=32, D=128, Tmax=4096, bits=8, dtype="fp16", mix=8),
        # long contexts with grouped heads and a 4-bit cache
        dict(name="weights_long", op="weights", B=8, Hq=32, Hkv=8, D=128, Tmax=65536, bits=4, dtype="bf16", mix=9),
        # a small cache that just overran its budget
        dict(name="evict_small", op="evict", B=2, Hkv=2, D=64, Tmax=300, budget=128, recent=32, bits=8, mix=10),
        # the batched decode cache halved
        dict(name="evict_batch", op="evict", B=16, Hkv=32, D=128, Tmax=4096, budget=2048, recent=256, bits=8, mix=11),
        # one very long context cut to a sixth
        dict(name="evict_long", op="evict", B=1, Hkv=8, D=128, Tmax=100001, budget=16384, recent=1024, bits=4,
             mix=12),
    ]


def _log(rng, lo, hi):
    """An integer of [lo, hi], uniform in its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["prompt", "shared", "weights", "evict"])
    D = rng.choice([64, 128])
    bits = rng.choice([8, 4])
    dtype = rng.choice(["fp16", "bf16"])
    Hkv = rng.choice([1, 2, 3, 4, 8])
    Hq = Hkv * rng.choice([1, 2, 3, 4, 6, 8])
    if Hq > 32:
        Hq = Hkv
    mix = rng.randrange(1 << 30)
    if op == "prompt":
        return dict(op=op, B=_log(rng, 1, 48), longest=_log(rng, 1, 8192), Hq=Hq, Hkv=Hkv, D=D, dtype=dtype,
                    pad=rng.choice([0, 0, 1, 17]), mix=mix)
    if op == "shared":
        return dict(op=op, B=_log(rng, 1, 128), Hq=Hq, Hkv=Hkv, D=D, P=_log(rng, 1, 32768), Tmax=_log(rng, 1, 1024),
                    bits=bits, dtype=dtype, mix=mix)
    if op == "weights":
        return dict(op=op, B=_log(rng, 1, 16), Hq=Hq, Hkv=Hkv, D=D, Tmax=_log(rng, 1, 32768), bits=bits, dtype=dtype,
                    mix=mix)
    Tmax = _log(rng, 2, 100001)
    budget = _log(rng, 1, Tmax)
    return dict(op=op, B=_log(rng, 1, 8), Hkv=Hkv, D=D, Tmax=Tmax, budget=budget, recent=rng.randint(0, budget),
                bits=bits, mix=mix)


def _lengths(case):
    """The lengths of the case's sequences (host list): one takes the whole room, the others are
    spread below it.  Suffixes may be empty; a cache of the other operators holds a token."""
    rng = random.Random(case["mix"])
    B, op = case["B"], case["op"]
    if op == "prompt":
        out = [_log(rng, 1, case["longest"]) for _ in range(B)]
        out[rng.randrange(B)] = case["longest"]
        return out
    top = case["Tmax"]
    low = {"shared": 0, "weights": (top + 3) // 4, "evict": min(top, max(1, case.get("budget", 1) // 2))}[op]
    out = [rng.randint(low, top) for _ in range(B)]
    out[rng.randrange(B)] = top
    return out


def work(case):
    op, D = case["op"], case["D"]
    lens = _lengths(case)
    total = sum(lens)
    if op == "prompt":
        Hq, Hkv = case["Hq"], case["Hkv"]
        pairs = sum(n * (n + 1) // 2 for n in lens)
        return {"bytes": 2 * total * D * (2 * Hq + 2 * Hkv), "flops": 4 * Hq * D * pairs}
    per = D + 2 if case["bits"] == 8 else D // 2 + 4          # one cached row: codes, scale (and zero point)
    if op == "shared":
        B, Hq, Hkv, P = case["B"], case["Hq"], case["Hkv"], case["P"]
        return {"bytes": 2 * Hkv * (P + total) * per + 4 * B * Hq * D + 4 * B,
                "flops": 4 * Hq * D * (B * P + total)}
    if op == "weights":
        B, Hq, Hkv = case["B"], case["Hq"], case["Hkv"]
        return {"bytes": 2 * Hkv * total * per + 8 * Hkv * total + 4 * B * Hq * D + 4 * B,
                "flops": 4 * Hq * D * total + Hq * total}
    # evict: every weight is read; a kept row's codes, parameters, weight and index are written
    B, Hkv, budget = case["B"], case["Hkv"], case["budget"]
    kept = sum(min(n, budget) for n in lens)
    return {"bytes": Hkv * (4 * total + kept * (4 * per + 8)) + 8 * B, "flops": Hkv * total}


# --------------------------------------------------------------------------- inputs

def _quantize(x, bits):
    """Per-row KV8 / KV4 quantization of ``x [..., D]`` (fp32): ``(codes, scales, zeros)``."""
    if bits == 8:
        s = (x.abs().amax(-1) / 127.0).half()
        s = torch.where(s == 0, torch.ones_like(s), s)
        return torch.round(x / s.float()[..., None]).clamp_(-127, 127).to(torch.int8), s, None
    mn, mx = x.amin(-1), x.amax(-1)
    s = ((mx - mn) / 15.0).half()
    s = torch.where(s == 0, torch.ones_like(s), s)
    z = torch.round(-mn / s.float()) + 0.0
    u = (torch.round(x / s.float()[..., None]) + z[..., None]).clamp_(0, 15).to(torch.int32)
    u = u.reshape(*u.shape[:-1], -1, 8)
    words = u[..., 0].clone()
    for i in range(1, 8):
        words |= u[..., i] << (4 * i)
    return words, s, z.half()


def _cache(g, shape, bits, dtype, outliers):
    """A quantized cache of normal rows, a few entries eight times as large if ``outliers``."""
    x = torch.randn(shape, generator=g, device="cuda")
    if outliers:
        x = torch.where(torch.rand(shape, generator=g, device="cuda") < 0.02, x * 8.0, x)
    return _quantize(x.to(DTYPES[dtype]).float(), bits)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op, D, B = case["op"], case["D"], case["B"]
    lens = _lengths(case)
    st = dict(case=case, lens=lens)
    if op == "prompt":
        Hq, Hkv, T = case["Hq"], case["Hkv"], sum(lens) + case["pad"]
        # q, k and v are the column blocks of one fused projection's output
        qkv = torch.randn((T, (Hq + 2 * Hkv) * D), generator=g, device="cuda").to(DTYPES[case["dtype"]])
        st["q"] = qkv[:, :Hq * D].unflatten(1, (Hq, D))
        st["k"] = qkv[:, Hq * D:(Hq + Hkv) * D].unflatten(1, (Hkv, D))
        st["v"] = qkv[:, (Hq + Hkv) * D:].unflatten(1, (Hkv, D))
        cu = [0]
        for n in lens:
            cu.append(cu[-1] + n)
        st["cu"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
        st["out"] = torch.zeros((T, Hq, D), dtype=qkv.dtype, device="cuda")   # rows behind the last prompt stay 0
        return st
    st["lengths"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    Hkv, Tmax, bits = case["Hkv"], case["Tmax"], case["bits"]
    if op == "evict":
        shape = (B, Hkv, Tmax)
        Tout = min(case["budget"], Tmax)
        caches = []
        for _ in range(2):
            if bits == 8:
                codes = torch.randint(-127, 128, shape + (D,), generator=g, device="cuda", dtype=torch.int8)
                zeros = None
            else:
                codes = torch.randint(-(1 << 31), 1 << 31, shape + (D // 8,), generator=g, device="cuda",
                                      dtype=torch.int64).to(torch.int32)
                zeros = torch.randint(0, 16, shape, generator=g, device="cuda").half()
            scales = (torch.randn(shape, generator=g, device="cuda") * 0.3 - 3.5).exp().half()
            caches.append((codes, scales, zeros))
        st["k"], st["v"] = caches
        # accumulated softmax weight: a few tokens hold most of it, some hold none at all
        w = (torch.randn(shape, generator=g, device="cuda") * 2.0 - 4.0).exp()
        st["weights"] = torch.where(torch.rand(shape, generator=g, device="cuda") < 0.03, torch.zeros_like(w), w)

        def room(c):
            return tuple(None if t is None else torch.zeros((B, Hkv, Tout) + t.shape[3:], dtype=t.dtype, device="cuda")
                         for t in c)
        st["out"] = (room(st["k"]), room(st["v"]), torch.zeros((B, Hkv, Tout), device="cuda"),
                     torch.zeros(B, dtype=torch.int32, device="cuda"),
                     torch.zeros((B, Hkv, case["budget"]), dtype=torch.int32, device="cuda"))
        return st
    Hq, dtype = case["Hq"], case["dtype"]
    st["q"] = (torch.randn((B, Hq, D), generator=g, device="cuda") * 1.5).to(DTYPES[dtype])
    st["k"] = _cache(g, (B, Hkv, Tmax, D), bits, dtype, True)
    st["v"] = _cache(g, (B, Hkv, Tmax, D), bits, dtype, False)
    st["out"] = torch.empty((B, Hq, D), dtype=DTYPES[dtype], device="cuda")
    if op == "shared":
        st["kp"] = _cache(g, (Hkv, case["P"], D), bits, dtype, True)
        st["vp"] = _cache(g, (Hkv, case["P"], D), bits, dtype, False)
    else:
        st["weights"] = torch.rand((B, Hkv, Tmax), generator=g, device="cuda") * 0.5
        st["sums"] = torch.zeros((B, Hkv, Tmax), device="cuda")      # entries behind a sequence stay 0
    return st


# --------------------------------------------------------------------------- the passes

def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(st):
    import w4a16_dequant_gemm_amd as W4
    case = st["case"]
    op = case["op"]
    if op == "prompt":
        return W4.attention_prompt(st["q"], st["k"], st["v"], st["cu"], out=st["out"])
    if op == "shared":
        return W4.kv_attention_decode_shared(st["q"], st["kp"], st["vp"], case["P"], st["k"], st["v"], st["lengths"],
                                             case["bits"], out=st["out"])
    if op == "weights":
        return W4.kv_attention_decode_weights(st["q"], st["k"], st["v"], st["lengths"], st["weights"], case["bits"],
                                              sums=st["sums"], out=st["out"])
    k, v, w, n, kept = W4.kv_evict(st["k"], st["v"], st["weights"], st["lengths"], case["budget"], case["recent"],
                                   case["bits"], out=st["out"])
    return [t for t in (*k, *v, w, n, kept) if t is not None]


def _dequantize(cache, bits):
    codes, s, z = cache
    if bits == 8:
        return codes.float() * s.float()[..., None]
    u = torch.stack([(codes >> (4 * i)) & 15 for i in range(8)], -1).flatten(-2)
    return (u.float() - z.float()[..., None]) * s.float()[..., None]


def _softmax_parts(sc):
    """Row maxima, exponentials and their sums of scores whose hidden entries are -inf; a row
    with nothing to attend to gets zeros."""
    m = sc.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    e = torch.exp(sc - m)
    return m, e, e.sum(-1, keepdim=True)


def _run_plain(st):
    case = st["case"]
    op = case["op"]
    if op == "prompt":
        return _plain_prompt(st)
    if op == "evict":
        return _plain_evict(st)
    B, Hq, Hkv, D, Tmax, bits = case["B"], case["Hq"], case["Hkv"], case["D"], case["Tmax"], case["bits"]
    G = Hq // Hkv
    q = st["q"].float() / math.sqrt(D)
    K, V = _dequantize(st["k"], bits), _dequantize(st["v"], bits)
    sc = torch.matmul(q.view(B, Hkv, G, D), K.transpose(2, 3))                     # [B, Hkv, G, Tmax]
    seen = torch.arange(Tmax, device="cuda")[None, :] < st["lengths"][:, None]
    sc = sc.masked_fill(~seen[:, None, None, :], -math.inf)
    if op == "shared":
        P = case["P"]
        Kp, Vp = _dequantize(st["kp"], bits), _dequantize(st["vp"], bits)
        qh = q.view(B, Hkv, G, D).transpose(0, 1).reshape(Hkv, B * G, D)
        sp = torch.matmul(qh, Kp.transpose(1, 2)).view(Hkv, B, G, P).transpose(0, 1)
        _, e, l = _softmax_parts(torch.cat([sp, sc], -1))
        ep = e[..., :P].transpose(0, 1).reshape(Hkv, B * G, P)
        o = torch.matmul(ep, Vp).view(Hkv, B, G, D).transpose(0, 1) + torch.matmul(e[..., P:], V)
        return (o / l).reshape(B, Hq, D).to(st["q"].dtype)
    _, e, l = _softmax_parts(sc)
    p = e / l
    out = torch.matmul(p, V).reshape(B, Hq, D).to(st["q"].dtype)
    sums = torch.where(seen[:, None, :], st["weights"] + p.sum(2), torch.zeros_like(st["weights"]))
    return out, sums


def _plain_prompt(st):
    case = st["case"]
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    G = Hq // Hkv
    out = torch.zeros_like(st["out"])
    at = 0
    for n in st["lens"]:
        k, v = st["k"][at:at + n].float(), st["v"][at:at + n].float()
        q = st["q"][at:at + n].float() / math.sqrt(D)
        hidden = torch.ones((n, n), dtype=torch.bool, device="cuda").triu_(1)
        for h in range(Hkv):                                   # one kv head's scores at a time: [G, n, n]
            sc = torch.matmul(q[:, h * G:(h + 1) * G].transpose(0, 1), k[:, h].t())
            _, e, l = _softmax_parts(sc.masked_fill_(hidden, -math.inf))
            out[at:at + n, h * G:(h + 1) * G] = (torch.matmul(e, v[:, h]) / l).transpose(0, 1).to(out.dtype)
        at += n
    return out


def _plain_evict(st):
    case = st["case"]
    B, Hkv, Tmax, budget, recent = case["B"], case["Hkv"], case["Tmax"], case["budget"], case["recent"]
    Tout = min(budget, Tmax)
    n = st["lengths"].long()[:, None, None]
    t = torch.arange(Tmax, device="cuda")
    # order of keeping: recent tokens first, then by weight, the earlier token first among equals
    w = torch.where(t >= n - recent, torch.full_like(st["weights"], math.inf), st["weights"])
    w = torch.where(t >= n, torch.full_like(w, -math.inf), w)
    order = torch.sort(w, dim=-1, descending=True, stable=True)[1]
    kept = torch.sort(torch.where(torch.arange(Tout, device="cuda") < n, order[..., :Tout], Tmax), dim=-1)[0]
    live = kept < Tmax
    src = torch.where(live, kept, 0)
    res = []
    for c in (st["k"], st["v"]):
        codes, s, z = c
        rows = torch.gather(codes, 2, src[..., None].expand(-1, -1, -1, codes.shape[-1]))
        res.append(torch.where(live[..., None], rows, torch.zeros_like(rows)))
        for p in (s, z):
            if p is not None:
                row = torch.gather(p, 2, src)
                res.append(torch.where(live, row, torch.zeros_like(row)))
    wk = torch.gather(st["weights"], 2, src)
    res.append(torch.where(live, wk, torch.zeros_like(wk)))
    res.append(st["lengths"].clamp(max=budget))
    index = torch.full((B, Hkv, budget), -1, dtype=torch.int32, device="cuda")
    index[..., :Tout] = torch.where(live, kept, -1).to(torch.int32)
    res.append(index)
    return res


# --------------------------------------------------------------------------- 64 bits

def _exact_rows(cache, bits):
    """The rows a cache stands for, ``s c`` or ``s (u - z)``, in 64 bits."""
    codes, s, z = cache
    if bits == 8:
        return codes.double().mul_(s.double().unsqueeze(-1))
    shifts = torch.arange(0, 32, 4, dtype=torch.int32, device=codes.device)
    u = torch.bitwise_and(torch.bitwise_right_shift(codes.unsqueeze(-1), shifts), 15)
    return u.reshape(*codes.shape[:-1], codes.shape[-1] * 8).double().sub_(z.double().unsqueeze(-1)).mul_(
        s.double().unsqueeze(-1))


def exact(case, seed):
    st = prepare(case, seed)
    op, D, lens = case["op"], case["D"], st["lens"]
    if op == "prompt":
        group = case["Hq"] // case["Hkv"]
        out = torch.zeros(st["out"].shape, dtype=torch.float64, device="cuda")
        first = 0
        for n in lens:
            last = first + n
            for h in range(case["Hq"]):
                keys, vals = st["k"][first:last, h // group].double(), st["v"][first:last, h // group].double()
                for a in range(0, n, 4096):                    # rows a .. b see keys 0 .. b - 1
                    b = min(n, a + 4096)
                    s = (st["q"][first + a:first + b, h].double() @ keys[:b].t()) * D ** -0.5
                    i = torch.arange(a, b, device="cuda").unsqueeze(1)
                    s[torch.arange(b, device="cuda") > i] = -math.inf
                    out[first + a:first + b, h] = torch.softmax(s, 1) @ vals[:b]
            first = last
        return out
    bits = case["bits"]
    if op == "evict":
        return _exact_evict(case, st)
    group = case["Hq"] // case["Hkv"]
    out = torch.zeros(st["out"].shape, dtype=torch.float64, device="cuda")
    sums = torch.zeros(case["B"], case["Hkv"], case["Tmax"], dtype=torch.float64, device="cuda")
    pk = pv = None
    if op == "shared":
        pk, pv = _exact_rows(st["kp"], bits), _exact_rows(st["vp"], bits)
    for b, n in enumerate(lens):
        part = lambda c: tuple(None if t is None else t[b, :, :n] for t in c)
        keys, vals = _exact_rows(part(st["k"]), bits), _exact_rows(part(st["v"]), bits)
        for h in range(case["Hkv"]):
            kk, vv = keys[h], vals[h]
            if pk is not None:
                kk, vv = torch.cat([pk[h], kk]), torch.cat([pv[h], vv])
            qs = st["q"][b, h * group:(h + 1) * group].double()
            p = torch.softmax((qs @ kk.t()) * D ** -0.5, 1)
            out[b, h * group:(h + 1) * group] = p @ vv
            if op == "weights":
                sums[b, h, :n] = st["weights"][b, h, :n].double() + p.sum(0)
    return out if op == "shared" else (out, sums)


def _exact_evict(case, st):
    """What is kept, by sorting every head's tokens on the host."""
    import numpy as np
    budget, recent = case["budget"], case["recent"]
    dst = [None if t is None else torch.zeros_like(t) for t in (*st["out"][0], *st["out"][1], st["out"][2])]
    src = [*st["k"], *st["v"], st["weights"]]
    index = torch.full(st["out"][4].shape, -1, dtype=torch.int32)
    weights = st["weights"].cpu().numpy()
    for b, n in enumerate(st["lens"]):
        for h in range(case["Hkv"]):
            old = max(0, n - recent)
            if n <= budget:
                keep = np.arange(n)
            else:
                best = np.argsort(-weights[b, h, :old].astype(np.float64), kind="stable")[:budget - recent]
                keep = np.concatenate([np.sort(best), np.arange(old, n)])
            index[b, h, :len(keep)] = torch.from_numpy(keep.astype(np.int32))
            at = torch.from_numpy(keep).cuda()
            for d, s in zip(dst, src):
                if d is not None:
                    d[b, h, :len(keep)] = s[b, h][at]
    kept = torch.tensor([min(n, budget) for n in st["lens"]], dtype=torch.int32, device="cuda")
    return [t for t in dst if t is not None] + [kept, index.cuda()]
