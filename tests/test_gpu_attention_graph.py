"""The attention and eviction entry points in a captured HIP graph: captured once with preallocated
outputs and workspaces, replayed several times with other eager work (the same calls on other data,
synchronizations) in between and with inputs changed in place, every replay equal bit for bit to the
eager call on the same inputs."""

from __future__ import annotations

import pytest
import torch

import w4a16_dequant_gemm_amd as W4
from tests.kv_util import make_cache

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _needs_gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    W4.lib()


def _flat(r):
    out = []
    for t in r if isinstance(r, (list, tuple)) else [r]:
        out += _flat(t) if isinstance(t, (list, tuple)) else [t] if t is not None else []
    return out


def test_replays_equal_eager_calls():
    dt = torch.float16
    g = torch.Generator(device="cuda").manual_seed(1)
    B, Hq, Hkv, D, T = 3, 8, 2, 128, 600
    lengths = torch.tensor([600, 0, 333], dtype=torch.int32, device="cuda")
    q = torch.randn((B, Hq, D), generator=g, device="cuda").to(dt)
    k, v = make_cache((B, Hkv, T, D), 8, dt, 1), make_cache((B, Hkv, T, D), 8, dt, 2)
    k4, v4 = make_cache((B, Hkv, T, D), 4, dt, 3), make_cache((B, Hkv, T, D), 4, dt, 4)
    kp, vp = make_cache((Hkv, 500, D), 8, dt, 5), make_cache((Hkv, 500, D), 8, dt, 6)
    w = torch.rand((B, Hkv, T), generator=g, device="cuda")
    x = torch.randn((700, 12 * D), generator=g, device="cuda").to(dt)
    pq, pk, pv = (t.unflatten(1, (-1, D)) for t in x.split([8 * D, 2 * D, 2 * D], dim=1))
    cu = torch.tensor([0, 500, 500, 690], dtype=torch.int32, device="cuda")

    def room(c, n):
        return tuple(None if t is None else torch.zeros((B, Hkv, n) + t.shape[3:], dtype=t.dtype, device="cuda") for t in c)

    def evict_out():
        return (room(k4, 256), room(v4, 256), torch.zeros((B, Hkv, 256), device="cuda"), torch.zeros_like(lengths),
                torch.zeros((B, Hkv, 200), dtype=torch.int32, device="cuda"))
    ws = torch.empty(W4.kv_attention_shared_workspace(B, Hq, Hkv, 500, T, D), device="cuda")
    ww = torch.empty(W4.kv_attention_weights_workspace(B, Hq, Hkv, T, D), device="cuda")
    calls = [
        (lambda o: W4.attention_prompt(pq, pk, pv, cu, out=o), lambda: torch.zeros((700, 8, D), dtype=dt, device="cuda")),
        (lambda o: W4.kv_attention_decode_shared(q, kp, vp, 500, k, v, lengths, 8, out=o, work=ws),
         lambda: torch.zeros_like(q)),
        (lambda o: W4.kv_attention_decode_shared(q, kp, vp, 100, k, v, lengths, 8, out=o), lambda: torch.zeros_like(q)),
        (lambda o: W4.kv_attention_decode_weights(q, k4, v4, lengths, w, 4, sums=o[1], out=o[0], work=ww),
         lambda: (torch.zeros_like(q), torch.zeros_like(w))),
        (lambda o: W4.kv_evict(k4, v4, w, lengths, 200, 20, 4, out=o), evict_out),
    ]
    outs = [make() for _, make in calls]
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        for (fn, _), o in zip(calls, outs):
            fn(o)
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=side):
            for (fn, _), o in zip(calls, outs):
                fn(o)
    torch.cuda.synchronize()
    for rep in range(4):
        # other inputs in the same memory, other lengths
        q.copy_(torch.randn(q.shape, generator=g, device="cuda"))
        x.copy_(torch.randn(x.shape, generator=g, device="cuda"))
        w.copy_(torch.rand(w.shape, generator=g, device="cuda"))
        lengths.copy_(torch.tensor([[600, 1, 200], [0, 600, 599], [201, 200, 64], [5, 555, 128]][rep],
                                   dtype=torch.int32))
        want = [_flat(fn(make())) for fn, make in calls]
        for o in _flat(outs):
            o.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for i, (o, ref) in enumerate(zip(outs, want)):
            for a, b in zip(_flat(o), ref):
                assert torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8)), f"replay {rep}, call {i}"
