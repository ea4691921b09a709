"""The layer operators together with the ring, as an attention layer uses them.

Training: projection -> rotary into the ring's load-balanced shard order -> ring attention -> output projection with
residual, and the whole chain backwards.  Serving: the prompt's keys and values go to the 4-bit cache, then single tokens
run linear -> rotary -> append -> attention -> linear.
"""
import math

import numpy as np
import pytest
import torch

from layer_util import f64, need_gpu, randn
from oracle import layer as ol

pytestmark = pytest.mark.gpu


def rel(a, b):
    return float(np.linalg.norm(a - b) / np.linalg.norm(b))


def test_training_layer(psr):
    need_gpu()
    S, P, Hq, Hkv, d, E = 2048, 4, 4, 2, 64, 192
    g = torch.Generator().manual_seed(0)
    x = randn(g, (S, E), "bf16")
    wqkv, wo = randn(g, ((Hq + 2 * Hkv) * d, E), "bf16", E**-0.5), randn(g, (E, Hq * d), "bf16", (Hq * d)**-0.5)
    bqkv, dy = randn(g, ((Hq + 2 * Hkv) * d,), "bf16", 0.1), randn(g, (S, E), "bf16")
    table = psr.rotary_table(d)
    kw = dict(P=P, causal=psr.CAUSAL_BALANCED)
    heads = lambda t, a, b: t.view(1, S, -1, d)[:, :, a:b].transpose(1, 2)

    qkv, _, _ = psr.linear(x, wqkv, bqkv)
    q, k = psr.rotary(heads(qkv, 0, Hq), heads(qkv, Hq, Hq + Hkv), table, **kw)
    v = heads(qkv, Hq + Hkv, Hq + 2 * Hkv).contiguous()
    o, lse, ws = psr.ring_attn_fwd(q, k, v, **kw)
    assert psr.get_stats(ws)["status"] == 0
    flat = o[0].transpose(0, 1).reshape(S, Hq * d)
    y, _, _ = psr.linear(flat, wo, None, x)

    dflat, dwo, _, _ = psr.linear_bwd(dy, flat, wo, need_db=False)
    do = heads(dflat, 0, Hq).contiguous()
    dq, dk, dv, _ = psr.ring_attn_bwd(q, k, v, o, lse, do, **kw)
    dqkv = torch.empty_like(qkv)
    psr.rotary_bwd(dq, dk, table, q_out=heads(dqkv, 0, Hq), k_out=heads(dqkv, Hq, Hq + Hkv), **kw)
    heads(dqkv, Hq + Hkv, Hq + 2 * Hkv).copy_(dv)
    dx, dwqkv, dbqkv, _ = psr.linear_bwd(dqkv, x, wqkv)

    # the same layer in 64 bits, with autograd, in the order of the positions
    pos = ol.shard_positions(S, P, True)
    X, WQ, WO, BQ = (t.double().cpu().requires_grad_() for t in (x, wqkv, wo, bqkv))
    z = X @ WQ.T + BQ
    Q, K, V = (z.view(S, -1, d)[:, a:b].transpose(0, 1) for a, b in ((0, Hq), (Hq, Hq + Hkv), (Hq + Hkv, Hq + 2 * Hkv)))
    ang = torch.from_numpy(pos[:, None] * ol.frequencies(d)[None])
    c, s = torch.cos(ang), torch.sin(ang)
    turn = lambda t: torch.cat([t[..., :d // 2] * c - t[..., d // 2:] * s, t[..., d // 2:] * c + t[..., :d // 2] * s], -1)
    Q, K = turn(Q), turn(K).repeat_interleave(Hq // Hkv, 0)
    sc = Q @ K.transpose(1, 2) / math.sqrt(d)
    p = torch.from_numpy(pos)
    sc = sc.masked_fill(p[None, :] > p[:, None], -math.inf)
    O = torch.softmax(sc, -1) @ V.repeat_interleave(Hq // Hkv, 0)
    Y = O.transpose(0, 1).reshape(S, Hq * d) @ WO.T + X
    (Y * dy.double().cpu()).sum().backward()
    # each bf16 tensor between two steps is off by at most 2^-8 of its values (2^-8 / sqrt 3 rms): six of them forward
    # (qkv, q/k, P, o, y) stay below 2^-7 in the 2-norm; backward passes through twice as many
    assert rel(f64(y), Y.detach().numpy()) <= 2.0**-7
    dx = dx.double() + dy.double()  # the residual's gradient
    for got, want, name in ((dx, X, "dx"), (dwqkv, WQ, "dwqkv"), (dwo, WO, "dwo"), (dbqkv, BQ, "dbqkv")):
        assert rel(f64(got), want.grad.numpy()) <= 2.0**-6, name


def test_serving_layer(psr):
    need_gpu()
    B, Hq, Hkv, d, E, page, prompt, steps = 2, 8, 2, 128, 256, 32, 512, 3
    g = torch.Generator().manual_seed(1)
    wqkv, wo = randn(g, ((Hq + 2 * Hkv) * d, E), "bf16", E**-0.5), randn(g, (E, Hq * d), "bf16", (Hq * d)**-0.5)
    table = psr.rotary_table(d)
    n_max = (prompt + steps + page - 1) // page
    cache = psr.kv4_cache(B * n_max, Hkv, d, page)
    pages = torch.randperm(B * n_max, generator=g).view(B, n_max).to(torch.int32).cuda()
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    x = randn(g, (B, prompt, E), "bf16")
    heads = lambda t, S, a, b: t.view(B, S, -1, d)[:, :, a:b].transpose(1, 2)

    qkv, _, _ = psr.linear(x.view(B * prompt, E), wqkv)
    q, k = psr.rotary(heads(qkv, prompt, 0, Hq), heads(qkv, prompt, Hq, Hq + Hkv), table)
    v = heads(qkv, prompt, Hq + Hkv, Hq + 2 * Hkv)
    psr.kv4_append(k, v, cache, pages, lens, page=page)
    # attention over the cached prompt, through the ring and through the cache: the same rows
    kr, vr = psr.kv4_read(cache, pages, lens, S=prompt, Hkv=Hkv, d=d, page=page)
    o_ring, lse_ring, _ = psr.ring_attn_fwd(q, kr, vr, P=1, causal=True)
    lens += prompt
    last = 5
    o_kv4, lse_kv4, _ = psr.kv4_attn(q[:, :, -last:], cache, pages, lens, Hkv=Hkv, page=page)
    # the ring reads K and V rounded to bf16 (2^-8 of each value), the cache's attention as they stand
    assert rel(f64(o_kv4), f64(o_ring[:, :, -last:])) <= 2.0**-6
    assert np.abs(f64(lse_kv4) - f64(lse_ring[:, :, -last:])).max() <= 0.05

    def step(x, pos):
        qkv, _, _ = psr.linear(x, wqkv)
        q, k = psr.rotary(heads(qkv, 1, 0, Hq), heads(qkv, 1, Hq, Hq + Hkv), table, positions=pos)
        psr.kv4_append(k, heads(qkv, 1, Hq + Hkv, Hq + 2 * Hkv), cache, pages, lens, page=page)
        o, _, _ = psr.kv4_attn(q, cache, pages, lens + 1, Hkv=Hkv, page=page)
        y, _, _ = psr.linear(o.view(B, Hq * d), wo, None, x)
        return q, o, y
    for _ in range(steps):
        x1 = randn(g, (B, E), "bf16")
        q1, o1, y1 = step(x1, lens.long()[:, None].contiguous())
        lens += 1
        n = int(lens[0])
        ro, _, to, _ = ol.kv4_attention(f64(q1), cache.cpu().numpy(), pages.cpu().numpy(), [n] * B, page, Hkv, 1 / math.sqrt(d))
        assert (np.abs(f64(o1) - ro) <= to + 2.0**-8 * np.abs(ro) * 1.01).all()
        ry, _ = ol.linear(f64(o1).reshape(B, -1), f64(wo), None, f64(x1))
        assert rel(f64(y1), ry) <= 2.0**-8

    # the whole step in a graph: lengths and positions move on the device
    x1, pos = randn(g, (B, E), "bf16"), lens.long()[:, None].contiguous()
    keep = cache.clone()
    want = step(x1, pos)
    cache.copy_(keep)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(x1, pos)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_calls_with_the_same_shapes(psr):
    # what a call finds out about its arguments serves the next one: other values, strides, types and places count
    need_gpu()
    g = torch.Generator().manual_seed(3)
    B, Hq, Hkv, d, page, n = 2, 4, 2, 64, 16, 40
    cache = psr.kv4_cache(6, Hkv, d, page)
    table = torch.arange(6, dtype=torch.int32, device="cuda").view(B, 3)
    lens = torch.full((B,), n, dtype=torch.int32, device="cuda")
    psr.kv4_append(randn(g, (B, Hkv, n, d), "bf16"), randn(g, (B, Hkv, n, d), "bf16"), cache, table, lens * 0, page=page)
    q = randn(g, (B, Hq, 1, d), "bf16")
    scale = torch.tensor(0.125)
    for s in (0.125, 0.5, 0.125):
        scale.fill_(s)  # a number, whatever holds it
        got = psr.kv4_attn(q, cache, table, lens, Hkv=Hkv, page=page, scale=scale)[0]
        ro, _, to, _ = ol.kv4_attention(f64(q), cache.cpu().numpy(), table.cpu().numpy(), [n] * B, page, Hkv, s)
        assert (np.abs(f64(got) - ro) <= to + 2.0**-8 * np.abs(ro) * 1.01).all(), s
    rot = psr.rotary_table(d)
    x = randn(g, (1, 2, 8, d), "f32")
    for off in (0, 5, 1 << 40, 0):
        y = psr.rotary(x, None, rot, offset=off)[0]
        assert torch.equal(y, psr.rotary(x, None, rot, positions=torch.arange(8, device="cuda") + off)[0]), off
    for t in ("bf16", "f16", "bf16"):
        for shift in (0, 1, 0):
            a, w = randn(g, (3 * 64 + 1,), t)[shift:shift + 192].view(3, 64), randn(g, (40, 64), t, 0.125)
            ref, _ = ol.linear(f64(a), f64(w))
            y = psr.linear(a, w)[0]
            assert y.dtype == a.dtype and rel(f64(y), ref) <= 2.0**-8
            y2 = psr.linear(a[:, :32], w[:, 32:])[0]
            assert rel(f64(y2), ol.linear(f64(a[:, :32]), f64(w[:, 32:]))[0]) <= 2.0**-8
    with pytest.raises(ValueError, match="w must have shape"):
        psr.linear(a, w[:, :32])
    with pytest.raises(ValueError, match="w must be torch.bfloat16"):
        psr.linear(a, w.half())
