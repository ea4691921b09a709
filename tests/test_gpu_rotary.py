"""GPU parity of psr_rotary against the fp64 oracle, through the binding.

Tolerance: cos and sin come from the angle modulo a turn cut to 2^-32 of a turn (2 pi 2^-32 < 2^-29 radians) by a
function with a few units of 2^-24, the two products and their sum add three roundings of 2^-24: together below
2^-20 a (|x1| + |x2|).  Then one rounding to the type (half a step of the value; below the smallest normal fp16
number 2^-25 absolute).  Copied columns are equal.
"""
import numpy as np
import pytest
import torch

from layer_util import TYPES, check, f64, need_gpu, randn
from oracle import layer as ol

pytestmark = pytest.mark.gpu


def reference(x, pos, freq, t, amplitude=1.0, **kw):
    x = f64(x)
    y = ol.rotary(x, pos, freq, amplitude, **kw)
    n = len(freq)
    size = np.zeros_like(x)
    a, b = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if kw.get("interleaved") else (slice(0, n), slice(n, 2 * n))
    size[..., a] = size[..., b] = abs(amplitude) * (np.abs(x[..., a]) + np.abs(x[..., b]))
    return y, ol.HALF_STEP[t] * np.abs(y) + 2.0**-20 * size + (2.0**-25 if t == "f16" else 0.0) * (size > 0)


CASES = [  # B S Hq Hkv d rot interleaved type
    (1, 1, 1, 1, 2, 2, False, "bf16"),
    (1, 7, 2, 1, 64, 64, False, "bf16"),
    (2, 33, 4, 2, 128, 128, False, "bf16"),
    (2, 33, 4, 2, 128, 128, True, "bf16"),
    (3, 5, 3, 3, 80, 40, False, "f16"),
    (3, 5, 3, 3, 80, 48, True, "f16"),
    (1, 129, 8, 1, 64, 16, False, "f32"),
    (1, 129, 8, 1, 64, 24, True, "f32"),
    (2, 9, 5, 1, 65, 62, False, "bf16"),
    (2, 9, 5, 1, 65, 62, True, "f32"),
    (1, 300, 32, 8, 128, 96, False, "f16"),
    (1, 3, 2, 2, 1024, 1024, False, "bf16"),
]


@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("case", CASES, ids=str)
def test_rotary(psr, case, inverse):
    need_gpu()
    B, S, Hq, Hkv, d, rot, inter, t = case
    g = torch.Generator().manual_seed(sum(case[:6]))
    q, k = randn(g, (B, Hq, S, d), t), randn(g, (B, Hkv, S, d), t)
    f = psr.rotary_bwd if inverse else psr.rotary
    qo, ko = f(q, k, psr.rotary_table(rot), interleaved=inter, offset=11, amplitude=1.25)
    pos = [range(11, 11 + S)]
    for x, y in ((q, qo), (k, ko)):
        assert y.is_contiguous() and y.dtype == x.dtype
        check(y, *reference(x, pos, ol.frequencies(rot), t, 1.25, interleaved=inter, inverse=inverse), str(case))
        assert torch.equal(y[..., rot:], x[..., rot:])


@pytest.mark.parametrize("causal,P,S", [(2, 1, 6), (2, 4, 64), (2, 3, 30), (1, 4, 64), (0, 4, 64)])
def test_rotary_takes_positions_from_the_shard_order(psr, causal, P, S):
    need_gpu()
    g = torch.Generator().manual_seed(S + P)
    q, k = randn(g, (2, 2, S, 64), "bf16"), randn(g, (2, 1, S, 64), "bf16")
    pos = [ol.shard_positions(S, P, causal == 2) + 1000]
    for x, y in zip((q, k), psr.rotary(q, k, psr.rotary_table(64), P=P, causal=causal, offset=1000)):
        check(y, *reference(x, pos, ol.frequencies(64), "bf16"), f"causal={causal} P={P}")


@pytest.mark.parametrize("shape", ["S", "BS", "broadcast"])
def test_rotary_positions_given_near_and_far(psr, shape):
    # an angle in fp32 has no correct digit left at the far ones
    need_gpu()
    g = torch.Generator().manual_seed(5)
    far = torch.tensor([0, 1, -1, 131071, 2**24 + 1, 2**31 - 1, 2**31, 2**40 + 12345, -2**40, 2**62 + 1, -2**63])
    S, B = len(far), 3
    q = randn(g, (B, 2, S, 64), "f32")
    pos = {"S": far, "BS": torch.stack([far, far.flip(0), far * 3 // 4]), "broadcast": far.expand(B, S)}[shape]
    want = [[int(p) for p in row] for row in (pos if pos.dim() == 2 else pos[None])]
    # the table holds each frequency to 2^-64 of a turn per position: the oracle takes it as held
    table = psr.rotary_table(64)
    got, none = psr.rotary(q, None, table, positions=pos.cuda())
    assert none is None
    turns = [int(v) for v in table.cpu()]
    ang = np.array([[[(p * w % 2**64) / 2**64 * 2 * np.pi for w in turns] for p in row] for row in want])[:, None]
    x = f64(q)
    c, s = np.cos(ang), np.sin(ang)
    ref = np.concatenate([x[..., :32] * c - x[..., 32:] * s, x[..., 32:] * c + x[..., :32] * s], -1)
    size = np.abs(x[..., :32]) + np.abs(x[..., 32:])
    check(got, ref, 2.0**-24 * np.abs(ref) + 2.0**-20 * np.concatenate([size, size], -1), shape)


def test_rotary_of_projection_views_and_in_place(psr):
    need_gpu()
    g = torch.Generator().manual_seed(8)
    B, S, Hq, Hkv, d = 2, 37, 4, 2, 64
    qkv = randn(g, (B, S, Hq + 2 * Hkv, d), "bf16")
    q, k = qkv[:, :, :Hq].transpose(1, 2), qkv[:, :, Hq:Hq + Hkv].transpose(1, 2)
    table = psr.rotary_table(64)
    qo, ko = psr.rotary(q, k, table)
    for x, y in ((q, qo), (k, ko)):
        check(y, *reference(x, [range(S)], ol.frequencies(64), "bf16"), "views")
    before = qkv.clone()
    a, b = psr.rotary(q, k, table, q_out=q, k_out=k)  # in place, inside the projection's rows
    assert a is q and b is k and torch.equal(q, qo) and torch.equal(k, ko)
    assert torch.equal(qkv[:, :, Hq + Hkv:], before[:, :, Hq + Hkv:])
    # odd offsets and strides: one element off a 16-byte boundary, padded rows
    wide = torch.zeros(B * S * Hq * 67 + 1, dtype=torch.bfloat16, device="cuda")
    odd = wide[1:].view(B, Hq, S, 67)[..., 1:65]
    odd.copy_(before[:, :, :Hq].transpose(1, 2))
    out, _ = psr.rotary(odd, None, table, q_out=odd)
    assert torch.equal(out, qo)
    assert int((wide != 0).sum()) == int((qo != 0).sum())


def test_rotary_broadcast_input(psr):
    need_gpu()
    g = torch.Generator().manual_seed(9)
    k = randn(g, (1, 1, 5, 64), "bf16")
    y, _ = psr.rotary(k.expand(3, 4, 5, 64), None, psr.rotary_table(64))
    z, _ = psr.rotary(k, None, psr.rotary_table(64))
    assert torch.equal(y, z.expand(3, 4, 5, 64))


def test_rotary_no_rows(psr):
    need_gpu()
    e = torch.empty((2, 4, 0, 64), dtype=torch.bfloat16, device="cuda")
    a, b = psr.rotary(e, e[:, :2], psr.rotary_table(64))
    assert a.shape == (2, 4, 0, 64) and b.shape == (2, 2, 0, 64)


def test_rotary_bwd_is_the_gradient(psr):
    # the map is linear: <rotary(x), g> = <x, rotary_bwd(g)>, and the oracle's difference quotient along g
    need_gpu()
    g = torch.Generator().manual_seed(10)
    x, dy = randn(g, (2, 3, 17, 64), "f32"), randn(g, (2, 3, 17, 64), "f32")
    table = psr.rotary_table(48, scaling="by_parts", factor=4.0, original_length=4096)
    kw = dict(amplitude=1.1, interleaved=True)
    dx, _ = psr.rotary_bwd(dy, None, table, **kw)
    freq = ol.frequencies(48, scaling="by_parts", factor=4.0, original=4096)
    f = lambda v: (ol.rotary(v, [range(17)], freq, 1.1, True) * f64(dy)).sum()
    rng = np.random.default_rng(0)
    for _ in range(5):
        step = rng.standard_normal(x.shape)
        want = (f(f64(x) + 1e-3 * step) - f(f64(x) - 1e-3 * step)) / 2e-3
        got = (f64(dx) * step).sum()
        # rounding of dx: a random walk below 2^-20 of each term's size
        assert abs(got - want) <= 2.0**-20 * np.abs(f64(dx) * step).sum() + 1e-9 * abs(want) + 1e-6


def test_rotary_infinities_stay_in_their_pair(psr):
    need_gpu()
    x = torch.ones((1, 1, 4, 64), dtype=torch.bfloat16, device="cuda")
    x[0, 0, 2, 5] = float("inf")
    x[0, 0, 3, 40] = float("nan")
    y, _ = psr.rotary(x, None, psr.rotary_table(64))
    odd = ~torch.isfinite(y[0, 0])
    assert odd.nonzero().tolist() == [[2, 5], [2, 37], [3, 8], [3, 40]]


def test_rotary_graph_and_streams(psr):
    need_gpu()
    g = torch.Generator().manual_seed(12)
    q, k = randn(g, (4, 8, 1, 128), "bf16"), randn(g, (4, 2, 1, 128), "bf16")
    pos = torch.tensor([[3], [70], [900], [12]], device="cuda")
    table = psr.rotary_table(128)
    want = psr.rotary(q, k, table, positions=pos)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = psr.rotary(q, k, table, positions=pos, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    out = [torch.zeros_like(t) for t in want]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        psr.rotary(q, k, table, positions=pos, q_out=out[0], k_out=out[1])
    for _ in range(2):
        q.neg_()
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, want))
