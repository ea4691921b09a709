"""GPU parity of psr_linear and psr_linear_bwd against the fp64 oracle, through the binding.

Tolerance.  A product's fp32 sum of K terms is off by at most K 2^-23 sum |x| |w| (each addition rounds or truncates,
2^-23), bias and residual add a rounding each, the activation a few units of 2^-24 of |z| + 1 (its slope is at most
1.13 in size), and the result is rounded once to its type (half a step; 2^-25 absolute below the normal fp16
numbers).  Backward: act' is evaluated in fp32 (2^-19 |dy|), dz is rounded to the type before the products, which adds
half a step of |dz| |w| (|dz| |x|); db sums the unrounded dz.
"""
import numpy as np
import pytest
import torch

from layer_util import check, f64, need_gpu, randn
from oracle import layer as ol

pytestmark = pytest.mark.gpu

TINY = {"bf16": 0.0, "f16": 2.0**-25}


def sum_tol(a, b):
    """|a| [M, K], |b| [N, K] -> bound on the fp32 sum of a b^T."""
    return a.shape[1] * 2.0**-23 * (np.abs(a) @ np.abs(b).T)


def check_forward(got_y, got_z, x, w, bias, res, act, t, what):
    a = [None if v is None else f64(v) for v in (x, w, bias, res)]
    y, z = ol.linear(a[0], a[1], a[2], a[3], act)
    e = sum_tol(a[0], a[1]) + 2.0**-23 * np.abs(z)
    r = np.zeros_like(y) if res is None else a[3]
    h = ol.HALF_STEP[t]
    check(got_y, y, h * np.abs(y) * 1.01 + 1.13 * e + 2.0**-20 * (np.abs(z) + np.abs(r) + 1) * (act != "none" or res is not None)
          + TINY[t], what)
    if got_z is not None:
        check(got_z, z, h * np.abs(z) * 1.01 + e + TINY[t], what + " z")


def check_backward(got, dy, x, w, z, act, t, what):
    d = [None if v is None else f64(v) for v in (dy, x, w, z)]
    dx, dw, db, dz = ol.linear_bwd(d[0], d[1], d[2], d[3], act)
    h = ol.HALF_STEP[t]
    edz = (2.0**-19 * np.abs(d[0]) + h * np.abs(dz) * 1.01 + TINY[t]) if act != "none" else np.zeros_like(dz)
    if got[0] is not None:
        check(got[0], dx, h * np.abs(dx) * 1.01 + edz @ np.abs(d[2]) + sum_tol(dz, d[2].T) + TINY[t], what + " dx")
    if got[1] is not None:
        check(got[1], dw, h * np.abs(dw) * 1.01 + edz.T @ np.abs(d[1]) + sum_tol(dz.T, d[1].T) + TINY[t], what + " dw")
    if got[2] is not None:
        slope = 2.0**-19 * np.abs(d[0]).sum(0) if act != "none" else 0.0
        check(got[2], db, h * np.abs(db) * 1.01 + slope + len(dz) * 2.0**-23 * np.abs(dz).sum(0) + TINY[t], what + " db")


ACTS = ["none", "relu", "gelu", "gelu_tanh", "silu"]

FORWARD = [  # M N K act bias residual z type
    (1, 8, 8, "none", False, False, False, "bf16"),
    (1, 1, 1, "none", True, True, True, "bf16"),
    (1, 256, 512, "silu", True, True, True, "bf16"),
    (1, 1000, 4104, "none", True, True, False, "f16"),
    (2, 264, 72, "gelu", False, True, False, "bf16"),
    (3, 33, 17, "relu", True, False, True, "f16"),
    (5, 640, 2048, "gelu_tanh", True, False, True, "bf16"),
    (8, 128, 64, "none", False, False, False, "f16"),
    (9, 136, 1032, "silu", True, True, True, "bf16"),
    (16, 72, 192, "relu", True, True, False, "bf16"),
    (17, 512, 256, "gelu", True, True, True, "f16"),
    (31, 1024, 776, "none", True, False, False, "bf16"),
    (33, 96, 520, "silu", False, False, True, "bf16"),
    (64, 256, 128, "none", True, True, True, "bf16"),
    (65, 200, 136, "gelu_tanh", True, True, True, "bf16"),
    (100, 77, 50, "gelu", True, True, True, "bf16"),
    (127, 264, 64, "relu", True, True, True, "f16"),
    (128, 256, 64, "none", False, False, False, "bf16"),
    (129, 512, 328, "silu", True, True, True, "bf16"),
    (255, 520, 96, "gelu", True, False, True, "f16"),
    (256, 256, 256, "none", True, True, False, "bf16"),
    (257, 776, 200, "gelu_tanh", True, True, True, "bf16"),
    (300, 1288, 40, "relu", True, True, True, "bf16"),
    (513, 264, 1000, "none", True, True, True, "f16"),
    (1000, 8, 24, "silu", True, True, True, "bf16"),
    (1100, 1032, 264, "gelu", True, True, True, "bf16"),
    (1, 301, 515, "silu", True, True, True, "bf16"),
    (6, 301, 515, "relu", True, True, True, "f16"),
    (70, 1001, 515, "gelu", True, True, True, "bf16"),
    (300, 517, 333, "silu", True, True, True, "f16"),
    (1300, 901, 77, "relu", True, True, True, "bf16"),
]


@pytest.mark.parametrize("case", FORWARD, ids=str)
def test_linear(psr, case):
    need_gpu()
    M, N, K, act, bias, res, save, t = case
    g = torch.Generator().manual_seed(M * 7 + N)
    x, w = randn(g, (M, K), t), randn(g, (N, K), t, K**-0.5)
    b = randn(g, (N,), t) if bias else None
    r = randn(g, (M, N), t) if res else None
    y, z, ws = psr.linear(x, w, b, r, activation=act, save_z=save)
    assert psr.get_stats(ws)["status"] == 0
    assert (z is not None) == save
    check_forward(y, z, x, w, b, r, act, t, str(case))


# several rounds of 512-column tiles over the pairs of SMs, with halves of tiles first and last, and an odd last half
ROUNDS = [(700, 3900, 40), (2600, 2600, 72), (2600, 5200, 64), (5000, 4400, 136), (9000, 1100, 64)]


@pytest.mark.parametrize("M,N,K", ROUNDS)
def test_linear_rounds_of_tiles(psr, M, N, K):
    need_gpu()
    g = torch.Generator().manual_seed(M)
    x, w, b, r = randn(g, (M, K), "bf16"), randn(g, (N, K), "bf16", K**-0.5), randn(g, (N,), "bf16"), randn(g, (M, N), "bf16")
    y, z, ws = psr.linear(x, w, b, r, activation="relu", save_z=True)
    assert psr.get_stats(ws)["status"] == 0
    check_forward(y, z, x, w, b, r, "relu", "bf16", str((M, N, K)))


BACKWARD = [  # M N K act type
    (1, 8, 8, "none", "bf16"),
    (1, 1, 1, "gelu", "bf16"),
    (1, 264, 136, "silu", "bf16"),
    (3, 33, 17, "relu", "f16"),
    (7, 128, 512, "none", "bf16"),
    (40, 520, 72, "gelu_tanh", "bf16"),
    (63, 64, 64, "relu", "bf16"),
    (64, 256, 512, "none", "f16"),
    (65, 264, 520, "gelu", "bf16"),
    (100, 77, 50, "silu", "bf16"),
    (129, 384, 256, "gelu_tanh", "f16"),
    (257, 1000, 264, "silu", "bf16"),
    (511, 136, 1288, "relu", "bf16"),
    (1027, 520, 264, "gelu", "bf16"),
    (2000, 16, 8, "none", "bf16"),
    (70, 5200, 2600, "relu", "bf16"),
    (301, 515, 333, "none", "bf16"),
    (301, 515, 333, "gelu", "f16"),
    (2600, 136, 5200, "none", "bf16"),
]


@pytest.mark.parametrize("case", BACKWARD, ids=str)
def test_linear_bwd(psr, case):
    need_gpu()
    M, N, K, act, t = case
    g = torch.Generator().manual_seed(M + 3 * N)
    dy, x, w = randn(g, (M, N), t), randn(g, (M, K), t), randn(g, (N, K), t, K**-0.5)
    z = randn(g, (M, N), t) if act != "none" else None
    dx, dw, db, ws = psr.linear_bwd(dy, x, w, z, activation=act)
    assert psr.get_stats(ws)["status"] == 0
    check_backward((dx, dw, db), dy, x, w, z, act, t, str(case))


@pytest.mark.parametrize("need", [(1, 0, 0), (0, 1, 0), (0, 0, 1), (1, 1, 0), (0, 0, 0)], ids=str)
@pytest.mark.parametrize("act", ["none", "silu"])
def test_linear_bwd_of_some(psr, need, act):
    need_gpu()
    g = torch.Generator().manual_seed(4)
    M, N, K = 70, 136, 264
    dy, x, w, z = (randn(g, s, "bf16") for s in ((M, N), (M, K), (N, K), (M, N)))
    got = psr.linear_bwd(dy, x, w, z, activation=act, need_dx=need[0], need_dw=need[1], need_db=need[2])[:3]
    assert [v is not None for v in got] == [bool(v) for v in need]
    check_backward(got, dy, x, w, z, act, "bf16", str(need))


@pytest.mark.parametrize("pad,shift", [(8, 0), (1, 0), (0, 1), (8, 8)])
@pytest.mark.parametrize("M", [1, 5, 70, 300])
def test_linear_strided_rows(psr, pad, shift, M):
    # rows on 16-byte boundaries and off them
    need_gpu()
    g = torch.Generator().manual_seed(pad + M)
    N, K, t = 264, 136, "bf16"

    def padded(rows, cols, std=1.0):
        flat = randn(g, (rows * (cols + pad) + shift,), t, std)[shift:]
        return flat.view(rows, cols + pad)[:, :cols]
    x, w, r, y, z, dy = padded(M, K), padded(N, K, K**-0.5), padded(M, N), padded(M, N), padded(M, N), padded(M, N)
    edge = torch.as_strided(y, (M, pad), (N + pad, 1), y.storage_offset() + N).clone()
    a, b, _ = psr.linear(x, w, None, r, activation="gelu", out=y, z=z)
    assert a is y and b is z
    check_forward(y, z, x, w, None, r, "gelu", t, "strided")
    if M > 1:  # between the rows nothing is written
        last = slice(0, M - 1 if shift or pad else M)
        assert torch.equal(torch.as_strided(y, (M, pad), (N + pad, 1), y.storage_offset() + N)[last], edge[last])
    got = psr.linear_bwd(dy, x, w, z, activation="gelu")[:3]
    check_backward(got, dy, x, w, z, "gelu", t, "strided bwd")


def test_linear_residual_in_place(psr):
    need_gpu()
    for M in (1, 40, 300):
        g = torch.Generator().manual_seed(M)
        x, w, r = randn(g, (M, 128), "bf16"), randn(g, (264, 128), "bf16", 0.1), randn(g, (M, 264), "bf16")
        keep = r.clone()
        y, _, _ = psr.linear(x, w, None, r, out=r)
        assert y is r
        check_forward(y, None, x, w, None, keep, "none", "bf16", "in place")


def test_linear_no_rows(psr):
    need_gpu()
    x, w = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda"), torch.ones((16, 64), dtype=torch.bfloat16, device="cuda")
    y, z, _ = psr.linear(x, w, save_z=True)
    assert y.shape == z.shape == (0, 16)
    dx, dw, db, _ = psr.linear_bwd(y, x, w)
    assert dx.shape == (0, 64) and not dw.any() and not db.any() and dw.shape == (16, 64) and db.shape == (16,)


def test_linear_rows_do_not_mix(psr):
    # a NaN or an infinity in a row of x stays in that row, one in a row of w in that column, at the edges of tiles too
    need_gpu()
    for M, N, K in ((1, 264, 136), (20, 264, 136), (300, 264, 136)):
        g = torch.Generator().manual_seed(N)
        x, w = randn(g, (M, K), "bf16"), randn(g, (N, K), "bf16")
        x[M - 1, K - 1] = float("nan")
        w[N - 1, 0] = float("inf")
        y = psr.linear(x, w)[0]
        bad = ~torch.isfinite(y)
        want = torch.zeros_like(bad)
        want[M - 1] = True
        want[:, N - 1] = True
        assert torch.equal(bad, want)


def test_linear_is_deterministic_and_graph_safe(psr):
    need_gpu()
    g = torch.Generator().manual_seed(2)
    for M, N, K in ((1, 1032, 2056), (24, 520, 4104), (400, 520, 264)):
        x, w, r = randn(g, (M, K), "bf16"), randn(g, (N, K), "bf16", K**-0.5), randn(g, (M, N), "bf16")
        want = psr.linear(x, w, None, r, activation="silu", save_z=True)[:2]
        dwant = psr.linear_bwd(r, x, w, want[1], activation="silu")[:3]
        for _ in range(3):
            assert all(torch.equal(a, b) for a, b in zip(psr.linear(x, w, None, r, activation="silu", save_z=True)[:2], want))
            assert all(torch.equal(a, b) for a, b in zip(psr.linear_bwd(r, x, w, want[1], activation="silu")[:3], dwant))
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        got = psr.linear(x, w, None, r, activation="silu", save_z=True, stream=side)[:2]
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        out = [torch.zeros_like(v) for v in (*want, *dwant)]
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            psr.linear(x, w, None, r, activation="silu", out=out[0], z=out[1])
            psr.linear_bwd(r, x, w, out[1], activation="silu", dx=out[2], dw=out[3], db=out[4])
        for _ in range(2):
            graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, (*want, *dwant)))


@pytest.mark.parametrize("act", ACTS)
def test_linear_bwd_is_the_gradient(psr, act):
    # against difference quotients of the oracle's forward along random directions
    need_gpu()
    g = torch.Generator().manual_seed(6)
    M, N, K = 33, 40, 24
    x, w, b, dy = (randn(g, s, "f16", std) for s, std in (((M, K), 1), ((N, K), K**-0.5), ((N,), 0.5), ((M, N), 1)))
    y, z, _ = psr.linear(x, w, b, activation=act, save_z=True)
    grads = [f64(v) for v in psr.linear_bwd(dy, x, w, z, activation=act)[:3]]
    args = [f64(v) for v in (x, w, b)]
    rng = np.random.default_rng(1)
    for i in range(3):
        step = rng.standard_normal(args[i].shape)
        f = lambda h: (ol.linear(*[v + (h * step if j == i else 0) for j, v in enumerate(args)], None, act)[0] * f64(dy)).sum()
        want = (f(1e-5) - f(-1e-5)) / 2e-5
        # z, dz and the gradients are fp16 (2^-11 each, random signs); relu changes slope where a difference crosses 0
        assert abs((grads[i] * step).sum() - want) <= 2.0**-8 * np.linalg.norm(grads[i]) * 4, (act, i)


@pytest.mark.parametrize("act", ACTS)
def test_linear_bwd_of_large_z(psr, act):
    # where the square of z is infinite in fp32 the slopes are still 0 and 1
    need_gpu()
    z = torch.tensor([[-3e38, -1e20, -1e10, -300.0, 300.0, 1e10, 1e20, 3e38]] * 2, dtype=torch.bfloat16, device="cuda")
    one = torch.ones((8, 8), dtype=torch.bfloat16, device="cuda")
    db = psr.linear_bwd(torch.ones_like(z), one[:2], one, z, activation=act, need_dx=False, need_dw=False)[2]
    want = torch.ones_like(db) if act == "none" else (z[0] > 0).to(torch.bfloat16)
    assert torch.equal(db, 2 * want), (act, db)
    dx = psr.linear_bwd(torch.ones_like(z), one[:2], one, z, activation=act, need_dw=False, need_db=False)[0]
    assert torch.equal(dx, torch.full_like(dx, 8.0 if act == "none" else 4.0)), act


def test_linear_between_columns_of_one_buffer(psr):
    # input, output, z and residual as column ranges of the same rows
    need_gpu()
    for M in (1, 20, 300):
        g = torch.Generator().manual_seed(M)
        rows = randn(g, (M, 136 + 3 * 264), "bf16")
        w, keep = randn(g, (264, 136), "bf16", 0.1), rows.clone()
        cut = lambda t, i: t[:, 136 + 264 * i:136 + 264 * (i + 1)]
        y, z, _ = psr.linear(rows[:, :136], w, None, cut(rows, 2), activation="gelu", out=cut(rows, 0), z=cut(rows, 1))
        check_forward(y, z, keep[:, :136], w, None, cut(keep, 2), "gelu", "bf16", "one buffer")
        assert torch.equal(rows[:, :136], keep[:, :136]) and torch.equal(cut(rows, 2), cut(keep, 2))


@pytest.mark.parametrize("M,N,K", [(1, 264, 136), (12, 72, 64), (1, 301, 515), (70, 264, 136), (600, 1032, 264)])
def test_linear_operands_off_their_boundary(psr, M, N, K):
    need_gpu()
    g = torch.Generator().manual_seed(M + K)
    off = lambda rows, cols, std=1.0: randn(g, (rows * cols + 3,), "bf16", std)[3:].view(rows, cols)
    x, w, dy, z = off(M, K), off(N, K, K**-0.5), off(M, N), off(M, N)
    y, _, ws = psr.linear(x, w, dy[0], z, activation="silu")
    assert psr.get_stats(ws)["status"] == 0
    check_forward(y, None, x, w, dy[0], z, "silu", "bf16", "odd")
    for act in ("none", "silu"):
        got = psr.linear_bwd(dy, x, w, z if act != "none" else None, activation=act)
        assert psr.get_stats(got[3])["status"] == 0
        check_backward(got[:3], dy, x, w, z if act != "none" else None, act, "bf16", "odd bwd")


@pytest.mark.parametrize("K", [8, 248, 256, 264, 2040, 2048, 2056, 4088, 4096, 4104, 6144, 8192, 8200])
def test_linear_one_row_of_any_length(psr, K):
    need_gpu()
    g = torch.Generator().manual_seed(K)
    x, w, b = randn(g, (1, K), "f16"), randn(g, (41, K), "f16", K**-0.5), randn(g, (41,), "f16")
    check_forward(psr.linear(x, w, b)[0], None, x, w, b, None, "none", "f16", str(K))


def test_linear_of_two_streams_at_once(psr):
    need_gpu()
    g = torch.Generator().manual_seed(12)
    calls = [(randn(g, (M, K), "bf16"), randn(g, (N, K), "bf16", K**-0.5), randn(g, (N,), "bf16"), randn(g, (M, N), "bf16"))
             for M, N, K in ((1, 4096, 4096), (24, 4096, 2048), (300, 1024, 4096), (1500, 2048, 512))]
    want = [psr.linear(*c, activation="silu", save_z=True)[:2] for c in calls]
    back = [psr.linear_bwd(c[3], c[0], c[1], y[1], activation="silu")[:3] for c, y in zip(calls, want)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    for _ in range(5):
        got = [psr.linear(*c, activation="silu", save_z=True, stream=s) for c, s in zip(calls, streams)]
        grads = [psr.linear_bwd(c[3], c[0], c[1], y[1], activation="silu", stream=s) for c, y, s in zip(calls, want, streams)]
        torch.cuda.synchronize()
        assert all(psr.get_stats(x[-1])["status"] == 0 for x in got + grads)
        assert all(torch.equal(a, b) for x, y in zip(got, want) for a, b in zip(x, y))
        assert all(torch.equal(a, b) for x, y in zip(grads, back) for a, b in zip(x, y))


# whole rounds of tiles with a last one that is split along K, in two to ten parts, and calls of split tiles only
@pytest.mark.parametrize("M,N,K", [(768, 8192, 2200), (2600, 2304, 2600), (70, 130, 4100), (300, 260, 9000), (520, 1030, 3000),
                                   (257, 20000, 1300)])
def test_linear_split_last_round(psr, M, N, K):
    need_gpu()
    g = torch.Generator().manual_seed(M)
    x, w, b, r = randn(g, (M, K), "bf16"), randn(g, (N, K), "bf16", K**-0.5), randn(g, (N,), "bf16"), randn(g, (M, N), "bf16")
    y, z, ws = psr.linear(x, w, b, r, activation="relu", save_z=True)
    assert psr.get_stats(ws)["status"] == 0
    check_forward(y, z, x, w, b, r, "relu", "bf16", str((M, N, K)))
    got = psr.linear_bwd(r, x, w, need_db=False)
    assert psr.get_stats(got[3])["status"] == 0
    check_backward(got[:3], r, x, w, None, "none", "bf16", str((M, N, K)) + " bwd")


@pytest.mark.parametrize("M,N,K", [(65, 264, 520), (96, 1000, 1032), (127, 4096, 512), (128, 130, 4104), (128, 4104, 520), (112, 64, 2050)])
def test_linear_up_to_128_rows(psr, M, N, K):
    need_gpu()
    g = torch.Generator().manual_seed(M + N)
    x, w, b, r = randn(g, (M, K), "f16"), randn(g, (N, K), "f16", K**-0.5), randn(g, (N,), "f16"), randn(g, (M, N), "f16")
    y, z, ws = psr.linear(x, w, b, r, activation="gelu", save_z=True)
    assert psr.get_stats(ws)["status"] == 0
    check_forward(y, z, x, w, b, r, "gelu", "f16", str((M, N, K)))
    got = psr.linear_bwd(r, x, w, z, activation="gelu")
    assert psr.get_stats(got[3])["status"] == 0
    check_backward(got[:3], r, x, w, z, "gelu", "f16", str((M, N, K)) + " bwd")


@pytest.mark.parametrize("M,N,K", [(4096, 4096, 256), (5000, 2600, 200), (2048, 2560, 4096), (9000, 1100, 64)])
def test_linear_many_tiles_repeat(psr, M, N, K):
    # many tiles to a pair: accumulators and barriers go round, and the same call gives the same bits
    need_gpu()
    g = torch.Generator().manual_seed(K)
    x, w, b, r = randn(g, (M, K), "bf16"), randn(g, (N, K), "bf16", K**-0.5), randn(g, (N,), "bf16"), randn(g, (M, N), "bf16")
    y, z, ws = psr.linear(x, w, b, r, activation="silu", save_z=True)
    z32 = x.float() @ w.float().t() + b.float()
    # z is rounded once (2^-8), and either side's sums are off by at most K 2^-23 sum |x| |w|
    tol = 2.0**-8 * z32.abs() * 1.01 + 2 * K * 2.0**-23 * (x.float().abs() @ w.float().abs().t()) + 1e-6
    assert ((z.float() - z32).abs() <= tol).all()
    for _ in range(20):
        y2, z2, _ = psr.linear(x, w, b, r, activation="silu", save_z=True, workspace=ws)
        assert torch.equal(y, y2) and torch.equal(z, z2)
        assert psr.get_stats(ws)["status"] == 0


@pytest.mark.parametrize("N,K", [(31, 72), (97, 72), (129, 128), (257, 128), (1000, 72), (9741, 520)])  # tiles that are not split
@pytest.mark.parametrize("M", [17, 40, 64])
def test_linear_streamed_last_columns(psr, M, N, K):
    # more than 16 tokens, and a last group of 32 columns that only some of a warp's lanes have
    need_gpu()
    g = torch.Generator().manual_seed(M + N)
    x, w, b, r = randn(g, (M, K), "bf16"), randn(g, (N, K), "bf16", K**-0.5), randn(g, (N,), "bf16"), randn(g, (M, N), "bf16")
    for act in ("gelu", "silu"):
        y, z, ws = psr.linear(x, w, b, r, activation=act, save_z=True)
        assert psr.get_stats(ws)["status"] == 0
        check_forward(y, z, x, w, b, r, act, "bf16", f"{act} {M} x {N} x {K}")


def test_linear_status_of_no_rows(psr):
    # a workspace that holds anything, and one on another stream
    need_gpu()
    x, w = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda"), torch.ones((16, 64), dtype=torch.bfloat16, device="cuda")
    dy, side = torch.empty((0, 16), dtype=torch.bfloat16, device="cuda"), torch.cuda.Stream()
    for stream in (None, side):
        for dtype in (torch.uint8, torch.float32):
            size = max(psr.linear_workspace_bytes(0, 16, 64), psr.linear_workspace_bytes(0, 16, 64, backward=True))
            for call in (lambda ws: psr.linear(x, w, workspace=ws, stream=stream), lambda ws: psr.linear_bwd(dy, x, w, workspace=ws, stream=stream)):
                ws = torch.full((size,), 0xFF, dtype=torch.uint8, device="cuda").view(dtype)
                side.wait_stream(torch.cuda.current_stream())
                assert call(ws)[-1] is ws
                torch.cuda.synchronize()
                assert psr.get_stats(ws)["status"] == 0 and psr.get_stats(ws)["error_site"] == 0


# A one-hot x makes z an exact grid.  gelu = z Phi(z): the kernel's Phi is off by 4e-5 of itself, and the exponent of its tail, up
# to 104 in powers of two, by three roundings of 2^-24 of that, 1.3e-5 together; 2^-14 bounds the two.  The slope is Phi + z phi with
# the same two bounds on its terms.  Results below the smallest normal number may be flushed.
@pytest.mark.parametrize("t", ["bf16", "f16"])
@pytest.mark.parametrize("M", [1, 40, 300])
def test_gelu_keeps_the_digits_of_its_tails(psr, t, M):
    from layer_util import TYPES
    need_gpu()
    grid = torch.linspace(-12, 12, 4801, dtype=torch.float64).to(TYPES[t])
    w = torch.zeros((len(grid), 64), dtype=TYPES[t])
    w[:, 0] = grid
    x = torch.zeros((M, 64), dtype=TYPES[t])
    x[:, 0] = 1
    y, z, _ = psr.linear(x.cuda(), w.cuda(), activation="gelu", save_z=True)
    assert torch.equal(z, grid.cuda().expand(M, -1))
    g = f64(grid)
    want = ol.act(g, "gelu")
    tiny = TINY[t] + 2.0**-120
    check(y, np.broadcast_to(want, (M, len(g))), np.abs(want) * (ol.HALF_STEP[t] * 1.01 + 2.0**-14) + tiny, "gelu")
    db = psr.linear_bwd(torch.ones_like(z), x.cuda(), w.cuda(), z, activation="gelu", need_dx=False, need_dw=False)[2]
    slope, phi = ol.act_slope(g, "gelu"), np.exp(-g * g / 2) / np.sqrt(2 * np.pi)
    terms = want / np.where(g == 0, 1, g) + np.abs(g) * phi
    # over M rows the sum has M - 1 roundings of 2^-24 as well
    check(db, M * slope, M * np.abs(slope) * (ol.HALF_STEP[t] * 1.01 + M * 2.0**-24) + M * 2.0**-14 * terms + tiny, "slope")


def test_linear_bwd_of_very_many_columns(psr):
    # 65536 blocks of 32 columns where rows are not on 16-byte boundaries, two chunks of rows
    need_gpu()
    M, N, K = 66, 32 * 65535 + 1, 8
    g = torch.Generator().manual_seed(8)
    dy, x, w, z = randn(g, (M, N), "bf16"), randn(g, (M, K), "bf16"), randn(g, (N, K), "bf16"), randn(g, (M, N), "bf16")
    dx, dw, db, ws = psr.linear_bwd(dy, x, w, z, activation="silu")
    assert psr.get_stats(ws)["status"] == 0
    got = dx, dw[-300:], db[-300:]
    check_backward((None, dw[:300], db[:300]), dy[:, :300], x, w[:300], z[:, :300], "silu", "bf16", "first columns")
    check_backward((None, *got[1:]), dy[:, -300:], x, w[-300:], z[:, -300:], "silu", "bf16", "last columns")
    s = torch.sigmoid(z.float())
    dz = (dy.float() * s * (1 + z.float() * (1 - s))).to(torch.bfloat16).double()
    want = dz @ w.double()
    # dz may have been rounded the other way (2^-8 of it, random signs: 2^-8 of the root of the sum of squares, by 6), sums of N
    # products in fp32 drift by 2^-24 of their size a step (random signs again), and the result is rounded
    size = ((dz**2) @ (w.double()**2)).sqrt()
    assert ((dx.double() - want).abs() <= 2.0**-8 * want.abs() * 1.01 + (6 * 2.0**-8 + 2.0**-24 * N**0.5) * size).all()
