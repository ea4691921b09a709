"""GPU tests of psr_xent and psr_xent_bwd against the fp64 oracle, through the binding.

Tolerance.  A logit, an fp32 sum of K products, is off by at most e = K 2^-23 sum |x| |w| (each addition rounds or truncates).
lse moves by at most the largest e of its row, plus the roundings of the sum of exponentials: the exponent's (2^-23 of |l| + |lse|, in
units of 1), the exponential's (2^-22) and those of up to 2^10 additions one after another (2^-24 each): below 2^-13 in all,
and one of lse itself.  The loss adds e of the target, the smoothed mean e of all.  Slopes: p moves by p times what l and lse move,
the fp32 arithmetic adds 2^-22 of the row's g (1 + 2 z |lse|), and the slope is rounded once to the type (fp16: its subnormal numbers
are 2^-24, 2^-13 of g max): half a step.  These carry through the products with |w| and |x|, whose own sums are fp32, and the
result is rounded once.
"""
import numpy as np
import pytest
import torch

from layer_util import check, f64, need_gpu, randn
from oracle import ends, layer as ol

pytestmark = pytest.mark.gpu

TINY = {"bf16": 0.0, "f16": 2.0**-25}


def logit_error(x, w):
    return x.shape[1] * 2.0**-23 * (np.abs(x) @ np.abs(w).T)


def clean(x, t, V, ignore):
    """x with zeros in the rows that do not count: whatever stands there has no part in anything."""
    x = x.copy()
    x[[i for i, v in enumerate(t) if v == ignore or not 0 <= v < V]] = 0
    return x


def check_loss(loss, lse, x, w, t, what, smoothing=0.0, z=0.0, ignore=-100):
    t = t.tolist()
    xs, ws = clean(f64(x), t, len(w), ignore), f64(w)
    ref, ref_lse = ends.linear_xent(xs, ws, t, smoothing, z, ignore)
    e = logit_error(xs, ws).max(1)
    tol = e + 2.0**-13 + 2.0**-23 * np.abs(ref_lse)
    check(lse, ref_lse, tol, what + " lse")
    size = np.abs(xs @ ws.T).max(1)
    check(loss, ref, tol * (1 + 2 * z * np.abs(ref_lse)) + e + 2.0**-23 * (np.abs(ref) + size), what + " loss")


def check_gradients(dx, dw, dloss, x, w, t, lse, typ, what, smoothing=0.0, z=0.0, ignore=-100):
    t, g = t.tolist(), f64(dloss)
    xs, ws, ls = clean(f64(x), t, len(w), ignore), f64(w), f64(lse)
    counts = np.array([v != ignore and 0 <= v < len(w) for v in t])
    g, ls = np.where(counts, g, 0.0), np.where(counts, ls, 0.0)
    d, p = ends.xent_slope(g, xs, ws, t, ls, smoothing, z, ignore)
    h = ol.HALF_STEP[typ]
    top = (np.abs(g) * (1 + 2 * z * np.abs(ls)))[:, None]
    e = logit_error(xs, ws) + 2.0**-22 + 2.0**-23 * (np.abs(xs @ ws.T) + np.abs(ls)[:, None])
    ed = top * (p * np.expm1(e) + 2.0**-22) + 1.01 * h * np.abs(d) + (2.0**-38 * top.max() if typ == "f16" else 0.0)
    ed[~counts] = 0
    M, V = d.shape
    if dx is not None:
        ref = d @ ws
        tol = ed @ np.abs(ws) + V * 2.0**-23 * (np.abs(d) @ np.abs(ws)) + h * 1.01 * np.abs(ref) + TINY[typ]
        check(dx, ref, tol, what + " dx")
        assert not f64(dx)[~counts].any(), what
    if dw is not None:
        ref = d.T @ xs
        tol = ed.T @ np.abs(xs) + M * 2.0**-23 * (np.abs(d).T @ np.abs(xs)) + h * 1.01 * np.abs(ref) + TINY[typ]
        check(dw, ref, tol, what + " dw")


def inputs(gen, M, V, K, t, drop=0.0, spread=2.5):
    x, w = randn(gen, (M, K), t), randn(gen, (V, K), t, spread * K**-0.5)
    targets = torch.randint(0, V, (M,), generator=gen)
    if drop:
        targets[torch.rand(M, generator=gen) < drop] = -100
    g = torch.rand(M, generator=gen) * (2.0 if t == "bf16" else 2000.0)
    return x, w, targets.cuda(), g.cuda()


CASES = [  # M V K smoothing z drop type
    (1, 1, 1, 0.0, 0.0, 0.0, "bf16"), (1, 2, 8, 0.0, 0.0, 0.0, "f16"), (1, 300, 17, 0.1, 0.0, 0.0, "bf16"),
    (1, 5000, 64, 0.1, 1e-3, 0.0, "bf16"), (1, 1000, 2056, 0.0, 0.0, 0.0, "f16"), (1, 777, 4104, 0.0, 0.0, 0.0, "bf16"),
    (2, 33, 40, 0.0, 0.0, 0.0, "bf16"), (3, 127, 515, 0.2, 0.0, 0.3, "f16"), (5, 1001, 264, 0.0, 1e-2, 0.3, "bf16"),
    (16, 4096, 128, 0.0, 0.0, 0.0, "bf16"), (17, 40000, 72, 0.0, 0.0, 0.4, "bf16"), (40, 260, 1000, 0.1, 0.0, 0.0, "f16"),
    (63, 129, 64, 0.0, 0.0, 0.5, "bf16"), (64, 3001, 520, 0.0, 0.0, 0.0, "bf16"),
    (65, 1, 8, 0.0, 0.0, 0.0, "bf16"), (65, 2, 64, 0.0, 0.0, 0.0, "f16"), (66, 255, 17, 0.1, 0.0, 0.3, "bf16"),
    (70, 256, 515, 0.0, 0.0, 0.0, "f16"), (128, 257, 64, 0.0, 0.0, 0.0, "bf16"), (200, 5001, 72, 0.0, 1e-2, 0.5, "bf16"),
    (256, 512, 256, 0.1, 0.0, 0.0, "bf16"), (257, 777, 200, 0.0, 0.0, 0.1, "f16"), (300, 20000, 40, 0.0, 0.0, 0.0, "bf16"),
    (513, 264, 1000, 0.1, 1e-3, 0.7, "f16"), (900, 4100, 136, 0.0, 0.0, 0.0, "f16"), (1300, 901, 77, 0.0, 0.0, 0.6, "bf16"),
    (2600, 300, 8, 0.0, 0.0, 0.9, "bf16")]


@pytest.mark.parametrize("case", CASES, ids=str)
def test_loss_and_gradients(psr, case):
    need_gpu()
    M, V, K, smoothing, z, drop, t = case
    gen = torch.Generator().manual_seed(M * 3 + V + K)
    x, w, targets, g = inputs(gen, M, V, K, t, drop)
    more = dict(smoothing=smoothing, z_weight=z)
    loss, lse, ws = psr.linear_xent(x, w, targets, **more)
    assert psr.get_stats(ws)["status"] == 0
    check_loss(loss, lse, x, w, targets, str(case), smoothing, z)
    dx, dw, ws = psr.linear_xent_bwd(g, x, w, targets, lse, **more)
    assert psr.get_stats(ws)["status"] == 0
    check_gradients(dx, dw, g, x, w, targets, lse, t, str(case), smoothing, z)
    again = psr.linear_xent_bwd(g, x, w, targets, lse, workspace=ws, **more)
    assert torch.equal(again[0], dx) and torch.equal(again[1], dw)
    only, none, _ = psr.linear_xent_bwd(g, x, w, targets, lse, need_dw=False, **more)
    assert none is None and torch.equal(only, dx)
    none, only, _ = psr.linear_xent_bwd(g, x, w, targets, lse, need_dx=False, **more)
    assert none is None and torch.equal(only, dw)


@pytest.mark.parametrize("M", [1, 7, 64, 65, 300])
def test_rows_that_do_not_count(psr, M):
    """All, none or a few of the rows ignored, bad targets, and NaN or infinities where nothing may be read."""
    need_gpu()
    gen = torch.Generator().manual_seed(M)
    V, K = 333, 72
    x, w, targets, g = inputs(gen, M, V, K, "bf16")
    for drop in (list(range(M)), list(range(1, M)), list(range(0, M, 2))):
        t = targets.clone()
        t[drop] = torch.tensor(([5, -1, V, 2**40, -2**62, 5, 5] * M)[:len(drop)], dtype=torch.int64).cuda()
        t[[i for i in range(M) if i not in drop and t[i] == 5]] = 6
        y, gg = x.clone(), g.clone()
        y[drop] = float("nan")
        gg[drop] = float("inf")
        loss, lse, _ = psr.linear_xent(y, w, t, ignore=5)
        check_loss(loss, lse, y, w, t, f"{M} {len(drop)}", ignore=5)
        dx, dw, _ = psr.linear_xent_bwd(gg, y, w, t, lse, ignore=5)
        check_gradients(dx, dw, gg, y, w, t, lse, "bf16", f"{M} {len(drop)}", ignore=5)


def test_views_and_broadcasts(psr):
    need_gpu()
    gen = torch.Generator().manual_seed(2)
    for M in (9, 130):
        V, K = 401, 96
        x, w, _, _ = inputs(gen, M, V, K, "bf16")
        bx, bw = randn(gen, (M, 2 * K), "bf16"), randn(gen, (V, K + 5), "bf16")
        bx[:, 8:8 + K], bw[:, 3:3 + K] = x, w
        vx, vw = bx[:, 8:8 + K], bw[:, 3:3 + K]
        tokens = torch.randint(0, V, (M, 3), generator=gen).cuda()
        t, g = tokens[:, 1], torch.full((1,), 0.125, device="cuda").expand(M)
        loss, lse = torch.full((2, M + 1), 7.0, device="cuda")[:, :M]
        got = psr.linear_xent(vx, vw, t, loss=loss, lse=lse)
        assert got[0] is loss and got[1] is lse
        check_loss(loss, lse, x, w, t, "views")
        dx, dw = torch.empty_like(x), torch.empty_like(w)
        got = psr.linear_xent_bwd(g, vx, vw, t, lse, dx=dx, dw=dw)
        assert got[0] is dx and got[1] is dw
        check_gradients(dx, dw, g, x, w, t, lse, "bf16", "views")
        same = torch.tensor([4]).cuda().expand(M)
        check_loss(*psr.linear_xent(x, w, same)[:2], x, w, same, "one target")
        odd = [torch.empty(n * K + 1, dtype=x.dtype, device="cuda")[1:].view(n, K) for n in (M, V)]  # off every boundary
        psr.linear_xent_bwd(g, x, w, t, lse, dx=odd[0], dw=odd[1])
        assert torch.equal(odd[0], dx) and torch.equal(odd[1], dw)


@pytest.mark.parametrize("M", [3, 100])
def test_far_logits(psr, M):
    """Logits of hundreds of either sign: the sums of exponentials take their references from them."""
    need_gpu()
    gen = torch.Generator().manual_seed(9)
    x, w, t, g = inputs(gen, M, 1000, 64, "bf16", spread=80.0)
    for shift in (0.0, -600.0, 600.0):
        y, v = x.clone(), w.clone()
        y[:, 0], v[:, 0] = 1.0, shift
        loss, lse, _ = psr.linear_xent(y, v, t)
        check_loss(loss, lse, y, v, t, str(shift))
        dx, dw, _ = psr.linear_xent_bwd(g, y, v, t, lse)
        check_gradients(dx, dw, g, y, v, t, lse, "bf16", str(shift))


@pytest.mark.parametrize("M", [1, 3, 100])
def test_infinite_logits(psr, M):
    need_gpu()
    x = torch.ones((M, 8), dtype=torch.bfloat16, device="cuda")
    w = torch.zeros((300, 8), dtype=torch.bfloat16, device="cuda")
    t = torch.zeros(M, dtype=torch.int64, device="cuda")
    w[7, 0] = -float("inf")  # a column out of reach
    loss, lse, _ = psr.linear_xent(x, w, t)
    assert torch.allclose(lse.cpu(), torch.full((M,), float(np.log(299))), atol=1e-5) and torch.allclose(loss, lse)
    w[8, 0] = float("inf")
    loss, lse, _ = psr.linear_xent(x, w, t)
    assert (lse == float("inf")).all() and (loss == float("inf")).all()
    w[9, 0] = float("nan")
    loss, lse, _ = psr.linear_xent(x, w, t)
    assert lse.isnan().all() and loss.isnan().all()


def test_small_gradients_in_fp16(psr):
    """Probabilities of 1e-6 and a loss weight of 1e-4: below fp16's numbers, were the slopes not scaled."""
    need_gpu()
    gen = torch.Generator().manual_seed(11)
    for M in (20, 200):
        x, w, t, _ = inputs(gen, M, 20000, 64, "f16", spread=0.5)
        g = torch.full((M,), 0.5, device="cuda")
        _, lse, _ = psr.linear_xent(x, w, t)
        dx, dw, _ = psr.linear_xent_bwd(g, x, w, t, lse)
        small, _, _ = psr.linear_xent_bwd(g * 2.0**-13, x, w, t, lse, need_dw=False)
        d, _ = ends.xent_slope(f64(g), f64(x), f64(w), t.tolist(), f64(lse))
        ref = d @ f64(w)
        err = np.abs(f64(dx) - ref).max() / np.abs(ref).max()
        assert err < 2.0**-9, err  # two roundings of 2^-11, the slopes' and the result's, and fp32 sums
        assert np.abs(f64(small) * 2.0**13 - f64(dx)).max() <= 2.0**-12 + 2.0**-10 * np.abs(f64(dx)).max()


def test_gradients_are_differences(psr):
    """Along random directions of x and w, in steps that 16-bit inputs hold exactly."""
    need_gpu()
    gen = torch.Generator().manual_seed(12)
    for M in (8, 90):
        V, K, more = 200, 32, dict(smoothing=0.1, z_weight=1e-2)
        grid = lambda *s: (torch.randint(-16, 17, s, generator=gen) / 16).to(torch.bfloat16).cuda()
        x, w = grid(M, K), grid(V, K)
        t, g = torch.randint(0, V, (M,), generator=gen).cuda(), torch.rand(M, generator=gen).cuda()
        _, lse, _ = psr.linear_xent(x, w, t, **more)
        dx, dw, _ = psr.linear_xent_bwd(g, x, w, t, lse, **more)
        sx, sw = (torch.randint(-1, 2, s, generator=gen).to(torch.bfloat16).cuda() for s in ((M, K), (V, K)))
        h = 2.0**-6
        f = lambda a: (f64(psr.linear_xent(x + a * h * sx, w + a * h * sw, t, **more)[0]) * f64(g)).sum()
        slope = (f(1) - f(-1)) / (2 * h)
        want = (f64(dx) * f64(sx)).sum() + (f64(dw) * f64(sw)).sum()
        # gradients rounded to bf16 twice (2^-8 each); the difference's own error: a third of h^2 of the third derivative along
        # the directions (|s . x| up to some 30), and roundings of the losses over h
        size = (np.abs(f64(dx)) * np.abs(f64(sx))).sum() + (np.abs(f64(dw)) * np.abs(f64(sw))).sum()
        assert abs(slope - want) <= 2.0**-7 * size, (slope, want, size)


def test_pieces_of_the_vocabulary(psr):
    """Slopes of more bytes than a piece may have: dx is summed over pieces.  (The reference in 64 bits on the device.)"""
    need_gpu()
    gen = torch.Generator().manual_seed(13)
    M, V, K = 40000, 9001, 24
    x, w, t, g = inputs(gen, M, V, K, "bf16", drop=0.2)
    loss, lse, _ = psr.linear_xent(x, w, t)
    dx, dw, ws = psr.linear_xent_bwd(g, x, w, t, lse)
    assert psr.get_stats(ws)["status"] == 0
    keep = t != -100
    x8, w8 = x[keep].double(), w.double()
    l8 = x8 @ w8.T
    at = t[keep][:, None]
    lse8 = l8.logsumexp(1)
    assert (lse[keep].double() - lse8).abs().max() < 2.0**-13 and not lse[~keep].any()
    assert (loss[keep].double() - lse8 + l8.gather(1, at)[:, 0]).abs().max() < 2.0**-12 and not loss[~keep].any()
    d = (l8 - lse[keep].double()[:, None]).exp_()
    d.scatter_add_(1, at, torch.full((len(x8), 1), -1.0, dtype=torch.float64, device="cuda"))
    d *= g[keep].double()[:, None]
    rx, rw = d @ w8, d.T @ x8
    a = d.abs_()
    for got, ref, size in ((dx[keep], rx, a @ w8.abs()), (dw, rw, a.T @ x8.abs())):
        # a slope: half a step of bf16 and 2^-12 of p; the sums: fp32; the result: half a step
        tol = (2.0**-8 * 1.01 + 2.0**-11) * size + 2.0**-8 * 1.01 * ref.abs() + 2.0**-18 * size
        assert ((got.double() - ref).abs() <= tol).all()
    assert not dx[~keep].any()


@pytest.mark.parametrize("M", [1, 16, 64, 70])
def test_rows_off_boundaries_among_nan(psr, M):
    """W and x as views whose rows begin and end anywhere, with NaN between, before and behind them."""
    need_gpu()
    gen = torch.Generator().manual_seed(30 + M)
    for V, K, gap, t in ((129, 515, 0, "bf16"), (1000, 136, 3, "f16"), (257, 1029, 2, "bf16"), (128, 128, 1, "bf16"), (600, 260, 4, "f16")):
        x, w, targets, g = inputs(gen, M, V, K, t)
        views = []
        for m in (x, w):
            n = len(m)
            buffer = torch.full((n * (K + gap) + 7,), float("nan"), dtype=m.dtype, device="cuda")
            view = buffer[5:5 + n * (K + gap)].view(n, K + gap)[:, :K]
            view.copy_(m)
            views.append(view)
        loss, lse, ws = psr.linear_xent(*views, targets)
        assert psr.get_stats(ws)["status"] == 0
        check_loss(loss, lse, x, w, targets, str((V, K)))
        dx, dw, ws = psr.linear_xent_bwd(g, *views, targets, lse)
        assert psr.get_stats(ws)["status"] == 0
        check_gradients(dx, dw, g, x, w, targets, lse, t, str((V, K)))


@pytest.mark.parametrize("M", [40, 64, 65, 128, 129])
def test_gradients_leave_what_stands_around_them(psr, M):
    """Blocks of dx and dw that end inside a tile, in buffers whose other bytes stay as they were, with any number of rows that count."""
    need_gpu()
    gen = torch.Generator().manual_seed(21 + M)
    for V, K, drop in ((33, 8, 0.0), (300, 264, 0.5), (513, 40, 1.1)):
        x, w, targets, g = inputs(gen, M, V, K, "bf16", drop)
        _, lse, _ = psr.linear_xent(x, w, targets)
        buffers = [torch.full((n * K + 128,), 7.0, dtype=x.dtype, device="cuda") for n in (M, V)]
        dx, dw = (b[64:-64].view(n, K) for b, n in zip(buffers, (M, V)))
        psr.linear_xent_bwd(g, x, w, targets, lse, dx=dx, dw=dw)
        check_gradients(dx, dw, g, x, w, targets, lse, "bf16", str((V, K)))
        for b in buffers:
            assert (b[:64] == 7).all() and (b[-64:] == 7).all()


def test_few_rows_of_dx_split_and_joined(psr):
    """dx of few tiles and a long vocabulary: parts of the sum over V, joined, with fewer rows than the host knows of."""
    need_gpu()
    gen = torch.Generator().manual_seed(14)
    for drop, t in ((0.0, "bf16"), (0.8, "f16")):
        x, w, targets, g = inputs(gen, 700, 12000, 264, t, drop)
        _, lse, _ = psr.linear_xent(x, w, targets)
        dx, dw, ws = psr.linear_xent_bwd(g, x, w, targets, lse)
        assert psr.get_stats(ws)["status"] == 0
        check_gradients(dx, dw, g, x, w, targets, lse, t, str(drop))


@pytest.mark.parametrize("M", [4, 150])
def test_streams_and_graphs(psr, M):
    need_gpu()
    gen = torch.Generator().manual_seed(15)
    V, K = 3000, 128
    x, w, t, g = inputs(gen, M, V, K, "bf16", 0.3)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    loss, lse, _ = psr.linear_xent(x, w, t, stream=side)
    dx, dw, _ = psr.linear_xent_bwd(g, x, w, t, lse, stream=side)
    side.synchronize()
    check_loss(loss, lse, x, w, t, "side stream")
    check_gradients(dx, dw, g, x, w, t, lse, "bf16", "side stream")
    ws = [torch.empty(psr.linear_xent_workspace_bytes(M, V, K, backward=b), dtype=torch.uint8, device="cuda") for b in (False, True)]
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        psr.linear_xent(x, w, t, loss=loss, lse=lse, workspace=ws[0])
        psr.linear_xent_bwd(g, x, w, t, lse, dx=dx, dw=dw, workspace=ws[1])
    for drop in (0.0, 0.9, 1.1):  # the rows that count are counted at each replay
        nx, _, nt, ng = inputs(gen, M, V, K, "bf16", drop)
        x.copy_(nx), t.copy_(nt), g.copy_(ng)
        graph.replay()
        torch.cuda.synchronize()
        check_loss(loss, lse, x, w, t, f"replay {drop}")
        check_gradients(dx, dw, g, x, w, t, lse, "bf16", f"replay {drop}")


def test_two_calls_at_once(psr):
    """Calls of different sizes on two streams, each with a workspace of its own, give the bits that they give alone."""
    need_gpu()
    gen = torch.Generator().manual_seed(17)
    sets = [inputs(gen, M, V, 128, "bf16", 0.2) for M, V in ((40, 9000), (700, 5000))]
    streams = [torch.cuda.Stream() for _ in sets]

    def run(i, stream):
        x, w, t, g = sets[i]
        loss, lse, _ = psr.linear_xent(x, w, t, stream=stream)
        dx, dw, _ = psr.linear_xent_bwd(g, x, w, t, lse, stream=stream)
        de, _ = psr.embedding_bwd(dx, t, len(w), dw=dw.clone() if stream is None else None, stream=stream)
        return loss, lse, dx, dw, de
    alone = [run(i, None) for i in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        both = [run(i, streams[i]) for i in range(2)]
        torch.cuda.synchronize()
        for a, b in zip(alone, both):
            assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_the_two_ends_with_one_table(psr):
    """Tokens to rows, rows to a loss, and back: a table shared by both ends gets both gradients."""
    need_gpu()
    gen = torch.Generator().manual_seed(16)
    M, V, K = 300, 500, 64
    table = randn(gen, (V, K), "bf16", 0.3)
    ids, t = (torch.randint(0, V, (M,), generator=gen).cuda() for _ in range(2))
    g = torch.full((1,), 1.0 / M, device="cuda").expand(M)
    x = psr.embedding(ids, table, scale=2.0)
    loss, lse, _ = psr.linear_xent(x, table, t)
    dx, dw, _ = psr.linear_xent_bwd(g, x, table, t, lse)
    head = f64(dw).copy()
    psr.embedding_bwd(dx, ids, V, scale=2.0, dw=dw, accumulate=True)
    check_loss(loss, lse, x, table, t, "tied")
    ref, n, size = ends.embedding_bwd(f64(dx), ids.tolist(), V, 2.0, None, head)
    check(dw, ref, (n[:, None] + 3) * 2.0**-24 * size + 2.0**-8 * 1.01 * np.abs(ref), "tied dw")


def test_no_rows(psr):
    need_gpu()
    z = lambda *s, t=torch.bfloat16: torch.zeros(s, dtype=t, device="cuda")
    loss, lse, ws = psr.linear_xent(z(0, 8), z(20, 8), z(0, t=torch.int64))
    assert loss.shape == lse.shape == (0,) and psr.get_stats(ws)["status"] == 0
    dw = torch.ones_like(z(20, 8))
    dx, _, ws = psr.linear_xent_bwd(z(0, t=torch.float32), z(0, 8), z(20, 8), z(0, t=torch.int64), lse, dw=dw)
    assert dx.shape == (0, 8) and not dw.any() and psr.get_stats(ws)["status"] == 0


def test_refusals(psr):
    need_gpu()
    z = lambda *s, t=torch.bfloat16: torch.zeros(s, dtype=t, device="cuda")
    x, w, t, g = z(4, 16), z(9, 16), z(4, t=torch.int64), z(4, t=torch.float32)
    for call in (lambda: psr.linear_xent(x.float(), w.float(), t), lambda: psr.linear_xent(x, w.half(), t),
                 lambda: psr.linear_xent(x, z(9, 8), t), lambda: psr.linear_xent(x, w, t.int()), lambda: psr.linear_xent(x, w, t[:3]),
                 lambda: psr.linear_xent(x.cpu(), w, t), lambda: psr.linear_xent(x, w, t, loss=g.double()),
                 lambda: psr.linear_xent(x, w, t, loss=g, lse=g), lambda: psr.linear_xent(x, w, t, workspace=z(9, t=torch.uint8)),
                 lambda: psr.linear_xent_bwd(g.half(), x, w, t, g), lambda: psr.linear_xent_bwd(g, x, w, t, g[:2]),
                 lambda: psr.linear_xent_bwd(g, x, w, t, g, dx=z(4, 17)), lambda: psr.linear_xent_bwd(g, x, w, t, g, dw=w),
                 lambda: psr.linear_xent_bwd(g, x, w, t, g, dw=z(16, 9).t())):
        with pytest.raises(ValueError):
            call()
    for more in (dict(smoothing=1.0), dict(smoothing=-0.1), dict(smoothing=float("nan")), dict(z_weight=-1.0),
                 dict(z_weight=float("inf"))):
        with pytest.raises(psr.PsrError):
            psr.linear_xent(x, w, t, **more)
        with pytest.raises(psr.PsrError):
            psr.linear_xent_bwd(g, x, w, t, g, **more)


@pytest.mark.parametrize("t", ["bf16", "f16"])
@pytest.mark.parametrize("M", [2, 7, 40, 64, 65, 300])
def test_rows_that_do_not_count_among_infinite_weights(psr, M, t):
    """A weight that is infinite or NaN stays out of the gradients of rows without a target, and of dw through them."""
    need_gpu()
    gen = torch.Generator().manual_seed(M)
    for V, K in ((333, 72), (261, 67)):  # W on 16-byte boundaries and off them
        x, w, targets, g = inputs(gen, M, V, K, t)
        targets[targets == 7] = 8
        # logits of -inf at column 7 in every row that counts: its probability is 0, so dw is finite, and dx (0 times -inf) NaN
        x[:, 3] = x[:, 3].abs() + 1
        w[7, 3] = -float("inf")
        drop = list(range(0, M, 2))
        targets[drop] = torch.tensor(([-100, V, -1] * M)[:len(drop)], dtype=torch.int64).cuda()
        x[drop] = float("nan")
        loss, lse, _ = psr.linear_xent(x, w, targets)
        dx, dw, ws = psr.linear_xent_bwd(g, x, w, targets, lse)
        assert psr.get_stats(ws)["status"] == 0
        keep = np.setdiff1d(np.arange(M), drop)
        assert not f64(dx)[drop].any()
        assert np.isnan(f64(dx)[keep, 3]).all() and np.isfinite(np.delete(f64(dx)[keep], 3, 1)).all()
        assert not f64(dw)[7].any()
        finite = w.clone()
        finite[7] = 0  # (no probability and no target: for dw's other rows any weights do, with these lse)
        check_gradients(None, torch.cat((dw[:7], dw[8:])), g, x, torch.cat((finite[:7], finite[8:])),
                        torch.where(targets > 7, targets - 1, targets), lse, t, str((V, K)))
        w[9, 1], w[10, 2] = float("nan"), float("inf")
        targets.fill_(-100)
        loss, lse, _ = psr.linear_xent(x, w, targets)
        dx, dw, _ = psr.linear_xent_bwd(g, x, w, targets, lse)
        assert not loss.any() and not lse.any() and not dx.any() and not dw.any()


@pytest.mark.parametrize("t", ["bf16", "f16"])
@pytest.mark.parametrize("M", [5, 90])
def test_gradients_of_the_smallest_weights_of_the_loss(psr, M, t):
    """dloss down to fp32's smallest number, which times (1 - smoothing) is none: gradients that round to zero, and no NaN."""
    need_gpu()
    gen = torch.Generator().manual_seed(M)
    x, w, targets, _ = inputs(gen, M, 200, 40, t)
    for g, smoothing in ((2.0**-149, 0.75), (2.0**-149, 0.0), (2.0**-126, 0.75), (2.0**-100, 0.1)):
        g = torch.full((M,), g, device="cuda")
        _, lse, _ = psr.linear_xent(x, w, targets, smoothing=smoothing)
        dx, dw, _ = psr.linear_xent_bwd(g, x, w, targets, lse, smoothing=smoothing)
        for got in (dx, dw):  # slopes are at most 2 g, |x| and |w| below 8, sums of 200 terms
            assert (got.double().abs() <= g[0].item() * 2 * 8 * 200).all()


@pytest.mark.parametrize("M", [6, 100])
def test_smoothed_slopes_fit_fp16(psr, M):
    """Much smoothing of few columns with a penalty under which 1 + 2 z lse vanishes: the smoothing's share is then the largest slope."""
    need_gpu()
    gen = torch.Generator().manual_seed(M)
    for V, smoothing in ((1, 0.96875), (2, 0.9375), (3, 0.984375)):
        x = torch.randint(-2, 3, (M, 8), generator=gen).half().cuda() / 32
        w = torch.randint(-2, 3, (V, 8), generator=gen).half().cuda() / 4
        x[:, 0], w[:, 0] = 2.0, -1.0 - float(np.log(V)) / 2  # lse near -2
        targets, g = torch.randint(0, V, (M,), generator=gen).cuda(), torch.rand(M, generator=gen).cuda() + 0.5
        more = dict(smoothing=smoothing, z_weight=0.25)
        _, lse, _ = psr.linear_xent(x, w, targets, **more)
        assert (1 + 0.5 * lse).abs().max() < 0.1
        dx, dw, _ = psr.linear_xent_bwd(g, x, w, targets, lse, **more)
        check_gradients(dx, dw, g, x, w, targets, lse, "f16", str(V), smoothing, 0.25)


@pytest.mark.parametrize("M,K", [(1, 16384), (1, 16383), (40, 8192), (2, 16384), (40, 16384), (64, 32768), (17, 20488), (33, 16383), (40, 4096),
                                 (65, 16384), (300, 8192), (100, 16383)])
def test_long_logits_are_summed_in_parts(psr, M, K):
    """Sums of 1024 products that fp32 holds exactly, and longer ones that it does not: the logits are as exact as the additions of the parts.

    Products are integers (times a power of two): 512 pairs of 256 a + b, 64 <= a < 128, 0 <= b < 256, sum to less than 2^24, so a part of
    1024 has no rounding.  Adding n parts, or parts of parts, of sum L rounds by at most 2^-24 (2 + ... + n) / n of L: below 2^-24 (n + 3) / 2.
    lse moves by no more; the sums of exponentials of near logits, with at most 2^6 additions one after another (2^-24 each) and up to 32
    factors of ex2's (2^-22 each), give 2^-16, log2(e) and the result's rounding 2^-24 and 2^-23 of lse.  (Sums of 4096 products, whose
    last bits the tensor core cuts, come out too small by up to twice what is allowed at K = 16384, of 8192 products by six times.)
    """
    need_gpu()
    gen = torch.Generator(device="cuda").manual_seed(K + M)
    V = 20000  # more tiles than SMs: few rows' tiles are whole
    a = torch.randint(64, 128, (V, (K + 1) // 2), generator=gen, device="cuda") * 256
    b = torch.randint(0, 256, (V, (K + 1) // 2), generator=gen, device="cuda")
    w = (torch.stack((a, b), 2).view(V, -1)[:, :K] * 2.0**-21).to(torch.bfloat16).contiguous()
    power = torch.randint(-1, 1, (M, 1), generator=gen, device="cuda")
    x = (2.0**power).to(torch.bfloat16).expand(M, K).contiguous()
    t = torch.randint(0, V, (M,), generator=gen, device="cuda")
    loss, lse, ws = psr.linear_xent(x, w, t)
    assert psr.get_stats(ws)["status"] == 0
    logits = 2.0**power.double() * w.double().sum(1)
    ref = logits.logsumexp(1)
    parts = -(-K // 1024)
    most = 2.0**-24 * (parts + 3) / 2 * logits.amax(1)
    tol = most + 2.0**-16 + (2.0**-23 + 2.0**-24) * ref.abs()
    err = (lse.double() - ref).abs()
    assert (err <= tol).all(), (err / tol).max().item()
    at = logits.gather(1, t[:, None])[:, 0]
    err, tol = (loss.double() - (ref - at)).abs(), tol + most
    assert (err <= tol).all(), (err / tol).max().item()


def check_on_device(dx, dw, g, x, w, t, lse, typ, smoothing=0.0, z=0.0):
    """check_gradients for sizes that numpy takes too long for, with the same tolerance but for the logits: they, and lse, are
    off by 2^-12 at most (64 sums of 16 products to a part, each cut by less than 2^-23 of sums below 30)."""
    h, tiny = ol.HALF_STEP[typ], TINY[typ]
    keep = t != -100
    x8, w8, g8, l8, at = x[keep].double(), w.double(), g[keep].double(), lse[keep].double(), t[keep][:, None]
    p = (x8 @ w8.T - l8[:, None]).exp_()
    top = g8[:, None] * (1 + 2 * z * l8.abs())[:, None]
    ed = top * (p * 2.0**-11 + 2.0**-22)
    d = p.mul_((1 + 2 * z * l8)[:, None]).sub_(smoothing / len(w))
    d.scatter_add_(1, at, torch.full((len(x8), 1), smoothing - 1.0, dtype=torch.float64, device="cuda"))
    d *= g8[:, None]
    rx = None if dx is None else d @ w8
    rw = None if dw is None else d.T @ x8
    a = d.abs_()
    ed += 1.01 * h * a + (2.0**-38 * top.max() if typ == "f16" else 0.0)
    ed += max(len(w) * (rx is not None), len(x8) * (rw is not None)) * 2.0**-23 * a  # the sums
    for got, ref, tol in ((dx[keep] if rx is not None else None, rx, rx is not None and ed @ w8.abs()),
                          (dw, rw, rw is not None and ed.T @ x8.abs())):
        if ref is not None:
            over = (got.double() - ref).abs() - tol - 1.01 * h * ref.abs() - tiny
            assert (over <= 0).all(), over.max().item()
    assert dx is None or not dx[~keep].any()


@pytest.mark.parametrize("M,K", [(21760, 7936), (26880, 6400)])
def test_dx_where_two_ways_cost_the_same(psr, M, K):
    """Numbers of tiles for which whole and wide tiles of dx are worth exactly the same: its kernels decide alike, and write every row."""
    need_gpu()
    gen = torch.Generator(device="cuda").manual_seed(K)
    V = 7488
    x = torch.randn((M, K), generator=gen, device="cuda").to(torch.bfloat16)
    w = (torch.randn((V, K), generator=gen, device="cuda") * 2.5 * K**-0.5).to(torch.bfloat16)
    t = torch.randint(0, V, (M,), generator=gen, device="cuda")
    g = torch.rand(M, generator=gen, device="cuda")
    _, lse, _ = psr.linear_xent(x, w, t)
    dx = torch.full((M, K), float("nan"), dtype=x.dtype, device="cuda")
    _, _, ws = psr.linear_xent_bwd(g, x, w, t, lse, need_dw=False, dx=dx)
    assert psr.get_stats(ws)["status"] == 0 and not dx.isnan().any()
    rows = torch.arange(0, M, 61, device="cuda")  # of every tile
    check_on_device(dx[rows], None, g[rows], x[rows], w, t[rows], lse[rows], "bf16")


@pytest.mark.parametrize("M,V,K,drop,t,more", [
    (20000, 14000, 1000, 0.5, "bf16", {}),                            # two pieces, dx's last tiles in 14 and 13 parts
    (20000, 14000, 1003, 0.5, "f16", dict(smoothing=0.1)),            # the same, W and dx off 16-byte boundaries
    (9048, 29193, 1000, 0.0, "bf16", dict(z_weight=1e-3)),            # two pieces, dx in tiles of 512 columns
    (12183, 36851, 1001, 0.0, "f16", {}),                             # the same with halves of tiles in the last round
    (40000, 9001, 264, 0.1, "bf16", {}),                              # two pieces, whole tiles of several blocks of columns
    (700, 20011, 2104, 0.3, "bf16", {}), (1100, 12000, 4104, 0.0, "f16", {})],  # one piece, logits in three and five parts
    ids=str)
def test_gradients_of_many_rows_and_columns(psr, M, V, K, drop, t, more):
    """dx summed over pieces of the vocabulary in every form that its tiles take, and logits of several parts over several rounds of tiles."""
    need_gpu()
    gen = torch.Generator().manual_seed(M + K)
    x, w, targets, g = inputs(gen, M, V, K, t, drop)
    loss, lse, ws = psr.linear_xent(x, w, targets, **more)
    assert psr.get_stats(ws)["status"] == 0
    s, z, keep = more.get("smoothing", 0.0), more.get("z_weight", 0.0), targets != -100
    logits = x[keep].double() @ w.double().T
    ref = logits.logsumexp(1)
    # a logit is off by 2^-12 at most: 64 sums of 16 products to a part, each cut by less than 2^-23 of sums below 30, and some parts
    assert ((lse[keep].double() - ref).abs() <= 2.0**-12 + 2.0**-13 + 2.0**-22 * ref).all() and not lse[~keep].any()
    ref = ref + z * ref**2 - (1 - s) * logits.gather(1, targets[keep][:, None])[:, 0] - s * logits.mean(1)
    assert ((loss[keep].double() - ref).abs() <= 2.0**-11 + 2.0**-12 + 2.0**-22 * ref.abs()).all() and not loss[~keep].any()
    del logits
    dx, dw = (torch.full(m.shape, float("nan"), dtype=m.dtype, device="cuda") for m in (x, w))
    _, _, ws = psr.linear_xent_bwd(g, x, w, targets, lse, dx=dx, dw=dw, **more)
    assert psr.get_stats(ws)["status"] == 0
    check_on_device(dx, dw, g, x, w, targets, lse, t, s, z)
    again = psr.linear_xent_bwd(g, x, w, targets, lse, **more)
    assert torch.equal(again[0], dx) and torch.equal(again[1], dw)
