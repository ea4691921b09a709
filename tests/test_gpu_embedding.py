"""GPU tests of psr_embedding and psr_embedding_bwd against the fp64 oracle, through the binding.

Tolerance.  Lookup: scale * w is rounded to fp32 (2^-24) and once to the type.  Gradient: an fp32 sum of n rows is off by at
most n 2^-24 of the sum of their sizes (n additions, the join's among them), the scale and the addition to dw add a rounding
each, and the result is rounded once to its type (half a step; 2^-25 absolute below the normal fp16 numbers).
"""
import numpy as np
import pytest
import torch

from layer_util import check, f64, need_gpu, randn
from oracle import ends, layer as ol

pytestmark = pytest.mark.gpu

TINY = {"bf16": 0.0, "f16": 2.0**-25, "f32": 0.0}


def check_lookup(got, ids, w, scale, t, what):
    ref = ends.embedding(ids.tolist(), f64(w), scale)
    check(got, ref, (ol.HALF_STEP[t] * 1.01 + 2.0**-24) * np.abs(ref) + TINY[t], what)


def check_gradient(got, dy, ids, V, t, what, scale=1.0, padding=None, before=None):
    ref, n, size = ends.embedding_bwd(f64(dy), ids.tolist(), V, scale, padding, before)
    tol = (n[:, None] + 3) * 2.0**-24 * size + ol.HALF_STEP[t] * 1.01 * np.abs(ref) + TINY[t]
    check(got, ref, tol, what)
    named = n > 0
    assert not f64(got)[~named].any() if before is None else np.array_equal(f64(got)[~named], before[~named]), what


def tokens(gen, M, V, spread):
    """all: over the whole table; few: three ids; one: a single id; runs: sorted."""
    if spread == "one":
        return torch.full((M,), V - 1).cuda()
    ids = torch.randint(0, min(V, 3) if spread == "few" else V, (M,), generator=gen)
    return (ids.sort().values if spread == "runs" else ids).cuda()


LOOKUP = [  # M V K scale type
    (1, 1, 1, 1.0, "bf16"), (1, 7, 8, 2.0, "f16"), (3, 5, 17, 0.37, "bf16"), (32, 1000, 8192, 1.0, "bf16"),
    (33, 260, 514, 45.25, "f16"), (129, 50, 1000, 64.0, "f32"), (700, 333, 1001, 1.0, "f32"), (257, 77, 130, -3.0, "bf16")]


@pytest.mark.parametrize("case", LOOKUP, ids=str)
def test_lookup(psr, case):
    need_gpu()
    M, V, K, scale, t = case
    g = torch.Generator().manual_seed(M + K)
    w, ids = randn(g, (V, K), t), tokens(g, M, V, "all")
    check_lookup(psr.embedding(ids, w, scale=scale), ids, w, scale, t, str(case))


def test_lookup_views_and_bad_ids(psr):
    need_gpu()
    g = torch.Generator().manual_seed(1)
    w = randn(g, (40, 200), "bf16")[:, 8:108]
    ids = torch.tensor([3, -1, 39, 40, 0, -2**62, 2**40, 5]).cuda()
    wide = torch.stack([ids, ids + 1], 1)[:, 0]  # every second of a buffer
    buf = torch.full((8, 300), 7.0, dtype=torch.bfloat16).cuda()
    out = buf[:, 100:200]
    assert psr.embedding(wide, w, out=out) is out
    check_lookup(out, ids, w, 1.0, "bf16", "views")
    assert (buf[:, :100] == 7).all() and (buf[:, 200:] == 7).all()
    odd = randn(g, (41 * 100 + 1,), "bf16")[1:4101].view(41, 100)  # starts off every boundary
    check_lookup(psr.embedding(ids, odd, scale=2.0), ids, odd, 2.0, "bf16", "odd start")
    same = torch.tensor([4]).cuda().expand(6)
    check_lookup(psr.embedding(same, w), same, w, 1.0, "bf16", "one id for all")
    assert psr.embedding(ids[:0], w).shape == (0, 100)


def test_lookup_keeps_infinities(psr):
    need_gpu()
    w = torch.tensor([[float("inf"), float("nan"), -float("inf"), 1.0]] * 2, dtype=torch.float16).cuda()
    got = psr.embedding(torch.tensor([1]).cuda(), w, scale=2.0)
    check(got, np.array([[np.inf, np.nan, -np.inf, 2.0]]), 0.0, "infinities")


def test_lookup_far_rows(psr):
    """Rows past 2^31 elements of the table, and of the output."""
    need_gpu()
    w = torch.zeros((70000, 32768), dtype=torch.bfloat16, device="cuda")
    w[-1], w[65536] = 3.0, 2.0
    got = psr.embedding(torch.tensor([69999, 65536, 1]).cuda(), w)
    assert (got[0] == 3).all() and (got[1] == 2).all() and not got[2].any()
    dw, _ = psr.embedding_bwd(got, torch.tensor([69999, 65536, 69999]).cuda(), 70000, dw=w)
    assert (dw[69999] == 3).all() and (dw[65536] == 2).all() and not dw[:65536].any()


GRADIENT = [  # M V K spread scale type
    (1, 1, 1, "all", 1.0, "bf16"), (1, 9, 3, "one", 0.5, "f32"), (2, 2, 512, "few", 1.0, "f16"),
    (7, 100, 1000, "all", 1.0, "bf16"), (8, 100, 1000, "one", 3.0, "bf16"), (9, 4, 1001, "few", 1.0, "f16"),
    (31, 1 << 9, 8, "all", 1.0, "f32"), (32, (1 << 9) - 1, 16, "all", 1.0, "bf16"), (33, (1 << 18) + 3, 2, "all", 1.0, "bf16"),
    (255, 17, 130, "all", 45.25, "bf16"), (256, 300, 514, "runs", 1.0, "f16"), (257, 3, 96, "few", 1.0, "f32"),
    (1000, 260, 1001, "all", 1.0, "f32"), (1025, 1, 264, "one", 1.0, "bf16"), (2047, 5000, 72, "all", 32.0, "f16"),
    (8193, 100, 40, "runs", 1.0, "bf16"), (8200, 70000, 24, "all", 1.0, "f16"), (20000, 2, 8, "few", 1.0, "f32"),
    (40000, 999, 520, "all", 1.0, "bf16")]


@pytest.mark.parametrize("case", GRADIENT, ids=str)
def test_gradient(psr, case):
    need_gpu()
    M, V, K, spread, scale, t = case
    g = torch.Generator().manual_seed(M + V + K)
    dy, ids = randn(g, (M, K), t), tokens(g, M, V, spread)
    dw, ws = psr.embedding_bwd(dy, ids, V, scale=scale)
    assert psr.get_stats(ws)["status"] == 0
    check_gradient(dw, dy, ids, V, t, str(case), scale)
    again, _ = psr.embedding_bwd(dy, ids, V, scale=scale, workspace=ws)
    assert torch.equal(again.view(torch.uint8), dw.view(torch.uint8))


@pytest.mark.parametrize("K,step", [(4, 8), (2600, 16), (9000, 64)])
def test_gradient_of_runs_of_every_length(psr, K, step):
    """Runs of equal ids that end in, at and behind the borders of the blocks in which they are summed (of `step` positions)."""
    need_gpu()
    g = torch.Generator().manual_seed(K)
    lengths = torch.tensor([1, 2, step - 1, step, step + 1, 2 * step - 1, 2 * step, 2 * step + 1, 3 * step, 5 * step + 3, 3, 1, step // 2])
    lengths = lengths.repeat(4)[torch.randperm(52, generator=g)]
    ids = torch.repeat_interleave(torch.arange(52) * 3, lengths)
    ids = ids[torch.randperm(len(ids), generator=g)].cuda()
    dy = randn(g, (len(ids), K), "bf16")
    dw, _ = psr.embedding_bwd(dy, ids, 160)
    check_gradient(dw, dy, ids, 160, "bf16", str(K))


@pytest.mark.parametrize("M,V", [(2048, 100), (2049, 100), (300, (1 << 21) - 2), (300, (1 << 21) - 1), (2048, (1 << 21) - 2)])
def test_gradient_where_ranks_end(psr, M, V):
    """Numbers of tokens and rows around those up to which tokens are ranked by comparison; nothing is written around dw."""
    need_gpu()
    g = torch.Generator().manual_seed(M + V)
    ids = torch.randint(0, V, (M,), generator=g)
    ids[: M // 3] = ids[torch.randint(0, M, (M // 3,), generator=g)]
    ids[0], ids[1], ids[2] = V - 1, V, -1
    dy = randn(g, (M, 8), "f32")
    buffer = torch.full((V * 8 + 16,), 7.0, device="cuda")
    dw = buffer[8:-8].view(V, 8)
    psr.embedding_bwd(dy, ids.cuda(), V, dw=dw)
    keep = (ids >= 0) & (ids < V)
    named, at = torch.unique(ids[keep], return_inverse=True)
    check_gradient(dw[named.cuda()], dy[keep.cuda()], at, len(named), "f32", "named rows")
    dw[named.cuda()] = 0
    assert not dw.any() and (buffer[:8] == 7).all() and (buffer[-8:] == 7).all()


@pytest.mark.parametrize("K", [255, 257, 1001])
def test_gradient_of_long_runs_of_odd_rows(psr, K):
    need_gpu()
    g = torch.Generator().manual_seed(K)
    dy, ids = randn(g, (9000, K), "f32"), tokens(g, 9000, 20, "all")
    dw, _ = psr.embedding_bwd(dy, ids, 20)
    check_gradient(dw, dy, ids, 20, "f32", str(K))


@pytest.mark.parametrize("t", ["bf16", "f16", "f32"])
def test_gradient_leaves_out_and_adds(psr, t):
    need_gpu()
    g = torch.Generator().manual_seed(3)
    M, V, K = 600, 50, 136
    dy, ids = randn(g, (M, 2 * K), t)[:, K:], torch.randint(-3, V + 3, (M,), generator=g).cuda()
    ids[5] = 2**40 + 1
    dy[(ids < 0) | (ids == 7)] = float("nan")  # nothing of theirs is used
    base = randn(g, (V, K), t)
    dw = base.clone()
    got, _ = psr.embedding_bwd(dy, ids, V, padding=7, dw=dw, accumulate=True, scale=0.25)
    assert got is dw
    check_gradient(dw, dy, ids, V, t, "accumulate", 0.25, 7, f64(base))
    dw.fill_(9.0)
    psr.embedding_bwd(dy, ids, V, padding=7, dw=dw)
    check_gradient(dw, dy, ids, V, t, "padding", 1.0, 7)


def test_gradient_of_a_table_of_many_bits(psr):
    """Ids of 29 bits are sorted in four passes."""
    need_gpu()
    g = torch.Generator().manual_seed(8)
    V, M = (1 << 28) + 5, 5000
    ids = torch.randint(0, V, (M // 5,), generator=g).repeat(5)[torch.randperm(M, generator=g)]
    ids[0], ids[1] = V - 1, 0
    dy = randn(g, (M, 1), "f32")
    dw, _ = psr.embedding_bwd(dy, ids.cuda(), V)
    named, at = torch.unique(ids, return_inverse=True)
    ref, _, size = ends.embedding_bwd(f64(dy), at.tolist(), len(named))
    check(dw[named.cuda()], ref, 8 * 2.0**-24 * size, "named rows")
    dw[named.cuda()] = 0
    assert not dw.any()


def test_gradient_of_no_tokens(psr):
    need_gpu()
    dw = torch.full((5, 24), 3.0, dtype=torch.bfloat16, device="cuda")
    dy, ids = torch.empty((0, 24), dtype=torch.bfloat16, device="cuda"), torch.empty(0, dtype=torch.int64, device="cuda")
    psr.embedding_bwd(dy, ids, 5, dw=dw, accumulate=True)
    assert (dw == 3).all()
    _, ws = psr.embedding_bwd(dy, ids, 5, dw=dw)
    assert not dw.any() and psr.get_stats(ws)["status"] == 0


def test_gradient_is_the_forward_transposed(psr):
    """<dy, embedding(w)> = <dw, w>: by differences along any direction of w, the map being linear."""
    need_gpu()
    g = torch.Generator().manual_seed(4)
    w, dy, ids = randn(g, (90, 64), "f32"), randn(g, (500, 64), "f32"), tokens(g, 500, 90, "all")
    y = psr.embedding(ids, w, scale=3.0)
    dw, _ = psr.embedding_bwd(dy, ids, 90, scale=3.0)
    a, b = (f64(y) * f64(dy)).sum(), (f64(dw) * f64(w)).sum()
    assert abs(a - b) <= 32 * 2.0**-24 * (np.abs(f64(y)) * np.abs(f64(dy))).sum()


def test_streams_and_graphs(psr):
    need_gpu()
    g = torch.Generator().manual_seed(5)
    w, dy, ids = randn(g, (300, 256), "bf16"), randn(g, (900, 256), "bf16"), tokens(g, 900, 300, "all")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y = psr.embedding(ids, w, stream=side)
    dw, _ = psr.embedding_bwd(dy, ids, 300, stream=side)
    side.synchronize()
    check_lookup(y, ids, w, 1.0, "bf16", "side stream")
    check_gradient(dw, dy, ids, 300, "bf16", "side stream")
    out, dw2 = torch.empty_like(y), torch.empty_like(dw)
    ws = torch.empty(psr.embedding_workspace_bytes(900, 300, 256), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        psr.embedding(ids, w, out=out)
        psr.embedding_bwd(dy, ids, 300, dw=dw2, workspace=ws)
    for seed in (6, 7):
        g.manual_seed(seed)
        ids.copy_(tokens(g, 900, 300, "few" if seed == 6 else "all"))
        graph.replay()
        torch.cuda.synchronize()
        check_lookup(out, ids, w, 1.0, "bf16", "replay")
        check_gradient(dw2, dy, ids, 300, "bf16", "replay")


def test_refusals(psr):
    need_gpu()
    z = lambda *s, t=torch.bfloat16: torch.zeros(s, dtype=t, device="cuda")
    ids, w = z(4, t=torch.int64), z(9, 16)
    for call in (lambda: psr.embedding(ids.int(), w), lambda: psr.embedding(ids.cpu(), w), lambda: psr.embedding(ids, w.cpu()),
                 lambda: psr.embedding(ids.view(2, 2), w), lambda: psr.embedding(ids, w.double()),
                 lambda: psr.embedding(ids, w.t()), lambda: psr.embedding(ids, w, out=z(4, 17)),
                 lambda: psr.embedding(ids, w, out=z(4, 16, t=torch.float16)), lambda: psr.embedding(ids, w, out=w[:4]),
                 lambda: psr.embedding_bwd(z(5, 16), ids, 9), lambda: psr.embedding_bwd(z(4, 16), ids, 9, accumulate=True),
                 lambda: psr.embedding_bwd(z(4, 16), ids, 9, dw=z(8, 16)),
                 lambda: psr.embedding_bwd(z(4, 16), ids, 9, padding=9),
                 lambda: psr.embedding_bwd(z(1, 16).expand(4, 16), ids, 9),
                 lambda: psr.embedding_bwd(w[:4], ids, 9, dw=w),
                 lambda: psr.embedding_bwd(z(4, 16), ids, 9, workspace=z(100, t=torch.uint8))):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: psr.embedding(ids, z(0, 16)), lambda: psr.embedding(ids, w, scale=float("nan")),
                 lambda: psr.embedding_bwd(z(4, 16), ids, 0), lambda: psr.embedding_bwd(z(4, 16), ids, 9, scale=float("inf"))):
        with pytest.raises(psr.PsrError):
            call()


def block_of(psr, M, V, K):
    """Positions of a block, by what the workspace holds: 512 bytes, two lists of M pairs, a pair and two fp32 rows for each block."""
    up = lambda n: -(-n // 256) * 256
    total = psr.embedding_workspace_bytes(M, V, K)
    fits = [b for b in (8, 16, 32, 64) if total == 512 + 2 * up(8 * M) + up(8 * -(-M // b)) + up(8 * -(-M // b) * K)]
    assert len(fits) == 1, fits
    return fits[0]


@pytest.mark.parametrize("t,K,step", [("f16", 40, 8), ("f16", 520, 16), ("bf16", 520, 32), ("bf16", 520, 64), ("f32", 516, 64),
                                      ("f16", 514, 64), ("f32", 515, 64)])
def test_gradient_of_runs_around_whole_blocks(psr, t, K, step):
    """Runs of equal ids that end in, at and behind the borders of blocks of each length there is, the last block ragged."""
    need_gpu()
    g = torch.Generator().manual_seed(K + step)
    lengths = [1, 2, step // 2 - 1, step // 2, step // 2 + 1, step - 1, step, step + 1, 2 * step - 1, 2 * step, 2 * step + 1, 3 * step,
               5 * step + 3, 1, 3, 33]
    least = {8: 1000, 16: 38912 // 2, 32: 77824 // 2, 64: 155648 // 2}[step]
    n, total = [], 0
    while total < least or total % step <= step // 2:
        n.append(lengths[int(torch.randint(0, len(lengths), (), generator=g))])
        total += n[-1]
    V = 2 * len(n) + 3
    assert block_of(psr, total, V, K) == step
    ids = torch.repeat_interleave(torch.arange(len(n)) * 2 + 1, torch.tensor(n))
    for kind in ("sorted", "shuffled"):
        if kind == "shuffled":
            ids = ids[torch.randperm(total, generator=g)]
        dy = randn(g, (total, K), t)
        dw, ws = psr.embedding_bwd(dy, ids.cuda(), V)
        assert psr.get_stats(ws)["status"] == 0
        check_gradient(dw, dy, ids, V, t, kind)
    ids[torch.rand(total, generator=g) < 0.3] = V  # positions behind those of the table, from inside a block on
    dw, _ = psr.embedding_bwd(dy, ids.cuda(), V)
    check_gradient(dw, dy, ids, V, t, "named in part")
