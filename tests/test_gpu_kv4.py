"""GPU parity of the 4-bit KV cache (psr_kv4_append, psr_kv4_read, psr_kv4_attn) against the fp64 oracle.

Append and read are held to equality: the format defines every rounding.  Attention: the oracle's kv4_attention gives,
element by element, what the kernel's arithmetic may be off by (fp16 weights, fp32 sums); the output's rounding
adds half a step.
"""
import math

import numpy as np
import pytest
import torch

from layer_util import TYPES, check, f64, need_gpu, randn
from oracle import layer as ol

pytestmark = pytest.mark.gpu


def pages_for(rng, lens, page, extra=2, wide=0):
    """A shuffled table (unused entries -1) and the number of pages."""
    need = [(max(0, n) + page - 1) // page for n in lens]
    order = rng.permutation(sum(need) + extra)
    table = np.full((len(lens), max(1, wide, *need)), -1, np.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return table, sum(need) + extra


def random_cache(rng, n_pages, Hkv, d, page):
    """Cache bytes with random codes, scales and offsets."""
    blk = rng.integers(0, 256, (n_pages, Hkv, page // 16, 16 * (d + 8)), dtype=np.uint8)
    s = rng.uniform(0.05, 0.4, (n_pages, Hkv, page // 16, 32, 1))
    o = -7.5 * s + rng.normal(0, 0.4, s.shape)
    pair = (ol.to_bf16(np.concatenate([s, o], -1)).view(np.uint32) >> 16).astype(np.uint16)
    blk[..., 16 * d:] = np.ascontiguousarray(pair).view(np.uint8).reshape(*blk.shape[:3], 128)
    return blk.reshape(n_pages, Hkv, page * (d + 8))


@pytest.mark.parametrize("case", [  # B S Hkv d page type
    (1, 1, 1, 64, 16, "bf16"), (2, 5, 3, 64, 16, "f16"), (3, 40, 2, 128, 32, "bf16"), (1, 130, 1, 128, 64, "f16"),
    (2, 17, 2, 128, 256, "bf16"), (1, 2500, 1, 64, 64, "f16")], ids=str)
def test_append_and_read(psr, case):
    need_gpu()
    B, S, Hkv, d, page, t = case
    rng = np.random.default_rng(sum(case[:5]))
    g = torch.Generator().manual_seed(3)
    start = rng.integers(0, 40, B).astype(np.int32)
    count = rng.integers(0, S + 1, B).astype(np.int32)
    count[-1] = S
    table, n_pages = pages_for(rng, start + S, page)
    k, v = randn(g, (B, Hkv, S, d), t), randn(g, (B, Hkv, S, d), t, 0.01)
    k[0, 0, 0] = 0.0                 # constant rows
    v[0, 0, 0] = -3.0
    if S > 4:
        k[0, 0, 1, 3] = float("inf")
        v[0, 0, 2, 0] = float("nan")
        k[0, 0, 3] *= 30000.0        # near the largest fp16 numbers
        v[0, 0, 4] *= 1e-6
    cache = psr.kv4_cache(n_pages, Hkv, d, page)
    cache.copy_(torch.from_numpy(random_cache(rng, n_pages, Hkv, d, page)))
    want = cache.cpu().numpy()
    for b in range(B):
        for h in range(Hkv):
            for i in range(count[b]):
                for kv, x in ((0, k), (1, v)):
                    ol.kv4_write_row(want, table, page, b, h, int(start[b]) + i, kv, x[b, h, i].float().cpu().numpy())
    dev = [torch.from_numpy(a).cuda() for a in (table, start, count)]
    assert psr.kv4_append(k, v, cache, dev[0], dev[1], page=page, count=dev[2]) is cache
    got = cache.cpu().numpy()
    # a row that reads as NaN may hold any NaN pattern
    nan = ~np.isfinite((want.reshape(n_pages, Hkv, page // 16, -1)[..., 16 * d:].copy().view(np.uint16).astype(np.uint32)
                        << 16).astype(np.uint32).view(np.float32))
    a, b_ = (c.reshape(n_pages, Hkv, page // 16, -1) for c in (got, want))
    assert np.array_equal(a[..., :16 * d], b_[..., :16 * d])
    pa, pb = (c[..., 16 * d:].copy().view(np.uint16) for c in (a, b_))
    assert np.array_equal(pa[~nan], pb[~nan])
    kr, vr = psr.kv4_read(cache, dev[0], dev[1], S=S, Hkv=Hkv, d=d, page=page, count=dev[2], dtype=TYPES[t])
    for kv, r in ((0, kr), (1, vr)):
        ref = np.zeros((B, Hkv, S, d), np.float32)
        for b in range(B):
            for h in range(Hkv):
                for i in range(count[b]):
                    c, s, o = ol.kv4_row(want, table, page, b, h, int(start[b]) + i, kv, d)
                    ref[b, h, i] = (o + s * c).astype(np.float32)
        ref = torch.from_numpy(ref).to(TYPES[t])
        assert torch.equal(torch.isnan(r.cpu()), torch.isnan(ref))
        assert torch.equal(torch.nan_to_num(r.cpu()), torch.nan_to_num(ref))


def test_append_of_views_and_rows_without_a_place(psr):
    need_gpu()
    rng = np.random.default_rng(0)
    g = torch.Generator().manual_seed(1)
    B, S, Hkv, d, page = 3, 20, 2, 64, 16
    qkv = randn(g, (B, S, 8, d), "bf16")  # a projection's rows
    k, v = qkv[:, :, 4:6].transpose(1, 2), qkv[:, :, 6:8].transpose(1, 2)
    # sequence 0 runs past its table, 1 has a page of another cache in the middle, 2 starts below 0
    table = torch.tensor([[0, 1], [2, 99], [3, 4]], dtype=torch.int32, device="cuda")
    start = torch.tensor([25, 4, -3], dtype=torch.int32, device="cuda")
    cache = psr.kv4_cache(6, Hkv, d, page)
    ref = cache.cpu().numpy()
    for b, rows in ((0, range(0, 7)), (1, range(0, 12)), (2, range(3, 20))):
        for i in rows:
            for h in range(Hkv):
                for kv, x in ((0, k), (1, v)):
                    ol.kv4_write_row(ref, table.cpu().numpy(), page, b, h, int(start[b]) + i, kv, x[b, h, i].float().cpu().numpy())
    psr.kv4_append(k, v, cache, table, start, page=page)
    assert np.array_equal(cache.cpu().numpy(), ref)
    kr, vr = psr.kv4_read(cache, table, start, S=S, Hkv=Hkv, d=d, page=page)
    for b, bad in ((0, slice(7, 20)), (1, slice(12, 20)), (2, slice(0, 3))):
        assert torch.isnan(kr[b, :, bad]).all() and torch.isnan(vr[b, :, bad]).all()
    assert int(torch.isnan(kr).sum()) == Hkv * d * (13 + 8 + 3)


def run_attention(psr, case, seed, q_views=False):
    B, S, Hq, Hkv, d, page, lens, t = case
    rng = np.random.default_rng(seed)
    g = torch.Generator().manual_seed(seed)
    table, n_pages = pages_for(rng, lens, page, wide=3)
    cache = random_cache(rng, n_pages, Hkv, d, page)
    q = randn(g, (B, Hq, S, d), t)
    if q_views:
        q = randn(g, (B, S, Hq + 1, d), t)[:, :, :Hq].transpose(1, 2)
    o, lse, ws = psr.kv4_attn(q, torch.from_numpy(cache).cuda(), torch.from_numpy(table).cuda(),
                              torch.tensor(lens, dtype=torch.int32, device="cuda"), Hkv=Hkv, page=page)
    assert psr.get_stats(ws)["status"] == 0
    ro, rl, to, tl = ol.kv4_attention(f64(q), cache, table, lens, page, Hkv, 1 / math.sqrt(d))
    check(lse, rl, tl, f"{case} lse")
    check(o, ro, to + ol.HALF_STEP[t] * np.abs(ro) * 1.01 + (2.0**-25 if t == "f16" else 0.0), f"{case} o")


ATTN = [  # B S Hq Hkv d page lens type
    (1, 1, 1, 1, 64, 16, [1], "bf16"),
    (1, 1, 1, 1, 128, 16, [0], "bf16"),
    (2, 1, 4, 1, 128, 64, [17, 64], "bf16"),
    (3, 1, 8, 2, 128, 32, [33, 0, 100], "f16"),
    (2, 1, 8, 1, 64, 128, [129, 255], "bf16"),
    (1, 1, 5, 5, 64, 16, [300], "bf16"),
    (1, 1, 9, 1, 128, 64, [130], "bf16"),
    (1, 1, 40, 2, 128, 16, [70], "f16"),
    (2, 2, 4, 2, 64, 16, [1, 40], "bf16"),
    (3, 4, 4, 4, 128, 16, [3, 4, 37], "bf16"),
    (2, 5, 6, 2, 64, 32, [70, 2], "f16"),
    (1, 17, 4, 1, 128, 64, [90], "bf16"),
    (1, 33, 2, 2, 64, 16, [33], "bf16"),
    (1, 1, 16, 2, 128, 256, [1500], "bf16"),
    (5, 1, 2, 1, 64, 16, [1, 2, 15, 16, 400], "bf16"),
]


@pytest.mark.parametrize("case", ATTN, ids=str)
def test_attention(psr, case):
    need_gpu()
    run_attention(psr, case, 5)


def test_attention_of_query_views(psr):
    need_gpu()
    run_attention(psr, (2, 3, 4, 2, 64, 16, [50, 21], "bf16"), 6, q_views=True)
    run_attention(psr, (2, 1, 8, 2, 128, 32, [50, 21], "f16"), 7, q_views=True)


def test_attention_of_bad_lengths_and_pages(psr):
    # a length below 0 or past the table, or a page that the cache does not have: NaN; the others are not touched by it.
    # Where a sequence is cut into pieces depends on the whole batch's lengths, and with it the order of the fp32 sums:
    # the good sequence is held to the oracle's bound, not to the bits that it has in another batch.
    need_gpu()
    rng = np.random.default_rng(1)
    g = torch.Generator().manual_seed(1)
    B, Hq, Hkv, d, page = 6, 4, 2, 64, 16
    lens = [40, 40, 40, 40, 40, 40]
    table, n_pages = pages_for(rng, lens, page)
    cache = torch.from_numpy(random_cache(rng, n_pages, Hkv, d, page)).cuda()
    q = randn(g, (B, Hq, 1, d), "bf16")

    def run(table, lens):
        o, lse, _ = psr.kv4_attn(q, cache, torch.from_numpy(table).cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"),
                                 Hkv=Hkv, page=page)
        return o, lse
    run(table, lens)
    table2, lens2 = table.copy(), list(lens)
    lens2[0], lens2[1] = -1, 49
    table2[2, 0], table2[3, 2], lens2[3] = n_pages, -7, 33
    lens2[4] = 0
    table2[4] = -1
    o, lse = run(table2, lens2)
    for b in range(4):
        assert torch.isnan(o[b]).all() and torch.isnan(lse[b]).all(), b
    assert not o[4].any() and torch.isneginf(lse[4]).all()
    ro, rl, to, tl = ol.kv4_attention(f64(q[5:]), cache.cpu().numpy(), table[5:], [40], page, Hkv, 1 / math.sqrt(d))
    check(lse[5:], rl, tl, "lse beside bad sequences")
    check(o[5:], ro, to + 2.0**-8 * np.abs(ro) * 1.01, "o beside bad sequences")
    table3 = table.copy()
    table3[:, 2] = 1 << 30  # behind 32 positions the table is not looked at
    o, lse = run(table3, [32] * B)
    assert torch.isfinite(o).all() and torch.isfinite(lse).all()


def test_attention_extreme_values(psr):
    need_gpu()
    Hkv, d, page, n = 1, 64, 16, 20
    cache = psr.kv4_cache(2, Hkv, d, page)
    table = torch.tensor([[1, 0]], dtype=torch.int32, device="cuda")
    zero = torch.zeros(1, dtype=torch.int32, device="cuda")
    g = torch.Generator().manual_seed(2)
    k, v = randn(g, (1, 1, n, d), "bf16"), randn(g, (1, 1, n, d), "bf16")
    k[0, 0, 7] *= 1e4   # one key takes every weight
    psr.kv4_append(k, v, cache, table, zero, page=page)
    kr, vr = psr.kv4_read(cache, table, zero, S=n, Hkv=1, d=d, page=page)
    q = (kr[:, :, 7:8] / 1e3).contiguous()
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    o, lse, _ = psr.kv4_attn(q, cache, table, lens, Hkv=1, page=page)
    assert torch.allclose(o[0, 0, 0].float(), vr[0, 0, 7].float(), rtol=2.0**-7, atol=2.0**-7)
    # rows behind the length may hold anything, NaN and infinities too
    cache2 = cache.clone()
    k[0, 0, 12:] = float("nan")
    v[0, 0, 12:] = float("inf")
    psr.kv4_append(k, v, cache2, table, zero, page=page)
    short = torch.tensor([12], dtype=torch.int32, device="cuda")
    a, b = psr.kv4_attn(q, cache, table, short, Hkv=1, page=page), psr.kv4_attn(q, cache2, table, short, Hkv=1, page=page)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]) and torch.isfinite(a[0]).all()
    # a NaN row inside the length shows
    o, lse, _ = psr.kv4_attn(q, cache2, table, lens, Hkv=1, page=page)
    assert torch.isnan(o).all() and torch.isnan(lse).all()


def test_attention_draft_queries_do_not_see_later_rows(psr):
    # with S = 3 the first query must not change when the last rows do, NaN among them
    need_gpu()
    rng = np.random.default_rng(4)
    g = torch.Generator().manual_seed(4)
    Hq, Hkv, d, page, n = 4, 2, 128, 32, 40
    table, n_pages = pages_for(rng, [n], page)
    cache = torch.from_numpy(random_cache(rng, n_pages, Hkv, d, page)).cuda()
    tab, lens = torch.from_numpy(table).cuda(), torch.tensor([n], dtype=torch.int32, device="cuda")
    q = randn(g, (1, Hq, 3, d), "bf16")
    a = psr.kv4_attn(q, cache, tab, lens, Hkv=Hkv, page=page)
    bad = torch.full((1, Hkv, 2, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    psr.kv4_append(bad, bad, cache, tab, lens - 2, page=page)
    b = psr.kv4_attn(q, cache, tab, lens, Hkv=Hkv, page=page)
    assert torch.equal(a[0][:, :, 0], b[0][:, :, 0]) and torch.equal(a[1][:, :, 0], b[1][:, :, 0])
    assert torch.isnan(b[0][:, :, 1:]).all()


def test_attention_long_cache_offsets(psr):
    # byte offsets past 2^31 and 2^32 in the cache: pages at its end hold the sequence
    need_gpu()
    Hkv, d, page = 8, 128, 256
    n_pages = (1 << 32) // (Hkv * page * (d + 8)) + 40
    cache = psr.kv4_cache(n_pages, Hkv, d, page)
    small = psr.kv4_cache(5, Hkv, d, page)
    g = torch.Generator().manual_seed(3)
    k, v = randn(g, (1, Hkv, 1200, d), "bf16"), randn(g, (1, Hkv, 1200, d), "bf16")
    q = randn(g, (1, 32, 1, d), "bf16")
    zero, lens = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.tensor([1200], dtype=torch.int32, device="cuda")
    got = []
    for c, first in ((cache, n_pages - 5), (small, 0)):
        table = torch.arange(first, first + 5, dtype=torch.int32, device="cuda")[None].contiguous()
        psr.kv4_append(k, v, c, table, zero, page=page)
        got.append((*psr.kv4_attn(q, c, table, lens, Hkv=Hkv, page=page)[:2],
                    *psr.kv4_read(c, table, zero, S=1200, Hkv=Hkv, d=d, page=page)))
    assert all(torch.equal(a, b) for a, b in zip(*got))


def test_attention_graph_streams_and_repeats(psr):
    need_gpu()
    rng = np.random.default_rng(9)
    g = torch.Generator().manual_seed(9)
    lens = [700, 1, 90, 0]
    Hq, Hkv, d, page = 8, 2, 128, 64
    table, n_pages = pages_for(rng, lens, page)
    cache = torch.from_numpy(random_cache(rng, n_pages, Hkv, d, page)).cuda()
    tab, ln = torch.from_numpy(table).cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda")
    q = randn(g, (4, Hq, 1, d), "bf16")
    want = psr.kv4_attn(q, cache, tab, ln, Hkv=Hkv, page=page)[:2]
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(psr.kv4_attn(q, cache, tab, ln, Hkv=Hkv, page=page)[:2], want))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = psr.kv4_attn(q, cache, tab, ln, Hkv=Hkv, page=page, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got[:2], want))
    out, lse = torch.zeros_like(want[0]), torch.zeros_like(want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        psr.kv4_attn(q, cache, tab, ln, Hkv=Hkv, page=page, out=out, lse=lse)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    ln -= 1  # the lengths are read when the graph runs
    ln.clamp_(min=0)
    graph.replay()
    torch.cuda.synchronize()
    again = psr.kv4_attn(q, cache, tab, ln, Hkv=Hkv, page=page)[:2]
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])


def test_empty_batches(psr):
    need_gpu()
    cache = psr.kv4_cache(2, 2, 64, 16)
    for B, S in ((0, 1), (2, 0)):
        e = torch.empty((B, 2, S, 64), dtype=torch.bfloat16, device="cuda")
        table = torch.zeros((B, 1), dtype=torch.int32, device="cuda")
        z = torch.zeros(B, dtype=torch.int32, device="cuda")
        psr.kv4_append(e, e, cache, table, z, page=16)
        k, v = psr.kv4_read(cache, table, z, S=S, Hkv=2, d=64, page=16)
        o, lse, _ = psr.kv4_attn(e, cache, table, z, Hkv=2, page=16)
        assert k.shape == o.shape == (B, 2, S, 64) and lse.shape == (B, 2, S)
    assert not cache.any()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("group,S", [(1, 1), (2, 1), (3, 1), (4, 1), (1, 2), (2, 2), (1, 3), (1, 4), (5, 1), (3, 2), (7, 1),
                                     (8, 1), (9, 1), (4, 4), (17, 1)])
def test_attention_rows_of_a_kv_head(psr, group, S, d):
    # last units of every fill, with one to seventeen query rows to a KV head
    need_gpu()
    lens = [0, 1, 2, 15, 16, 17, 31, 32, 33, 47, 48, 49, 64, 65, 300]
    run_attention(psr, (len(lens), S, 2 * group, 2, d, 16, lens, "f16" if group % 2 else "bf16"), 40 + group)


@pytest.mark.parametrize("Hq", [4, 8])
def test_attention_with_large_scores_in_one_block(psr, Hq):
    # one block of 16 tokens outweighs all others, wherever it stands, by more than fp32 or fp16 ratios hold
    need_gpu()
    n, d, page = 160, 64, 32
    rng = np.random.default_rng(8)
    for at in range(0, n, 16):
        cache = random_cache(rng, 5, 1, d, page)
        blocks = cache.reshape(5, 1, page // 16, 16 * (d + 8))
        pairs = blocks[at // page, 0, at % page // 16, 16 * d:].view(np.uint16).reshape(2, 16, 2)
        pairs[0, :, 1] = np.float32(60).view(np.uint32) >> 16  # offsets of K
        q = torch.full((1, Hq, 1, d), 0.5, dtype=torch.bfloat16, device="cuda")
        table = torch.arange(5, dtype=torch.int32, device="cuda")[None]
        lens = torch.tensor([n], dtype=torch.int32, device="cuda")
        o, lse, _ = psr.kv4_attn(q, torch.from_numpy(cache).cuda(), table, lens, Hkv=1, page=page, scale=1.0)
        ro, rl, to, tl = ol.kv4_attention(f64(q), cache, table.cpu().numpy(), [n], page, 1, 1.0)
        check(lse, rl, tl, f"block at {at}: lse")
        check(o, ro, to + ol.HALF_STEP["bf16"] * np.abs(ro) * 1.01, f"block at {at}: o")


def test_attention_of_shared_pages(psr):
    # sequences with the same first pages, and one with the same page over and over
    need_gpu()
    rng = np.random.default_rng(9)
    Hkv, d, page = 2, 128, 16
    cache = random_cache(rng, 6, Hkv, d, page)
    table = np.array([[0, 1, 2, 3], [0, 1, 4, 5], [2, 2, 2, 2]], np.int32)
    lens = [60, 49, 64]
    g = torch.Generator().manual_seed(9)
    q = randn(g, (3, 8, 2, d), "bf16")
    o, lse, _ = psr.kv4_attn(q, torch.from_numpy(cache).cuda(), torch.from_numpy(table).cuda(),
                             torch.tensor(lens, dtype=torch.int32, device="cuda"), Hkv=Hkv, page=page)
    ro, rl, to, tl = ol.kv4_attention(f64(q), cache, table, lens, page, Hkv, 1 / math.sqrt(d))
    check(lse, rl, tl, "shared pages: lse")
    check(o, ro, to + ol.HALF_STEP["bf16"] * np.abs(ro) * 1.01, "shared pages: o")


def test_attention_of_two_streams_at_once(psr):
    need_gpu()
    rng = np.random.default_rng(10)
    g = torch.Generator().manual_seed(10)
    Hkv, d, page = 4, 128, 64
    calls = []
    for lens in ([3000, 10, 900, 1], [40, 2500], [5000]):
        table, n_pages = pages_for(rng, lens, page)
        cache = torch.from_numpy(random_cache(rng, n_pages, Hkv, d, page)).cuda()
        calls.append((randn(g, (len(lens), 16, 1, d), "bf16"), cache, torch.from_numpy(table).cuda(),
                      torch.tensor(lens, dtype=torch.int32, device="cuda")))
    want = [psr.kv4_attn(*c, Hkv=Hkv, page=page)[:2] for c in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    for _ in range(5):
        got = [psr.kv4_attn(*c, Hkv=Hkv, page=page, stream=s)[:2] for c, s in zip(calls, streams)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for x, y in zip(got, want) for a, b in zip(x, y))


def rows_with_steps_at_a_tie(t, d):
    """Rows whose step is in the middle of two bf16 numbers or next to it, with that step from exact integers: multiples of 2^-20."""
    rng, wide = np.random.default_rng(3), 2048 if t == "f16" else 255  # integers up to it are exact
    rows, steps = [], []
    for m in range(128, 256):
        for high in (2048, 4096, 6144):
            span = 15 * (2 * m + 1)  # of a step m + 1/2, doubled
            for off in (0, 1, -1, 1024, -1024):  # of 2^-10
                low = high * 1024 - span * 1024 + off
                exact = torch.tensor(low / 1024.0).to(TYPES[t])
                if abs(low) > wide * 1024 or float(exact) != low / 1024.0:
                    continue
                row = rng.uniform(low / 1024.0, high, d)
                row[rng.choice(d, 2, replace=False)] = low / 1024.0, high
                rows.append(torch.from_numpy(row * 2.0**-10))
                up = off < 0 or (off == 0 and m % 2 == 1)  # a lower minimum is a longer span
                steps.append((m + up) * 2.0**-9)
    return torch.stack(rows).to(TYPES[t]), np.array(steps)


@pytest.mark.parametrize("t,d", [("f16", 64), ("f16", 128), ("bf16", 64), ("bf16", 128)])
def test_append_of_rows_whose_step_is_a_tie(psr, t, d):
    need_gpu()
    x, steps = rows_with_steps_at_a_tie(t, d)
    n, page = len(x), 64
    x = x.view(1, 1, n, d).cuda()
    cache = psr.kv4_cache((n + page - 1) // page, 1, d, page)
    table = torch.arange(cache.shape[0], dtype=torch.int32, device="cuda")[None]
    psr.kv4_append(x, x, cache, table, torch.zeros(1, dtype=torch.int32, device="cuda"), page=page)
    got, tab = cache.cpu().numpy(), table.cpu().numpy()
    want, s, o = ol.kv4_quantise(x[0, 0].float().cpu().numpy())
    for i in range(n):
        for kv in (0, 1):
            code, step, off = ol.kv4_row(got, tab, page, 0, 0, i, kv, d)
            assert step == steps[i] == s[i, 0], (i, kv, float(step), steps[i])
            assert off == o[i, 0] and np.array_equal(code, want[i]), (i, kv)


@pytest.mark.parametrize("d", [64, 128])
def test_append_of_rows_wider_than_fp32(psr, d):
    # the span of a row, and the distance of an element from its minimum, may pass the largest fp32 number
    need_gpu()
    rng = np.random.default_rng(d)
    n, page = 32, 16
    rows = rng.uniform(-1, 1, (n, d)) * np.linspace(0.25, 1, n)[:, None] * 1.99 * 2.0**127
    x = torch.from_numpy(rows).to(torch.bfloat16)
    assert torch.isfinite(x).all()
    cache = psr.kv4_cache(2, 1, d, page)
    table = torch.arange(2, dtype=torch.int32, device="cuda")[None]
    y = x.view(1, 1, n, d).cuda()
    psr.kv4_append(y, y, cache, table, torch.zeros(1, dtype=torch.int32, device="cuda"), page=page)
    got, tab, x = cache.cpu().numpy(), table.cpu().numpy(), f64(x)
    want, s, o = ol.kv4_quantise(x)
    for i in range(n):
        for kv in (0, 1):
            code, step, off = ol.kv4_row(got, tab, page, 0, 0, i, kv, d)
            assert step == s[i, 0] and off == o[i, 0] and np.array_equal(code, want[i]), (i, kv)
            # the nearest code, but for the rounding of the quotient (2 steps of 2^-24 below 16)
            assert (np.abs(np.clip((x[i] - off) / step, 0, 15) - code) <= 0.5 + 2.0**-19).all(), (i, kv)


def test_attention_status_of_empty_batches(psr):
    # a workspace that holds anything, through the binding and the C entry
    need_gpu()
    cache = psr.kv4_cache(2, 2, 64, 16)
    size = psr.kv4_attn_workspace_bytes(2, 2, 2, 1, 64, page=16, n_pages=2, max_pages=1)
    for B, S in ((0, 1), (2, 0)):
        e = torch.empty((B, 2, S, 64), dtype=torch.bfloat16, device="cuda")
        table, z = torch.zeros((B, 1), dtype=torch.int32, device="cuda"), torch.zeros(B, dtype=torch.int32, device="cuda")
        ws = torch.full((size,), 0xFF, dtype=torch.uint8, device="cuda")
        assert psr.kv4_attn(e, cache, table, z, Hkv=2, page=16, workspace=ws)[2] is ws
        assert psr.get_stats(ws)["status"] == 0
        ws.fill_(0xFF)
        some = torch.zeros(4096, dtype=torch.uint8, device="cuda")  # stands for the tensors: nothing of them is read
        at, st = some.data_ptr(), psr.Strides(128, 64, 64)
        sh = psr.Kv4Shape(B, 2, 2, S, 64, 16, 2, 1, psr.BF16, 0.0)
        assert psr.load().psr_kv4_attn(sh, at, st, cache.data_ptr(), at, at, at, st, at, ws.data_ptr(), size,
                                       torch.cuda.current_stream().cuda_stream) == 0
        assert psr.get_stats(ws)["status"] == 0 and not some.any()


@pytest.mark.parametrize("large", [2.0**30, 2.0**100, float("inf"), float("nan")])
@pytest.mark.parametrize("Hq", [3, 4, 8, 16])
@pytest.mark.parametrize("d", [64, 128])
def test_attention_heads_of_different_sizes(psr, d, Hq, large):
    # the rows of a KV head share matrix products: one with large or infinite elements leaves the others as they are
    need_gpu()
    rng = np.random.default_rng(Hq + d)
    g = torch.Generator().manual_seed(Hq)
    lens, page = [70, 33], 32
    table, n_pages = pages_for(rng, lens, page)
    cache = random_cache(rng, n_pages, 1, d, page)
    q = randn(g, (2, Hq, 1, d), "bf16")
    q[:, 0] *= large
    q[:, 1] *= 300
    q[:, 2] *= 2.0**-20
    o, lse, _ = psr.kv4_attn(q, torch.from_numpy(cache).cuda(), torch.from_numpy(table).cuda(),
                             torch.tensor(lens, dtype=torch.int32, device="cuda"), Hkv=1, page=page)
    ro, rl, to, tl = ol.kv4_attention(f64(q[:, 1:]), cache, table, lens, page, 1, 1 / math.sqrt(d))
    check(lse[:, 1:], rl, tl, "lse")
    check(o[:, 1:], ro, to + ol.HALF_STEP["bf16"] * np.abs(ro) * 1.01, "o")
    if math.isnan(large):
        assert torch.isnan(o[:, 0]).all() and torch.isnan(lse[:, 0]).all()
