"""CPU tests of the layer operators: the frequency table, the oracle's own pins, workspace and cache sizes, and what the C
ABI and the binding refuse before anything reaches a device."""
import numpy as np
import pytest
import torch

from oracle import layer as ol

PTR = 1 << 20  # stands for device memory: never read, every call here ends on the host


# ---- rotary table --------------------------------------------------------------------------------

@pytest.mark.parametrize("rot,base,kw", [
    (2, 10000.0, {}), (64, 10000.0, {}), (96, 500000.0, {}),
    (64, 10000.0, dict(scaling="linear", factor=8.0)),
    (128, 10000.0, dict(scaling="by_parts", factor=4.0, original_length=4096)),
    (48, 10000.0, dict(scaling="by_parts", factor=16.0, original_length=2048, beta_fast=16.0, beta_slow=2.0)),
    (64, 10000.0, dict(scaling="by_parts", factor=1.0, original_length=16))], ids=str)
def test_rotary_table_holds_the_frequencies(psr, rot, base, kw):
    got = psr.rotary_table(rot, base, device="cpu", **kw)
    want = ol.frequencies(rot, base, kw.get("scaling", "plain"), kw.get("factor", 1.0), kw.get("original_length", 0),
                          kw.get("beta_fast", 32.0), kw.get("beta_slow", 1.0))
    turns = got.numpy().astype(np.float64) / 2.0**64
    assert got.dtype == torch.int64 and got.shape == (rot // 2,)
    # the fixed point cuts below 2^-64 of a turn
    np.testing.assert_allclose(turns * 2 * np.pi, want, rtol=1e-14, atol=2 * np.pi * 2.0**-64)


@pytest.mark.parametrize("args,kw", [
    ((0,), {}), ((3,), {}), ((-2,), {}), ((2048,), {}), ((64, 1.0), {}), ((64, float("inf")), {}), ((64, float("nan")), {}),
    ((64,), dict(scaling="linear", factor=0.5)), ((64,), dict(scaling="by_parts", factor=2.0)),
    ((64,), dict(scaling="by_parts", factor=2.0, original_length=4096, beta_fast=1.0, beta_slow=1.0))], ids=str)
def test_rotary_table_refuses(psr, args, kw):
    with pytest.raises(psr.PsrError) as e:
        psr.rotary_table(*args, device="cpu", **kw)
    assert e.value.status == psr.ERR_ARG


def test_rotary_table_unknown_scaling(psr):
    with pytest.raises(ValueError, match="scaling"):
        psr.rotary_table(64, scaling="other", device="cpu")


# ---- the oracle ----------------------------------------------------------------------------------

def test_oracle_rotary_keeps_lengths_and_composes():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((2, 3, 5, 16))
    f = ol.frequencies(12)
    for inter in (False, True):
        y = ol.rotary(x, [range(5)], f, interleaved=inter)
        np.testing.assert_allclose((y**2).sum(-1), (x**2).sum(-1), rtol=1e-12)
        np.testing.assert_allclose(ol.rotary(y, [range(5)], f, interleaved=inter, inverse=True), x, atol=1e-13)
        z = ol.rotary(ol.rotary(x, [[2] * 5], f, interleaved=inter), [[3] * 5], f, interleaved=inter)
        np.testing.assert_allclose(z, ol.rotary(x, [[5] * 5], f, interleaved=inter), atol=1e-13)
    assert np.array_equal(ol.rotary(x, [[0] * 5], f), x)


def test_oracle_scores_depend_on_distance_alone():
    rng = np.random.default_rng(1)
    q, k = rng.standard_normal((2, 1, 1, 1, 16))
    f = ol.frequencies(16)
    dot = lambda a, b: (ol.rotary(q, [[a]], f) * ol.rotary(k, [[b]], f)).sum()
    assert abs(dot(7, 3) - dot(1 << 40, (1 << 40) - 4)) < 1e-9


def test_oracle_shard_positions():
    assert ol.shard_positions(8, 2, True).tolist() == [0, 1, 6, 7, 2, 3, 4, 5]
    assert ol.shard_positions(6, 3, False).tolist() == list(range(6))


@pytest.mark.parametrize("name", ["none", "relu", "gelu", "gelu_tanh", "silu"])
def test_oracle_linear_gradients_are_differences(name):
    rng = np.random.default_rng(2)
    x, w, b, dy = rng.standard_normal((5, 4)), rng.standard_normal((3, 4)), rng.standard_normal(3), rng.standard_normal((5, 3))
    _, z = ol.linear(x, w, b, None, name)
    dx, dw, db, _ = ol.linear_bwd(dy, x, w, z, name)
    f = lambda x, w, b: (ol.linear(x, w, b, None, name)[0] * dy).sum()
    for i, grad in enumerate((dx, dw, db)):
        s = rng.standard_normal(grad.shape)
        args = lambda h: [v + (h * s if j == i else 0) for j, v in enumerate((x, w, b))]
        assert abs((f(*args(1e-6)) - f(*args(-1e-6))) / 2e-6 - (grad * s).sum()) < 1e-6


def test_oracle_quantiser_is_within_half_a_step():
    rng = np.random.default_rng(3)
    x = ol.to_bf16(rng.standard_normal((50, 64)) * np.exp(rng.uniform(-8, 8, (50, 1))))
    c, s, o = ol.kv4_quantise(x)
    back = o + s * c
    # half a step, the rounding of the scale (15 steps of 2^-8) and of the offset
    assert (np.abs(back - x) <= s * (0.5 + 15 * 2.0**-8) + 2.0**-8 * np.abs(o)).all()
    c, s, o = ol.kv4_quantise(np.array([[3.0] * 4, [0.0] * 4, [1, np.nan, 0, 0], [np.inf, 0, 0, 0], [-3e38, 3e38, 0, 0]]))
    assert not c[:4].any() and s[:2].tolist() == [[0], [0]] and np.isnan(s[2:4]).all() and np.isfinite(s[4]).all()
    assert c[4].tolist() == [0, 15, 8, 8] or c[4].tolist() == [0, 15, 7, 7]


def test_oracle_step_is_the_nearest_bf16_number():
    # 15 t for a t in the middle of two bf16 numbers: to the even one; a little above or below: to that side
    for m in range(128, 256):
        for k in (-130, -20, 0, 100):
            low, high = m * 2.0**k, (m + 1) * 2.0**k
            even = low if m % 2 == 0 else high
            top = 8192.0 * 2.0**k
            span = 15 * (low + high) / 2
            assert ol.kv4_step(top - span, top) == even, (m, k)
            assert ol.kv4_step(top - span * (1 + 2.0**-30), top) == high and ol.kv4_step(top - span * (1 - 2.0**-30), top) == low
    assert ol.kv4_step(0.0, 0.0) == 0.0 and ol.kv4_step(-2.5, -2.5) == 0.0
    assert ol.kv4_step(-1.75 * 2.0**127, 1.75 * 2.0**127) == 239 * 2.0**117  # 238.9 of them


def test_oracle_quantiser_of_rows_wider_than_fp32():
    x = np.array([[-1.0, 1.0, 0.75, 0.5, -0.75, 0.125]]) * 1.9375 * 2.0**127
    c, s, o = ol.kv4_quantise(x)
    assert c.tolist() == [[0, 15, 13, 11, 2, 8]] and np.isfinite(s).all() and np.isfinite(o).all()  # 7.5 (1 + x / max)


# ---- sizes ---------------------------------------------------------------------------------------

def test_workspace_and_cache_sizes(psr):
    assert psr.linear_workspace_bytes(100, 200, 300) >= 256
    full = psr.linear_workspace_bytes(1000, 2000, 300, activation="gelu", backward=True)
    assert full >= 1000 * 2000 * 2 + 256
    assert psr.linear_workspace_bytes(0, 8, 8) > 0
    for bad in ((-1, 8, 8), (8, 0, 8), (8, 8, 0)):
        with pytest.raises(psr.PsrError):
            psr.linear_workspace_bytes(*bad)
    assert psr.kv4_cache(3, 2, 64, 16, device="cpu").shape == (3, 2, 16 * 72)
    for bad in ((0, 2, 64, 16), (3, 0, 64, 16), (3, 2, 96, 16), (3, 2, 64, 8), (3, 2, 64, 24), (3, 2, 64, 512)):
        with pytest.raises(psr.PsrError):
            psr.kv4_cache(*bad, device="cpu")


# ---- refusals of the C ABI -------------------------------------------------------------------------

def _st():
    import persistent_sm_ring_gb300 as p
    return p.Strides(4096, 64, 64)


def rotary_call(psr, shape=None, **over):
    sh = psr.RotaryShape(2, 4, 2, 16, 1, 64, 1, 64, 0, 0, psr.BF16, 1.0, 0)
    for k, v in (shape or {}).items():
        setattr(sh, k, v)
    a = dict(sh=sh, q=PTR, qs=_st(), qo=PTR, qos=_st(), k=PTR, ks=_st(), ko=PTR, kos=_st(), table=PTR, pos=None, pb=0)
    a.update(over)
    return psr.load().psr_rotary(a["sh"], a["q"], a["qs"], a["qo"], a["qos"], a["k"], a["ks"], a["ko"], a["kos"], a["table"],
                                 a["pos"], a["pb"], None)


def test_rotary_refuses(psr):
    for name in ("sh", "q", "qs", "qo", "qos", "k", "ks", "ko", "kos", "table"):
        assert rotary_call(psr, **{name: None}) == psr.ERR_ARG, name
    for name in ("q", "qo", "k", "ko", "pos"):
        assert rotary_call(psr, **{name: PTR + 1}) == psr.ERR_ARG, name
    assert rotary_call(psr, table=PTR + 4) == psr.ERR_ARG
    for bad in (dict(B=-1), dict(S=-1), dict(Hq=0), dict(Hkv=-1), dict(P=0), dict(d=0), dict(d=1025), dict(rot=0), dict(rot=3),
                dict(rot=66), dict(type=3), dict(type=-1), dict(causal=3), dict(causal=-1)):
        assert rotary_call(psr, bad) == psr.ERR_ARG, bad
    assert rotary_call(psr, dict(P=3)) == psr.ERR_UNSUPPORTED
    assert rotary_call(psr, dict(P=16, causal=2)) == psr.ERR_UNSUPPORTED  # half-chunks of half a row


def linear_call(psr, shape=None, bwd=False, ws=1 << 30, **over):
    sh = psr.LinearShape(4, 16, 32, 0, psr.BF16, 0, 0, 0, 0, 0)
    for k, v in (shape or {}).items():
        setattr(sh, k, v)
    a = dict(sh=sh, x=PTR, w=PTR, b=PTR, r=PTR, y=PTR, z=PTR, wsp=PTR, dx=PTR, dw=PTR, db=PTR)
    a.update(over)
    lib = psr.load()
    if bwd:
        return lib.psr_linear_bwd(a["sh"], a["y"], a["z"], a["x"], a["w"], a["dx"], a["dw"], a["db"], a["wsp"], ws, 0, None)
    return lib.psr_linear(a["sh"], a["x"], a["w"], a["b"], a["r"], a["y"], a["z"], a["wsp"], ws, 0, None)


def test_linear_refuses(psr):
    for bwd in (False, True):
        for name in ("sh", "x", "w", "y", "wsp"):
            assert linear_call(psr, bwd=bwd, **{name: None}) == psr.ERR_ARG, name
        for name in ("x", "w", "y", "z") + (("dx", "dw", "db") if bwd else ("b", "r")):
            assert linear_call(psr, bwd=bwd, **{name: PTR + 1}) == psr.ERR_ARG, name
        assert linear_call(psr, bwd=bwd, wsp=PTR + 16) == psr.ERR_ARG
        for bad in (dict(M=-1), dict(N=0), dict(K=0), dict(act=5), dict(act=-1), dict(type=2), dict(ldx=31), dict(ldw=31),
                    dict(ldy=15), dict(ldz=15), dict(ldr=15), dict(ldx=-32)):
            assert linear_call(psr, bad, bwd=bwd) == psr.ERR_ARG, bad
    assert linear_call(psr, ws=8) == psr.ERR_ARG
    assert linear_call(psr, dict(act=2), bwd=True, z=None) == psr.ERR_ARG
    assert linear_call(psr, None, True, 8) == psr.ERR_ARG


def kv4_call(psr, what, shape=None, ws=1 << 30, **over):
    sh = psr.Kv4Shape(2, 4, 2, 3, 64, 16, 10, 4, psr.BF16, 0.0)
    for k, v in (shape or {}).items():
        setattr(sh, k, v)
    a = dict(sh=sh, k=PTR, ks=_st(), v=PTR, vs=_st(), cache=PTR, table=PTR, start=PTR, count=None, lse=PTR, wsp=PTR)
    a.update(over)
    lib = psr.load()
    if what == "append":
        return lib.psr_kv4_append(a["sh"], a["k"], a["ks"], a["v"], a["vs"], a["cache"], a["table"], a["start"], a["count"], None)
    if what == "read":
        return lib.psr_kv4_read(a["sh"], a["cache"], a["table"], a["start"], a["count"], a["k"], a["v"], None)
    return lib.psr_kv4_attn(a["sh"], a["k"], a["ks"], a["cache"], a["table"], a["start"], a["v"], a["vs"], a["lse"], a["wsp"],
                            ws, None)


def test_kv4_refuses(psr):
    for what in ("append", "read", "attn"):
        names = dict(append=("k", "ks", "v", "vs"), read=("k", "v"), attn=("k", "ks", "v", "vs", "lse", "wsp"))[what]
        for name in names + ("sh", "cache", "table", "start"):
            assert kv4_call(psr, what, **{name: None}) == psr.ERR_ARG, (what, name)
        for name in ("k", "v", "cache", "table", "start") + (("lse", "wsp") if what == "attn" else ("count",)):
            assert kv4_call(psr, what, **{name: PTR + 1}) == psr.ERR_ARG, (what, name)
        assert kv4_call(psr, what, cache=PTR + 8) == psr.ERR_ARG
        for bad in (dict(B=-1), dict(S=-1), dict(Hq=0), dict(Hkv=0), dict(n_pages=0), dict(max_pages=0), dict(type=2), dict(type=-1)):
            assert kv4_call(psr, what, bad) == psr.ERR_ARG, bad
        for bad in (dict(Hq=5), dict(d=96), dict(page=8), dict(page=24), dict(page=512), dict(max_pages=1 << 27)):
            assert kv4_call(psr, what, bad) == psr.ERR_UNSUPPORTED, bad
    assert kv4_call(psr, "attn", ws=8) == psr.ERR_ARG


# ---- refusals of the binding -------------------------------------------------------------------------

@pytest.fixture
def fake_device(monkeypatch):
    monkeypatch.setattr(torch.Tensor, "is_cuda", property(lambda self: True))


BF = torch.bfloat16


def test_binding_wants_cuda_tensors(psr):
    q = torch.zeros((1, 2, 4, 64), dtype=BF)
    with pytest.raises(ValueError, match="q must be a CUDA tensor"):
        psr.rotary(q, None, torch.zeros(32, dtype=torch.int64))
    with pytest.raises(ValueError, match="x must be a CUDA tensor"):
        psr.linear(torch.zeros((4, 8), dtype=BF), torch.zeros((8, 8), dtype=BF))
    with pytest.raises(ValueError, match="k must be a CUDA tensor"):
        psr.kv4_append(q, q, None, None, None, page=16)
    with pytest.raises(ValueError, match="q must be a CUDA tensor"):
        psr.kv4_attn(q, None, None, None, Hkv=2, page=16)


def test_rotary_binding_refuses(psr, fake_device):
    q, k, table = torch.zeros((2, 4, 6, 64), dtype=BF), torch.zeros((2, 2, 6, 64), dtype=BF), torch.zeros(32, dtype=torch.int64)
    bad = lambda match, *a, **kw: _refused(psr.rotary, match, *a, **kw)
    bad("q must be 4-d", q[0], k, table)
    bad("q must be bfloat16", q.double(), k.double(), table)
    bad("k must have shape", q, k[:, :, :5], table)
    bad("k must be torch.bfloat16", q, k.half(), table)
    bad("table must be torch.int64", q, k, table.float())
    bad("table must have shape", q, k, table.view(2, 16))
    bad("positions must have shape", q, k, table, positions=torch.zeros(5, dtype=torch.int64))
    bad("positions must have shape", q, k, table, positions=torch.zeros((3, 6), dtype=torch.int64))
    bad("positions must be torch.int64", q, k, table, positions=torch.zeros(6, dtype=torch.int32))
    bad("last axis must be contiguous", q.transpose(2, 3).contiguous().transpose(2, 3), k, table)
    bad("k_out without k", q, None, table, k_out=k)
    bad("q_out must have shape", q, k, table, q_out=k)
    bad("elements overlap", q, k, table, q_out=torch.zeros((1, 4, 6, 64), dtype=BF).expand(2, 4, 6, 64))
    bad("elements overlap", q, k, table, q_out=torch.zeros(4096, dtype=BF).as_strided((2, 4, 6, 64), (1536, 384, 32, 1)))
    whole = torch.zeros((2, 4, 7, 64), dtype=BF)
    bad("overlaps an input", whole[:, :, :6], None, table, q_out=whole[:, :, 1:])


def _refused(f, match, *a, **kw):
    with pytest.raises(ValueError, match=match):
        f(*a, **kw)


def test_linear_binding_refuses(psr, fake_device):
    x, w = torch.zeros((4, 16), dtype=BF), torch.zeros((24, 16), dtype=BF)
    b, r = torch.zeros(24, dtype=BF), torch.zeros((4, 24), dtype=BF)
    bad = lambda match, *a, **kw: _refused(psr.linear, match, *a, **kw)
    bad("x must be 2-d", x[0], w)
    bad("x must be bfloat16 or float16", x.float(), w.float())
    bad("w must have shape", x, w[:, :8])
    bad("w must be torch.bfloat16", x, w.half())
    bad("activation must be", x, w, activation="tanh")
    bad("bias must have shape", x, w, b[:3])
    bad("bias must be torch.bfloat16", x, w, b.float())
    bad("bias must be contiguous", x, w, torch.zeros(48, dtype=BF)[::2])
    bad("residual must have shape", x, w, b, r.t())
    bad("rows must be contiguous", torch.zeros((16, 4), dtype=BF).t(), w)
    bad("rows must not overlap", torch.zeros((1, 16), dtype=BF).expand(4, 16), w)
    bad("out must have shape", x, w, out=r[:3])
    bad("overlaps an input", x, torch.zeros((16, 16), dtype=BF), out=x)
    bad("overlaps an input", x, w, b, r, out=r, z=r)
    big = torch.zeros((5, 24), dtype=BF)
    bad("overlaps an input", x, w, None, big[:4], out=big[1:])
    bwd = lambda match, *a, **kw: _refused(psr.linear_bwd, match, *a, **kw)
    bwd("dy must have shape", r[:3], x, w)
    bwd("needs the forward's z", r, x, w, activation="gelu")
    bwd("z must have shape", r, x, w, r[:2], activation="gelu")
    bwd("dw must have shape", r, x, w, dw=w[:3])
    bwd("db must be torch.bfloat16", r, x, w, db=b.float())
    bwd("overlaps an input", r, x, w, dx=x)


def test_kv4_binding_refuses(psr, fake_device):
    cache = torch.zeros((6, 2, 16 * 72), dtype=torch.uint8)
    k, table, n = torch.zeros((3, 2, 4, 64), dtype=BF), torch.zeros((3, 2), dtype=torch.int32), torch.zeros(3, dtype=torch.int32)
    bad = lambda match, *a, **kw: _refused(psr.kv4_append, match, *a, page=kw.pop("page", 16), **kw)
    bad("k must be bfloat16 or float16", k.float(), k.float(), cache, table, n)
    bad("v must have shape", k, k[:, :1], cache, table, n)
    bad("cache must have shape", k, k, cache, table, n, page=32)
    bad("cache must have shape", k[:, :1], k[:, :1], cache, table, n)
    bad("cache must be torch.uint8", k, k, cache.int(), table, n)
    bad("cache must be contiguous", k, k, cache.transpose(0, 1).contiguous().transpose(0, 1), table, n)
    bad("table must be torch.int32", k, k, cache, table.long(), n)
    bad("table must have shape", k, k, cache, table[:2], n)
    bad("start must have shape", k, k, cache, table, n[:2])
    bad("count must be torch.int32", k, k, cache, table, n, count=n.long())
    bad = lambda match, *a, **kw: _refused(psr.kv4_read, match, *a, S=4, Hkv=kw.pop("Hkv", 2), d=64, page=16, **kw)
    bad("cache must have shape", cache, table, n, Hkv=1)
    bad("dtype must be bfloat16 or float16", cache, table, n, dtype=torch.float32)
    bad("k must have shape", cache, table, n, k=k[:, :, :3])
    q = torch.zeros((3, 4, 1, 64), dtype=BF)
    bad = lambda match, *a, **kw: _refused(psr.kv4_attn, match, *a, Hkv=2, page=16, **kw)
    bad("q must be 4-d", q[0], cache, table, n)
    bad("q must be bfloat16 or float16", q.float(), cache, table, n)
    bad("lens must have shape", q, cache, table, n[:1])
    bad("out must be torch.bfloat16", q, cache, table, n, out=q.half())
    bad("lse must be contiguous", q, cache, table, n, lse=torch.zeros((3, 4, 2))[..., :1])
    bad("overlaps an input", q, cache, table, n, out=q)
    bad("elements overlap", q, cache, table, n, out=torch.zeros((3, 1, 1, 64), dtype=BF).expand(3, 4, 1, 64))


def test_outputs_that_share_memory(psr, fake_device):
    q, k, table = torch.zeros((2, 4, 6, 64), dtype=BF), torch.zeros((2, 4, 6, 64), dtype=BF), torch.zeros(32, dtype=torch.int64)
    _refused(psr.rotary, "overlaps the other input", q, k, table, q_out=k)
    _refused(psr.rotary, "overlaps the other input", q, k, table, k_out=q)
    out = torch.zeros_like(q)
    _refused(psr.rotary, "the outputs overlap", q, k, table, q_out=out, k_out=out)
    x, w = torch.zeros((16, 16), dtype=BF), torch.zeros((16, 16), dtype=BF)
    dy, g = torch.zeros((16, 16), dtype=BF), torch.zeros((16, 16), dtype=BF)
    _refused(psr.linear_bwd, "the outputs overlap", dy, x, w, dx=g, dw=g)
    _refused(psr.linear_bwd, "the outputs overlap", dy, x, w, dw=g, db=g[3])


def test_columns_of_the_same_rows_are_apart(psr):
    rows = torch.zeros((5, 40), dtype=BF)
    apart = lambda a, b: psr._check_apart(a, b, "linear", False)
    apart(rows[:, 16:], rows[:, :16])
    apart(rows[:, :16], rows[:, 16:])
    apart(rows[1:, :16], rows[:-1, 16:])
    apart(rows[:-1, 30:], rows[1:, :30])
    for a, b in ((rows[:, 15:], rows[:, :16]), (rows[:, :17], rows[:, 16:]), (rows[1:, 10:], rows[:-1, :11]),
                 (rows[:, :8], rows[::2, 8:16])):
        with pytest.raises(ValueError, match="overlaps an input"):
            apart(a, b)


def test_linear_operands_off_their_boundary(psr):
    # off a 16-byte boundary only where the shape says so, and the workspace grows by a copy
    for bit, name in ((1, "x"), (2, "w"), (4, "y")):
        assert linear_call(psr, bwd=name == "y", **{name: PTR + 2}) == psr.ERR_ARG, name
        size = lambda odd: psr.load().psr_linear_workspace_bytes(psr.LinearShape(300, 400, 512, 0, 0, 0, 0, 0, 0, 0, odd), 1)
        assert size(bit) - size(0) >= 2 * {1: 300 * 512, 2: 400 * 512, 4: 300 * 400}[bit]
    assert linear_call(psr, dict(odd=8)) == linear_call(psr, dict(odd=-1)) == psr.ERR_ARG


def test_outputs_and_workspaces_share_nothing_with_other_tensors(psr, fake_device):
    cache = torch.zeros((6, 2, 16 * 72), dtype=torch.uint8)
    raw = torch.zeros(1 << 20, dtype=torch.uint8)
    at = lambda first, shape, dtype: raw[first:first + int(np.prod(shape)) * dtype.itemsize].view(dtype).view(shape)
    q, table, n = at(0, (3, 4, 1, 64), BF), at(2048, (3, 2), torch.int32), at(3000, (3,), torch.int32)
    attn = lambda match, **kw: _refused(psr.kv4_attn, match, q, cache, table, n, Hkv=2, page=16, **kw)
    for first in (1536 - 48, 2048 - 44, 2048, 3000, 3008):
        attn("overlaps an input", lse=at(first, (3, 4, 1), torch.float32))
        attn("the workspace overlaps a tensor", workspace=raw[first:])
    attn("overlaps an input", lse=cache.view(-1)[:48].view(torch.float32).view(3, 4, 1))
    out = at(8192, (3, 4, 1, 64), BF)
    attn("the outputs overlap", out=out, lse=at(8192, (3, 4, 1), torch.float32))
    attn("the workspace overlaps a tensor", out=out, workspace=raw[9000:])
    attn("the workspace overlaps a tensor", lse=at(8192, (3, 4, 1), torch.float32), workspace=raw[4096:])
    attn("overlaps an input", out=at(3008 - 1536 + 8, (3, 4, 1, 64), BF))
    read = lambda match, **kw: _refused(psr.kv4_read, match, cache, table, n, S=4, Hkv=2, d=64, page=16, **kw)
    read("overlaps an input", k=at(2016, (3, 2, 4, 64), BF))
    read("overlaps an input", count=at(9000, (3,), torch.int32), v=at(8192, (3, 2, 4, 64), BF))
    x, w, b, r = at(0, (4, 16), BF), at(4096, (24, 16), BF), at(8192, (24,), BF), at(12288, (4, 24), BF)
    for t in (x, w, b, r):
        _refused(psr.linear, "the workspace overlaps a tensor", x, w, b, r, workspace=raw[t.storage_offset() * t.element_size() + 2:])
    _refused(psr.linear, "the workspace overlaps a tensor", x, w, out=r, workspace=raw[8192:])
    _refused(psr.linear, "the workspace overlaps a tensor", x, w, z=r, workspace=raw[8192:])
    for kw in (dict(dx=at(16384, (4, 16), BF)), dict(dw=at(16384, (24, 16), BF)), dict(db=at(16384, (24,), BF)), dict(z=at(16384, (4, 24), BF))):
        _refused(psr.linear_bwd, "the workspace overlaps a tensor", r, x, w, activation="relu" if "z" in kw else "none",
                 workspace=raw[16000:], **kw)
    f = lambda first: at(first, (1, 1, 1, 64), torch.float32)
    freq, pos = at(2048, (32,), torch.int64), at(4096, (1,), torch.int64)
    for out in (f(2048), f(4096 - 252)):
        _refused(psr.rotary, "overlaps an input", f(0), None, freq, positions=pos, q_out=out)
        _refused(psr.rotary, "overlaps an input", f(0), f(1024), freq, positions=pos, k_out=out)


def test_overlap_of_a_row_without_a_stride(psr, fake_device):
    row = torch.zeros(16, dtype=BF).as_strided((1, 16), (0, 1))
    _refused(psr.linear, "overlaps an input", row, torch.zeros((16, 16), dtype=BF), out=row)


@pytest.mark.parametrize("scale", [float("nan"), float("inf"), float("-inf")])
def test_kv4_attention_refuses_a_scale_that_is_not_finite(psr, scale):
    assert kv4_call(psr, "attn", dict(scale=scale)) == psr.ERR_ARG
