"""CPU tests of the embedding and of the output projection's loss: the oracle's own pins, workspace sizes, and what the C ABI and the
binding refuse before anything reaches a device."""
import numpy as np
import pytest
import torch

from oracle import ends

PTR = 1 << 20  # stands for device memory: never read, every call here ends on the host
BF = torch.bfloat16


# ---- the oracle ----------------------------------------------------------------------------------

def test_oracle_embedding():
    w = np.arange(12.0).reshape(4, 3)
    y = ends.embedding([2, 0, -1, 4], w, 2.0)
    assert np.array_equal(y[:2], 2 * w[[2, 0]]) and np.isnan(y[2:]).all()
    dy = np.array([[1.0], [2.0], [4.0], [8.0], [16.0]])
    dw, n, size = ends.embedding_bwd(dy, [1, 3, 1, 7, 3], 4, 0.5, padding=3)
    assert dw.tolist() == [[0], [2.5], [0], [0]] and n.tolist() == [0, 2, 0, 0] and size.tolist() == [[0], [2.5], [0], [0]]
    assert ends.embedding_bwd(dy, [1, 3, 1, 7, 3], 4, dw=np.ones((4, 1)))[0].tolist() == [[1], [6], [1], [19]]


def test_oracle_loss_is_the_librarys():
    rng = np.random.default_rng(0)
    x, w, t = rng.standard_normal((6, 5)), rng.standard_normal((9, 5)), [0, 8, 3, -100, 3, 1]
    for smoothing in (0.0, 0.3):
        loss, lse = ends.linear_xent(x, w, t, smoothing)
        want = torch.nn.functional.cross_entropy(torch.tensor(x @ w.T), torch.tensor(t), reduction="none", label_smoothing=smoothing)
        np.testing.assert_allclose(loss, want.numpy(), atol=1e-12)
    assert lse[3] == 0 and np.isnan(ends.linear_xent(x, w, [9] * 6)[0]).all()
    assert np.allclose(ends.linear_xent(x, w, t, z=0.5)[0], ends.linear_xent(x, w, t)[0] + 0.5 * lse**2)


@pytest.mark.parametrize("smoothing,z", [(0.0, 0.0), (0.2, 0.05)])
def test_oracle_gradients_are_differences(smoothing, z):
    rng = np.random.default_rng(1)
    x, w, g, t = rng.standard_normal((5, 4)), rng.standard_normal((7, 4)), rng.standard_normal(5), [0, 6, -100, 2, 2]
    _, lse = ends.linear_xent(x, w, t, smoothing, z)
    dx, dw = ends.linear_xent_bwd(g, x, w, t, lse, smoothing, z)
    f = lambda x, w: (ends.linear_xent(x, w, t, smoothing, z)[0] * g).sum()
    sx, sw = rng.standard_normal(x.shape), rng.standard_normal(w.shape)
    h = 1e-6
    assert abs((f(x + h * sx, w) - f(x - h * sx, w)) / (2 * h) - (dx * sx).sum()) < 1e-7
    assert abs((f(x, w + h * sw) - f(x, w - h * sw)) / (2 * h) - (dw * sw).sum()) < 1e-7


# ---- sizes ---------------------------------------------------------------------------------------

def test_workspace_sizes(psr):
    assert psr.embedding_workspace_bytes(0, 5, 8) >= 256
    assert psr.embedding_workspace_bytes(1000, 5, 8) >= 1000 * 16 + 256
    for bad in ((-1, 5, 8), (1, 0, 8), (1, 5, 0), (1 << 29, 5, 8), (1, 5, (1 << 20) + 1)):
        with pytest.raises(psr.PsrError):
            psr.embedding_workspace_bytes(*bad)
    V, K = 64000, 4096
    logits = 2 * 8192 * V
    assert 256 <= psr.linear_xent_workspace_bytes(1, V, K) < 1 << 20
    assert psr.linear_xent_workspace_bytes(8192, V, K) < logits // 4
    # backward: a piece of the slopes, x's rows and the sums of dx, whatever the vocabulary
    a, b = (psr.linear_xent_workspace_bytes(8192, v, K, backward=True) for v in (V, 4 * V))
    assert b <= a + (64 << 20) and b < (512 << 20) + 8192 * K * 6 + (96 << 20)
    for bad in ((-1, 5, 8), (1, 0, 8), (1, 5, 0), ((1 << 24) + 1, 5, 8), (1, (1 << 28) + 1, 8)):
        with pytest.raises(psr.PsrError):
            psr.linear_xent_workspace_bytes(*bad)
    for s in (-0.1, 1.0, float("nan")):
        with pytest.raises(psr.PsrError):
            psr.linear_xent_workspace_bytes(4, 5, 8, smoothing=s)


# ---- refusals of the C ABI -------------------------------------------------------------------------

def embedding_call(psr, bwd=False, shape=None, ws=1 << 30, **over):
    sh = psr.EmbeddingShape(4, 9, 16, psr.BF16, 1, 0, 0, -1, 0, 1.0)
    for k, v in (shape or {}).items():
        setattr(sh, k, v)
    a = dict(sh=sh, ids=PTR, w=PTR, y=PTR, wsp=PTR)
    a.update(over)
    if bwd:
        return psr.load().psr_embedding_bwd(a["sh"], a["y"], a["ids"], a["w"], a["wsp"], ws, None)
    return psr.load().psr_embedding(a["sh"], a["ids"], a["w"], a["y"], None)


def test_embedding_refuses(psr):
    for bwd in (False, True):
        for name in ("sh", "ids", "w", "y") + (("wsp",) if bwd else ()):
            assert embedding_call(psr, bwd, **{name: None}) == psr.ERR_ARG, name
        for name, off in (("ids", 4), ("w", 1), ("y", 1)):
            assert embedding_call(psr, bwd, **{name: PTR + off}) == psr.ERR_ARG, name
            if name != "ids":
                assert embedding_call(psr, bwd, dict(type=psr.F32), **{name: PTR + 2}) == psr.ERR_ARG, name
        for bad in (dict(M=-1), dict(V=0), dict(K=0), dict(type=3), dict(type=-1), dict(ldw=15), dict(ldy=15), dict(ldy=-16),
                    dict(scale=float("nan")), dict(scale=float("inf"))):
            assert embedding_call(psr, bwd, bad) == psr.ERR_ARG, bad
        for bad in (dict(M=(1 << 28) + 1), dict(V=(1 << 30) + 1), dict(K=(1 << 20) + 1)):
            assert embedding_call(psr, bwd, bad) == psr.ERR_UNSUPPORTED, bad
    assert embedding_call(psr, True, ws=8) == psr.ERR_ARG
    assert embedding_call(psr, True, wsp=PTR + 16) == psr.ERR_ARG


def xent_call(psr, bwd=False, shape=None, ws=1 << 40, **over):
    sh = psr.XentShape(4, 9, 16, psr.BF16, 0, 0, 1, 1, -100, 0.0, 0.0, 0)
    for k, v in (shape or {}).items():
        setattr(sh, k, v)
    a = dict(sh=sh, x=PTR, w=PTR, t=PTR, loss=PTR, lse=PTR, wsp=PTR, g=PTR, dx=PTR, dw=PTR)
    a.update(over)
    lib = psr.load()
    if bwd:
        return lib.psr_xent_bwd(a["sh"], a["g"], a["x"], a["w"], a["t"], a["lse"], a["dx"], a["dw"], a["wsp"], ws, 0, None)
    return lib.psr_xent(a["sh"], a["x"], a["w"], a["t"], a["loss"], a["lse"], a["wsp"], ws, 0, None)


def test_xent_refuses(psr):
    for bwd in (False, True):
        for name in ("sh", "x", "w", "t", "lse", "wsp") + (("g",) if bwd else ("loss",)):
            assert xent_call(psr, bwd, **{name: None}) == psr.ERR_ARG, name
        for name, off in (("x", 1), ("w", 1), ("t", 4), ("lse", 2), ("wsp", 16)) + ((("g", 2), ("dx", 1), ("dw", 1)) if bwd else (("loss", 2),)):
            assert xent_call(psr, bwd, **{name: PTR + off}) == psr.ERR_ARG, name
        assert xent_call(psr, bwd, w=PTR + 2) == psr.ERR_ARG  # off a 16-byte boundary, and not said so
        for bad in (dict(M=-1), dict(V=0), dict(K=0), dict(type=psr.F32), dict(type=-1), dict(ldx=15), dict(ldw=15), dict(odd=4),
                    dict(smoothing=1.0), dict(smoothing=-0.5), dict(smoothing=float("nan")), dict(z_weight=-1.0),
                    dict(z_weight=float("inf")), dict(z_weight=float("nan"))):
            assert xent_call(psr, bwd, bad) == psr.ERR_ARG, bad
        for bad in (dict(M=(1 << 24) + 1), dict(V=(1 << 28) + 1), dict(K=(1 << 20) + 1)):
            assert xent_call(psr, bwd, bad) == psr.ERR_UNSUPPORTED, bad
        assert xent_call(psr, bwd, ws=8) == psr.ERR_ARG
    assert xent_call(psr, False, x=PTR + 2) == psr.ERR_ARG  # (the backward pass copies x's rows)


# ---- refusals of the binding -------------------------------------------------------------------------

@pytest.fixture
def fake_device(monkeypatch):
    monkeypatch.setattr(torch.Tensor, "is_cuda", property(lambda self: True))


def _refused(f, match, *a, **kw):
    with pytest.raises(ValueError, match=match):
        f(*a, **kw)


def test_binding_wants_cuda_tensors(psr):
    ids, w = torch.zeros(4, dtype=torch.int64), torch.zeros((9, 16), dtype=BF)
    _refused(psr.embedding, "w must be a CUDA tensor", ids, w)
    _refused(psr.embedding_bwd, "dy must be a CUDA tensor", w[:4], ids, 9)
    _refused(psr.linear_xent, "x must be a CUDA tensor", w[:4], w, ids)


def test_embedding_binding_refuses(psr, fake_device):
    ids, w = torch.zeros(4, dtype=torch.int64), torch.zeros((9, 16), dtype=BF)
    bad = lambda match, *a, **kw: _refused(psr.embedding, match, *a, **kw)
    bad("ids must be torch.int64", ids.int(), w)
    bad("ids must be 1-d", ids.view(2, 2), w)
    bad("w must be 2-d", ids, w[0])
    bad("w must be bfloat16, float16 or float32", ids, w.double())
    bad("rows must be contiguous", ids, w.t())
    bad("rows must not overlap", ids, w[:1].expand(9, 16))
    bad("out must have shape", ids, w, out=w[:3])
    bad("out must be torch.bfloat16", ids, w, out=torch.zeros((4, 16)))
    bad("overlaps an input", ids, w, out=w[:4])
    bad = lambda match, *a, **kw: _refused(psr.embedding_bwd, match, *a, **kw)
    bad("ids must have shape", w[:5], ids, 9)
    bad("dw must have shape", w[:4], ids, 9, dw=w[:8])
    bad("dw must be contiguous", torch.zeros((4, 9), dtype=BF), ids, 16, dw=w.t())
    bad("accumulate adds to dw", w[:4], ids, 9, accumulate=True)
    bad("padding must be an id", w[:4], ids, 9, padding=9)
    bad("rows must not overlap", w[:1].expand(4, 16), ids, 9)
    bad("overlaps an input", w[:4], ids, 9, dw=w)
    with pytest.raises(psr.PsrError):
        psr.embedding(ids, w, scale=float("inf"))
    with pytest.raises(psr.PsrError):
        psr.embedding_bwd(w[:4], ids, 0)


def test_sizes_and_numbers_beyond_their_fields(psr, fake_device):
    """Sizes of 2^32 and more are refused, not cut to their lowest bits."""
    x, w, t, g = torch.zeros((4, 16), dtype=BF), torch.zeros((9, 16), dtype=BF), torch.zeros(4, dtype=torch.int64), torch.zeros(4)
    far = 2**32 + 5
    for call in (lambda: psr.embedding_workspace_bytes(far, 5, 8), lambda: psr.embedding_workspace_bytes(4, -far, 8),
                 lambda: psr.linear_xent_workspace_bytes(4, far, 8), lambda: psr.linear_xent_workspace_bytes(4, 5, far, backward=True),
                 lambda: psr.embedding(t[:1].expand(far), w), lambda: psr.embedding_bwd(x, t, far),
                 lambda: psr.embedding_bwd(x, t, -far)):
        with pytest.raises(psr.PsrError):
            call()
    _refused(psr.linear_xent, "ignore must be an int64", x, w, t, ignore=2**64 - 100)
    _refused(psr.linear_xent_bwd, "ignore must be an int64", g, x, w, t, g, ignore=-2**63 - 1)


def test_xent_binding_refuses(psr, fake_device):
    x, w, t, g = torch.zeros((4, 16), dtype=BF), torch.zeros((9, 16), dtype=BF), torch.zeros(4, dtype=torch.int64), torch.zeros(4)
    bad = lambda match, *a, **kw: _refused(psr.linear_xent, match, *a, **kw)
    bad("x must be bfloat16 or float16", x.float(), w.float(), t)
    bad("w must be torch.bfloat16", x, w.half(), t)
    bad("w must have shape", x, w[:, :8], t)
    bad("targets must be torch.int64", x, w, t.int())
    bad("targets must have shape", x, w, t[:3])
    bad("targets must be 1-d", x, w, t.view(2, 2))
    bad("loss must be torch.float32", x, w, t, loss=g.double())
    bad("lse must be contiguous", x, w, t, lse=torch.zeros(8)[::2])
    bad("the outputs overlap", x, w, t, loss=g, lse=g)
    bwd = lambda match, *a, **kw: _refused(psr.linear_xent_bwd, match, *a, **kw)
    bwd("dloss must be torch.float32", g.half(), x, w, t, g)
    bwd("dloss must be 1-d", g[0], x, w, t, g)
    bwd("lse must have shape", g, x, w, t, g[:2])
    bwd("lse must be contiguous", g, x, w, t, torch.zeros(8)[::2])
    bwd("dx must have shape", g, x, w, t, g, dx=w)
    bwd("dw must be contiguous", g, x, w, t, g, dw=torch.zeros((16, 9), dtype=BF).t())
    bwd("overlaps an input", g, x, w, t, g, dw=w)
    both = torch.zeros((9, 16), dtype=BF)
    bwd("the outputs overlap", g, x, w, t, g, dx=both[:4], dw=both)
    for more in (dict(smoothing=1.0), dict(z_weight=-1.0)):
        with pytest.raises(psr.PsrError):
            psr.linear_xent(x, w, t, **more)
