"""The operators at the two ends of a training step around the attention layers, as cases that can be timed and compared.

Two families: the embedding (rows of a table looked up by token and scaled, and the table's gradient) and the loss of the
output projection (softmax cross entropy of x w^T over a large vocabulary, and its gradients with respect to x and w).
With `own` false every case runs in elementary torch operations in 32 bits (64 for long sums of 32-bit rows); with `own`
true it makes the library's calls.

Loss of a row with target t, logits l = x w^T and V columns: lse - (1 - smoothing) l_t - smoothing mean(l) + z lse^2, with
lse = log sum exp l.  Rows whose target is IGNORE have a loss and a lse of 0 and no gradient.
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZE = {"bf16": 2, "f16": 2, "f32": 4}
IGNORE = -100
SPAN = 512  # rows of one sequence, whose first tokens are the prompt: their targets are ignored


# ---- cases ---------------------------------------------------------------------------------------

def listed():
    return [
        # embedding: the next token of each of 32 sequences (latency)
        dict(name="embed token", op="embed", M=32, V=128000, K=8192, scale=1.0, type="bf16"),
        # a batch of prompts, rows scaled by the square root of their length
        dict(name="embed prompt", op="embed", M=16421, V=128000, K=4096, scale=64.0, type="bf16"),
        # gradient of a large table: most rows are zeros
        dict(name="embed grad", op="embed_grad", M=16384, V=128000, K=4096, scale=1.0, type="bf16"),
        # a table of bytes: few rows, each of them the sum of thousands of tokens, columns off 16-byte boundaries
        dict(name="embed grad bytes", op="embed_grad", M=65539, V=260, K=1001, scale=1.0, type="f32"),
        # odd sizes
        dict(name="embed grad ragged", op="embed_grad", M=2047, V=50021, K=1736, scale=32.0, type="f16"),
        # loss of a single token (latency)
        dict(name="loss token", op="loss", M=1, V=32000, K=4096, smooth=0.0, z=0.0, masked=0.0, type="bf16"),
        # the log-probabilities of a few continuations
        dict(name="loss few", op="loss", M=48, V=128000, K=4096, smooth=0.0, z=0.0, masked=0.0, type="bf16"),
        # odd sizes
        dict(name="loss ragged", op="loss", M=1531, V=50021, K=1736, smooth=0.1, z=0.0, masked=0.0, type="f16"),
        # evaluation of a batch of sequences
        dict(name="loss eval", op="loss", M=8192, V=128000, K=4096, smooth=0.0, z=0.0, masked=0.0, type="bf16"),
        # loss and gradients of a short fine-tuning sample
        dict(name="step few", op="step", M=40, V=32000, K=2048, smooth=0.0, z=0.0, masked=0.0, type="bf16"),
        # loss and gradients of a pre-training batch, with a penalty on the normaliser
        dict(name="step train", op="step", M=8192, V=64000, K=4096, smooth=0.0, z=1e-4, masked=0.0, type="bf16"),
        # a fine-tuning batch: prompts without loss, smoothed targets, odd sizes
        dict(name="step masked", op="step", M=4100, V=50021, K=2000, smooth=0.05, z=0.0, masked=0.4, type="f16"),
    ]


def log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["embed", "embed_grad", "embed_grad", "loss", "loss", "step", "step"])
    if op in ("embed", "embed_grad"):
        K = rng.choice([8 * log_int(rng, 8, 1024), log_int(rng, 64, 8192)])
        V = log_int(rng, 200, 128000)
        M = log_int(rng, 1, min(65536, (1 << 26) // K))
        return dict(op=op, M=M, V=V, K=K, scale=rng.choice([1.0, 1.0, 0.37, 45.25]),
                    type=rng.choice(["bf16", "bf16", "f16", "f32"]))
    K = 8 * log_int(rng, 8, 512) + rng.choice([0, 0, 0, 4, 1])
    V = log_int(rng, 200, 128000)
    most = (1 << 40) if op == "step" else (1 << 41)
    M = log_int(rng, 1, max(1, min(16384, most // (V * K))))
    return dict(op=op, M=M, V=V, K=K, smooth=rng.choice([0.0, 0.0, 0.1]), z=rng.choice([0.0, 0.0, 1e-3]),
                masked=rng.choice([0.0, 0.0, 0.25, 0.7]), type=rng.choice(["bf16", "bf16", "f16"]))


# ---- inputs --------------------------------------------------------------------------------------

def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    dev, t = "cuda", TYPES[case["type"]]
    M, V, K = case["M"], case["V"], case["K"]

    def normal(*shape, std=1.0):
        return (torch.randn(shape, generator=g, device=dev, dtype=torch.float32) * std).to(t)

    # tokens: token v comes about 1 / (v + 1) as often as the first
    u = torch.rand(M, generator=g, device=dev, dtype=torch.float64)
    ids = (torch.exp(u * math.log(V + 1)) - 1).long().clamp(0, V - 1)
    ids = torch.randperm(V, generator=g, device=dev)[ids]
    if case["op"] == "embed":
        return dict(case=case, ids=ids, w=normal(V, K))
    if case["op"] == "embed_grad":
        return dict(case=case, ids=ids, dy=normal(M, K))
    # logits with a deviation of 2.5; each row leans towards its target, by none to a lot (losses between 1 and 14)
    w = normal(V, K, std=2.5 * K ** -0.5)
    lean = 1.5 * torch.rand((M, 1), generator=g, device=dev)
    x = (torch.randn((M, K), generator=g, device=dev) + lean * w[ids].float()).to(t)
    span = min(M, SPAN)
    prompt = torch.arange(M, device=dev) % span < int(case["masked"] * span)
    s = dict(case=case, x=x, w=w, targets=torch.where(prompt, torch.full_like(ids, IGNORE), ids))
    if case["op"] == "step":  # the mean over the rows that count; in fp16 the loss is scaled, as such training does
        each = (32768.0 if case["type"] == "f16" else 1.0) / rows_of(case)
        s["dloss"] = torch.full((1,), each, device=dev).expand(M)
    return s


def rows_of(case):
    """Rows that count: those that are not in a prompt."""
    span = min(case["M"], SPAN)
    return sum(1 for i in range(case["M"]) if i % span >= int(case["masked"] * span))


# ---- plain forms ---------------------------------------------------------------------------------

def plain_loss(s):
    """loss, lse; and what the gradients need: logits, the rows' shares of the targets, which rows count."""
    case, x, w, t = s["case"], s["x"].float(), s["w"].float(), s["targets"]
    eps, count = case["smooth"], t != IGNORE
    logits = torch.matmul(x, w.t())
    m = logits.amax(1, keepdim=True)
    lse = (m + torch.log(torch.exp(logits - m).sum(1, keepdim=True)))[:, 0]
    at = t.clamp(min=0)
    loss = lse - (1 - eps) * logits[torch.arange(len(t), device=t.device), at] + case["z"] * lse * lse
    if eps:
        loss = loss - eps * (logits.sum(1) / case["V"])
    zero = torch.zeros_like(lse)
    return torch.where(count, loss, zero), torch.where(count, lse, zero), x, w, logits, at, count


def run(s):
    case = s["case"]
    op, t = case["op"], TYPES[case["type"]]
    if own:
        import persistent_sm_ring_gb300 as psr
        if op == "embed":
            return (psr.embedding(s["ids"], s["w"], scale=case["scale"]),)
        if op == "embed_grad":
            return (psr.embedding_bwd(s["dy"], s["ids"], case["V"], scale=case["scale"])[0],)
        more = dict(smoothing=case["smooth"], z_weight=case["z"], ignore=IGNORE)
        loss, lse, _ = psr.linear_xent(s["x"], s["w"], s["targets"], **more)
        if op == "loss":
            return loss, lse
        dx, dw, _ = psr.linear_xent_bwd(s["dloss"], s["x"], s["w"], s["targets"], lse, **more)
        return loss, lse, dx, dw
    if op == "embed":
        return ((s["w"][s["ids"]].float() * case["scale"]).to(t),)
    if op == "embed_grad":
        wide = torch.float64 if t == torch.float32 else torch.float32
        dw = torch.zeros((case["V"], case["K"]), dtype=wide, device=s["dy"].device)
        dw.index_add_(0, s["ids"], s["dy"].to(wide))
        return ((dw * case["scale"]).to(t),)
    loss, lse, x, w, logits, at, count = plain_loss(s)
    if op == "loss":
        return loss, lse
    each = torch.where(count, s["dloss"], torch.zeros_like(lse))
    dl = torch.exp(logits - lse[:, None]) * (1 + 2 * case["z"] * lse)[:, None]
    dl = dl - case["smooth"] / case["V"]
    dl[torch.arange(len(at), device=at.device), at] -= 1 - case["smooth"]
    dl = torch.where(count[:, None], dl * each[:, None], torch.zeros_like(dl))
    return loss, lse, torch.matmul(dl, w).to(t), torch.matmul(dl.t(), x).to(t)


# ---- what a pass cannot do without ---------------------------------------------------------------

def work(case):
    op, es = case["op"], SIZE[case["type"]]
    M, V, K = case["M"], case["V"], case["K"]
    if op == "embed":  # the rows of the table that M tokens are expected to name
        v = torch.arange(V, dtype=torch.float64)
        p = (torch.log(v + 2) - torch.log(v + 1)) / math.log(V + 1)
        rows = float((1 - (1 - p) ** M).sum())
        return {"bytes": (M + rows) * K * es + 8 * M, "flops": M * K}
    if op == "embed_grad":
        return {"bytes": (M + V) * K * es + 8 * M, "flops": M * K}
    n = rows_of(case)
    if op == "loss":
        return {"bytes": (n + V) * K * es + 16 * M, "flops": 2 * n * V * K}
    # without the logits kept, the gradients compute them again: four products
    return {"bytes": 2 * (n + V) * K * es + 20 * M, "flops": 8 * n * V * K}


# ---- the definitions in 64 bits ------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    f8 = torch.float64
    if case["op"] == "embed":
        return (torch.index_select(s["w"], 0, s["ids"]).to(f8).mul_(case["scale"]),)
    if case["op"] == "embed_grad":  # the sum over the rows of each token, one token after another in their sorted order
        by, order = torch.sort(s["ids"], stable=True)
        total = torch.cumsum(s["dy"][order].to(f8) * case["scale"], 0)
        last = torch.ones(len(by), dtype=torch.bool, device=by.device)
        last[:-1] = by[1:] != by[:-1]
        total = total[last]
        total[1:] = total[1:] - total[:-1].clone()
        dw = torch.zeros((case["V"], case["K"]), dtype=f8, device="cuda")
        dw[by[last]] = total
        return (dw,)
    keep = torch.nonzero(s["targets"] != IGNORE)[:, 0]
    t, eps, n = s["targets"][keep], case["smooth"], case["M"]
    x, w = s["x"][keep].to(f8), s["w"].to(f8)
    logits = x @ w.T
    lse = torch.logsumexp(logits, 1)
    losses = lse + case["z"] * lse ** 2 - (1 - eps) * logits.gather(1, t[:, None])[:, 0] - eps * logits.mean(1)
    spread = lambda v: torch.zeros((n,) + v.shape[1:], dtype=f8, device="cuda").index_copy_(0, keep, v)  # noqa: E731
    if case["op"] == "loss":
        return spread(losses), spread(lse)
    d = logits.sub_(lse[:, None]).exp_().mul_((1 + 2 * case["z"] * lse)[:, None]).sub_(eps / case["V"])
    d.scatter_add_(1, t[:, None], torch.full((len(t), 1), eps - 1.0, dtype=f8, device="cuda"))
    d.mul_(s["dloss"][keep].to(f8)[:, None])
    return spread(losses), spread(lse), spread(d @ w), d.T @ x
