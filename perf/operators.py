"""The operators of one attention layer around the ring, as cases that can be timed and compared.

Three families: rotary positions for Q and K (forward and backward), the linear layer with bias, activation and
residual (forward and backward), and the 4-bit KV cache (append and read back, attention over its pages).  With
`own` false every case runs in elementary torch operations in 32 bits; with `own` true it makes the library's calls.

A page of the cache holds, for each KV head, page/16 blocks of 16 tokens (head dim d): 16 rows of d/2 bytes of K codes
(two codes to a byte, the even column in the low nibble), 16 rows of V codes, then 16 (scale, offset) bf16 pairs of K,
then of V.  A code c stands for offset + scale * c.
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZE = {"bf16": 2, "f16": 2, "f32": 4}
TWO_PI = 2.0 * math.pi


# ---- cases ---------------------------------------------------------------------------------------

def listed():
    return [
        # rotary: one new token of each of 32 sequences, each at its own position (latency)
        dict(name="rotary token", op="rotary", B=32, S=1, Hq=32, Hkv=8, d=128, rot=128, inter=False, P=1, causal=1,
             given=True, factor=1.0, back=False, fused=True, type="bf16"),
        # the whole ring's Q and K, views of one QKV projection, into the ring's layout, load-balanced shards
        dict(name="rotary ring", op="rotary", B=1, S=32768, Hq=32, Hkv=8, d=128, rot=128, inter=False, P=16, causal=2,
             given=False, factor=1.0, back=False, fused=True, type="bf16"),
        # gradients of interleaved pairs in part of the head, stretched positions, an odd length
        dict(name="rotary grad part", op="rotary", B=2, S=4099, Hq=16, Hkv=16, d=64, rot=48, inter=True, P=1, causal=1,
             given=False, factor=4.0, back=True, fused=False, type="f16"),
        # linear: the projection of a single token, with bias and residual
        dict(name="linear token", op="linear", M=1, N=8192, K=8192, act="none", bias=True, res=True, z=False,
             back=False, type="bf16"),
        # a serving batch through the wide matrix of a feed-forward block
        dict(name="linear batch", op="linear", M=24, N=28672, K=8192, act="silu", bias=False, res=False, z=False,
             back=False, type="bf16"),
        # odd sizes
        dict(name="linear ragged", op="linear", M=1531, N=5000, K=1736, act="relu", bias=True, res=False, z=False,
             back=False, type="f16"),
        # training forward: z is kept for the backward pass
        dict(name="linear train", op="linear", M=8192, N=8192, K=8192, act="gelu", bias=True, res=True, z=True,
             back=False, type="bf16"),
        # training backward: dx, dw and db
        dict(name="linear grad", op="linear", M=4100, N=8192, K=4096, act="gelu_tanh", bias=True, res=False, z=True,
             back=True, type="bf16"),
        # cache: a chunk of prompt tokens appended behind earlier ones, and read back for the ring
        dict(name="kv4 append", op="kv4_append", B=4, S=2000, Hkv=8, d=128, page=64, type="bf16"),
        # one sequence, one token (latency)
        dict(name="kv4 token", op="kv4_attn", B=1, Sq=1, Hq=32, Hkv=8, d=128, page=64, lo=4000, hi=4000, type="bf16"),
        # long contexts
        dict(name="kv4 long", op="kv4_attn", B=8, Sq=1, Hq=32, Hkv=8, d=128, page=64, lo=90000, hi=131072,
             type="bf16"),
        # many ragged sequences, four draft tokens each, small pages, no shared heads
        dict(name="kv4 draft", op="kv4_attn", B=48, Sq=4, Hq=16, Hkv=16, d=64, page=16, lo=1, hi=9000, type="f16"),
    ]


def log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["rotary", "linear", "linear", "kv4_append", "kv4_attn", "kv4_attn"])
    if op == "rotary":
        B, d, P = rng.choice([1, 2, 3, 16]), rng.choice([64, 80, 96, 128]), rng.choice([1, 1, 4, 8])
        S = log_int(rng, 1, 32768 // B)
        if P > 1:
            S = max(1, S // (2 * P)) * 2 * P
        Hkv = rng.choice([1, 4, 8])
        return dict(op=op, B=B, S=S, Hq=Hkv * rng.choice([1, 2, 4]), Hkv=Hkv, d=d,
                    rot=rng.choice([d, d, d // 2, d // 4 * 3 // 2 * 2]), inter=rng.random() < 0.4, P=P,
                    causal=2 if P > 1 and rng.random() < 0.7 else 1, given=rng.random() < 0.3,
                    factor=rng.choice([1.0, 1.0, 4.0, 8.0]), back=rng.random() < 0.4, fused=rng.random() < 0.5,
                    type=rng.choice(["bf16", "bf16", "f16", "f32"]))
    if op == "linear":
        back = rng.random() < 0.35
        N, K = 8 * log_int(rng, 8, 1024), 8 * log_int(rng, 8, 1024)
        M = log_int(rng, 1, max(1, min(8192, (1 << 37) // (N * K))))
        act = rng.choice(["none", "relu", "gelu", "gelu_tanh", "silu"])
        return dict(op=op, M=M, N=N, K=K, act=act, bias=rng.random() < 0.6, res=not back and rng.random() < 0.5,
                    z=not back and rng.random() < 0.4, back=back, type=rng.choice(["bf16", "bf16", "f16"]))
    Hkv, d, page = rng.choice([1, 2, 4, 8]), rng.choice([64, 128, 128]), rng.choice([16, 32, 64, 128])
    if op == "kv4_append":
        B = rng.choice([1, 2, 5, 32])
        return dict(op=op, B=B, S=log_int(rng, 1, 16384 // B), Hkv=Hkv, d=d, page=page,
                    type=rng.choice(["bf16", "bf16", "f16"]))
    B = log_int(rng, 1, 64)
    hi = log_int(rng, 1, min(131072, (1 << 22) // (B * Hkv)))
    return dict(op=op, B=B, Sq=rng.choice([1, 1, 1, 2, 3, 5, 8]), Hq=Hkv * rng.choice([1, 2, 4, 5, 8]), Hkv=Hkv, d=d,
                page=page, lo=max(0, hi // rng.choice([1, 2, 50])), hi=hi, type=rng.choice(["bf16", "bf16", "f16"]))


def lens_of(case):
    """Cached lengths: spread between lo and hi, the longest first."""
    lo, hi = case["lo"], case["hi"]
    return [hi - int((hi - lo) * ((b * 0.6180339887498949) % 1.0)) for b in range(case["B"])]


# ---- inputs --------------------------------------------------------------------------------------

def inv_freq(rot, base, factor, original):
    """rot/2 frequencies in radians per position, float64.  factor 1: base^(-2i/rot).  Otherwise frequencies that turn
    less than once over the original length are divided by the factor, those that turn more than 32 times are kept,
    and the ones between are blended linearly in the dimension index."""
    i = torch.arange(0, rot, 2, dtype=torch.float64)
    f = base ** (-i / rot)
    if factor == 1.0:
        return f

    def dim(turns):
        return rot * math.log(original / (turns * TWO_PI)) / (2.0 * math.log(base))
    low, high = max(math.floor(dim(32.0)), 0), min(math.ceil(dim(1.0)), rot - 1)
    ramp = ((i / 2 - low) / max(high - low, 0.001)).clamp(0.0, 1.0)
    return f * (1.0 - ramp) + f / factor * ramp


def amplitude_of(factor):
    return 1.0 if factor == 1.0 else 0.1 * math.log(factor) + 1.0


def rotary_positions(case):
    """Position of every stored row of the sequence axis (contiguous or load-balanced shards)."""
    S, P = case["S"], case["P"]
    s = torch.arange(S, dtype=torch.int64)
    if case["causal"] != 2:
        return s
    half = S // P // 2
    r, i = s // (2 * half), s % (2 * half)
    return torch.where(i < half, r * half + i, (2 * P - 1 - r) * half + i - half)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    dev, t = "cuda", TYPES[case["type"]]

    def normal(*shape, std=1.0):
        return (torch.randn(shape, generator=g, device=dev, dtype=torch.float32) * std).to(t)

    op = case["op"]
    if op == "rotary":
        B, S, Hq, Hkv, d = (case[k] for k in ("B", "S", "Hq", "Hkv", "d"))
        if case["fused"]:  # views of a QKV projection's rows
            qkv = normal(B, S, Hq + 2 * Hkv, d)
            q, k = qkv[:, :, :Hq].transpose(1, 2), qkv[:, :, Hq:Hq + Hkv].transpose(1, 2)
        else:
            q, k = normal(B, Hq, S, d), normal(B, Hkv, S, d)
        turns = inv_freq(case["rot"], 10000.0, case["factor"], 4096) / TWO_PI
        table = (turns * 2.0 ** 64).to(torch.int64).to(dev)
        pos = None
        if case["given"]:
            pos = torch.randint(0, 131072, (B, S), generator=g, device=dev, dtype=torch.int64)
        return dict(case=case, q=q, k=k, table=table, positions=pos, rows=rotary_positions(case).to(dev),
                    amplitude=amplitude_of(case["factor"]))
    if op == "linear":
        M, N, K = case["M"], case["N"], case["K"]
        s = dict(case=case, x=normal(M, K), w=normal(N, K, std=K ** -0.5))
        s["bias"] = normal(N, std=0.5) if case["bias"] else None
        if case["back"]:
            s["dy"] = normal(M, N)
            s["z"] = normal(M, N) if case["act"] != "none" else None
        else:
            s["res"] = normal(M, N) if case["res"] else None
        return s
    Hkv, d, page, B = case["Hkv"], case["d"], case["page"], case["B"]
    if op == "kv4_append":
        S = case["S"]
        start = [(37 * b + 5) % 300 for b in range(B)]
        need = [(x + S + page - 1) // page for x in start]
        k = normal(B, Hkv, S, d) * normal(1, Hkv, 1, d).abs()
        v = normal(B, Hkv, S, d)
    else:
        lens = lens_of(case)
        need = [(n + page - 1) // page for n in lens]
    wide = max(1, max(need))
    n_pages = sum(need) + 3
    order = torch.randperm(n_pages, generator=g, device=dev)
    cpu = torch.full((B, wide), -1, dtype=torch.int64)
    at = 0
    for b, n in enumerate(need):
        cpu[b, :n] = torch.arange(at, at + n)
        at += n
    table = cpu.to(dev)
    table = torch.where(table >= 0, order[table.clamp(min=0)], table).to(torch.int32)
    blocks = n_pages * Hkv * page // 16
    cache = torch.empty((blocks, 16 * (d + 8)), dtype=torch.uint8, device=dev)
    cache[:, :16 * d] = torch.randint(0, 256, (blocks, 16 * d), generator=g, device=dev, dtype=torch.uint8)
    scale = 0.12 + 0.2 * torch.rand((blocks, 32, 1), generator=g, device=dev)
    off = -7.5 * scale + 0.3 * torch.randn((blocks, 32, 1), generator=g, device=dev)
    cache[:, 16 * d:] = torch.cat([scale, off], -1).to(torch.bfloat16).reshape(blocks, 64).view(torch.uint8)
    s = dict(case=case, cache=cache.view(n_pages, Hkv, page * (d + 8)), table=table)
    if op == "kv4_append":
        s.update(k=k, v=v, start=torch.tensor(start, dtype=torch.int32, device=dev))
    else:
        s.update(q=normal(B, case["Hq"], case["Sq"], d), lens=torch.tensor(lens, dtype=torch.int32, device=dev))
    return s


# ---- plain forms ---------------------------------------------------------------------------------

def plain_rotary(x, turns, pos, sign, amplitude, inter):
    """x [B, H, S, d]; pos [B or 1, S]; the angle of a far position needs 64 bits."""
    rot = 2 * turns.numel()
    a = pos.to(torch.float64)[:, None, :, None] * turns
    a = (a - torch.floor(a)) * TWO_PI
    c, s = (torch.cos(a) * amplitude).float(), (torch.sin(a) * (sign * amplitude)).float()
    y = x.float().clone()
    if inter:
        x1, x2 = y[..., 0:rot:2].clone(), y[..., 1:rot:2].clone()
        y[..., 0:rot:2], y[..., 1:rot:2] = x1 * c - x2 * s, x2 * c + x1 * s
    else:
        x1, x2 = y[..., :rot // 2].clone(), y[..., rot // 2:rot].clone()
        y[..., :rot // 2], y[..., rot // 2:rot] = x1 * c - x2 * s, x2 * c + x1 * s
    return y.to(x.dtype)


def act_of(z, act):
    if act == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    if act == "silu":
        return z / (1 + torch.exp(-z))
    return z


def slope_of(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(TWO_PI)
    if act == "gelu_tanh":
        t = torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * z * z)
    if act == "silu":
        s = 1 / (1 + torch.exp(-z))
        return s * (1 + z * (1 - s))
    return torch.ones_like(z)


def plain_codes(x):
    """Codes, scales and offsets of rows x [..., d]."""
    x = x.float()
    mn, mx = x.amin(-1, keepdim=True), x.amax(-1, keepdim=True)
    scale = (mx / 15 - mn / 15).to(torch.bfloat16)
    off = mn.to(torch.bfloat16)
    c = torch.round((x - off.float()) / scale.float()).clamp(0, 15)
    c = torch.where(scale.float() > 0, c, torch.zeros_like(c))
    return c.to(torch.uint8), scale, off


def plain_rows(cache, table, Hkv, d, page):
    """Dequantised K and V of the tables' pages, float32 [B, Hkv, wide * page, d]."""
    B, wide = table.shape
    blk = cache.view(cache.shape[0], Hkv, page // 16, -1)[table.clamp(min=0).long()].transpose(1, 2)

    def part(codes, pair):  # of [B, Hkv, wide, page / 16, bytes]
        c = blk[..., codes:codes + 8 * d].reshape(B, Hkv, wide * page, d // 2)
        c = torch.stack([c & 15, c >> 4], -1).reshape(B, Hkv, wide * page, d).float()
        p = blk[..., pair:pair + 64].contiguous().view(torch.bfloat16).reshape(B, Hkv, wide * page, 2).float()
        return c.mul_(p[..., :1]).add_(p[..., 1:])
    return part(0, 16 * d), part(8 * d, 16 * d + 64)


def plain_append(s):
    case = s["case"]
    B, S, Hkv, d, page = (case[k] for k in ("B", "S", "Hkv", "d", "page"))
    cache = s["cache"].view(-1, Hkv, page // 16, 16 * (d + 8))
    pos = s["start"].long()[:, None] + torch.arange(S, device=cache.device)
    pg, blk, at = torch.gather(s["table"].long(), 1, pos // page), pos % page // 16, pos % 16
    pg, blk = pg[..., None, None], blk[..., None, None]
    col = torch.arange(d // 2, device=cache.device)
    byte = torch.arange(4, device=cache.device)
    out = []
    for j, x in enumerate((s["k"], s["v"])):
        c, scale, off = plain_codes(x)
        code = (c[..., 0::2] | (c[..., 1::2] << 4)).permute(0, 2, 1, 3)
        pair = torch.cat([scale, off], -1).contiguous().view(torch.uint8).permute(0, 2, 1, 3)
        head = torch.arange(Hkv, device=cache.device)[:, None]
        cache[pg, head, blk, (j * 8 * d + at * (d // 2))[..., None, None] + col] = code
        cache[pg, head, blk, (16 * d + j * 64 + at * 4)[..., None, None] + byte] = pair
        out.append((off.float() + scale.float() * c.float()).to(x.dtype))
    return tuple(out)


def plain_attn(s):
    case = s["case"]
    B, Sq, Hq, Hkv, d, page = (case[k] for k in ("B", "Sq", "Hq", "Hkv", "d", "page"))
    k, v = plain_rows(s["cache"], s["table"], Hkv, d, page)
    q = s["q"].float().view(B, Hkv, Hq // Hkv * Sq, d)
    x = torch.matmul(q, k.transpose(2, 3)) / math.sqrt(d)
    x = x.view(B, Hkv, Hq // Hkv, Sq, -1)
    last = s["lens"].long()[:, None] - Sq + torch.arange(Sq, device=q.device)
    keep = torch.arange(x.shape[-1], device=q.device) <= last[..., None]
    x = torch.where(keep[:, None, None], x, torch.full_like(x, float("-inf")))
    m = x.amax(-1, keepdim=True)
    m = torch.where(torch.isfinite(m), m, torch.zeros_like(m))
    p = torch.exp(x - m)
    t = p.sum(-1, keepdim=True)
    o = torch.matmul((p / torch.where(t > 0, t, torch.ones_like(t))).view(B, Hkv, -1, x.shape[-1]), v)
    lse = (m + torch.log(t)).view(B, Hq, Sq)
    return o.view(B, Hq, Sq, d).to(s["q"].dtype), lse


def run(s):
    case = s["case"]
    op = case["op"]
    if own:
        import persistent_sm_ring_gb300 as psr
        if op == "rotary":
            f = psr.rotary_bwd if case["back"] else psr.rotary
            return f(s["q"], s["k"], s["table"], P=case["P"], causal=case["causal"], positions=s["positions"],
                     interleaved=case["inter"], amplitude=s["amplitude"])
        if op == "linear" and case["back"]:
            dx, dw, db, _ = psr.linear_bwd(s["dy"], s["x"], s["w"], s["z"], activation=case["act"],
                                           need_db=case["bias"])
            return (dx, dw, db) if case["bias"] else (dx, dw)
        if op == "linear":
            y, z, _ = psr.linear(s["x"], s["w"], s["bias"], s["res"], activation=case["act"], save_z=case["z"])
            return (y, z) if case["z"] else (y,)
        if op == "kv4_append":
            psr.kv4_append(s["k"], s["v"], s["cache"], s["table"], s["start"], page=case["page"])
            return psr.kv4_read(s["cache"], s["table"], s["start"], S=case["S"], Hkv=case["Hkv"], d=case["d"],
                                page=case["page"], dtype=s["k"].dtype)
        o, lse, _ = psr.kv4_attn(s["q"], s["cache"], s["table"], s["lens"], Hkv=case["Hkv"], page=case["page"])
        return o, lse
    if op == "rotary":
        turns = s["table"].to(torch.float64) * 2.0 ** -64
        pos = s["rows"][None] if s["positions"] is None else s["positions"]
        sign = -1.0 if case["back"] else 1.0
        return tuple(plain_rotary(x, turns, pos, sign, s["amplitude"], case["inter"]) for x in (s["q"], s["k"]))
    if op == "linear" and case["back"]:
        dz = s["dy"].float()
        if case["act"] != "none":
            dz = dz * slope_of(s["z"].float(), case["act"])
        out = [torch.matmul(dz, s["w"].float()), torch.matmul(dz.t(), s["x"].float())]
        if case["bias"]:
            out.append(dz.sum(0))
        return tuple(o.to(s["x"].dtype) for o in out)
    if op == "linear":
        z = torch.matmul(s["x"].float(), s["w"].float().t())
        if s["bias"] is not None:
            z = z + s["bias"].float()
        y = act_of(z, case["act"])
        if s["res"] is not None:
            y = y + s["res"].float()
        t = s["x"].dtype
        return (y.to(t), z.to(t)) if case["z"] else (y.to(t),)
    return plain_append(s) if op == "kv4_append" else plain_attn(s)


# ---- what a pass cannot do without ---------------------------------------------------------------

def work(case):
    op, es = case["op"], SIZE[case["type"]]
    if op == "rotary":
        n = case["B"] * case["S"] * (case["Hq"] + case["Hkv"])
        extra = case["B"] * case["S"] * 8 if case["given"] else 0
        return {"bytes": 2 * n * case["d"] * es + case["rot"] * 4 + extra, "flops": 3 * n * case["rot"]}
    if op == "linear":
        M, N, K = case["M"], case["N"], case["K"]
        if case["back"]:
            n = M * N * (2 if case["act"] != "none" else 1) + 2 * (M * K + N * K) + (N if case["bias"] else 0)
            return {"bytes": n * es, "flops": 4 * M * N * K}
        n = M * K + N * K + M * N * (1 + case["res"] + case["z"]) + (N if case["bias"] else 0)
        return {"bytes": n * es, "flops": 2 * M * N * K}
    Hkv, d = case["Hkv"], case["d"]
    if op == "kv4_append":
        rows = case["B"] * case["S"] * Hkv
        return {"bytes": rows * (2 * d * es + (d + 8) + 2 * d * es), "flops": rows * 2 * d * 6}
    total = sum(lens_of(case))
    rows = case["B"] * case["Hq"] * case["Sq"]
    return {"bytes": total * Hkv * (d + 8) + rows * (2 * d * es + 4) + total // case["page"] * 4,
            "flops": 4 * total * case["Hq"] * case["Sq"] * d}


# ---- the definitions in 64 bits ------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    f8, op = torch.float64, case["op"]
    if op == "rotary":
        f = inv_freq(case["rot"], 10000.0, case["factor"], 4096).to("cuda")
        pos = (s["rows"][None].expand(case["B"], -1) if s["positions"] is None else s["positions"]).to(f8)
        ang = pos[..., None] * f * (-1.0 if case["back"] else 1.0)
        turn = torch.polar(torch.full_like(ang, s["amplitude"]), ang)[:, None]
        out = []
        for x in (s["q"], s["k"]):
            y, n = x.to(f8), case["rot"] // 2
            head, tail = y[..., :2 * n], y[..., 2 * n:]
            pairs = head.unflatten(-1, (n, 2)) if case["inter"] else head.unflatten(-1, (2, n)).transpose(-1, -2)
            z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
            z = z.flatten(-2) if case["inter"] else z.transpose(-1, -2).flatten(-2)
            out.append(torch.cat([z, tail], -1))
        return tuple(out)
    if op == "linear":
        x, w, act = s["x"].to(f8), s["w"].to(f8), case["act"]
        if case["back"]:
            dz = s["dy"].to(f8)
            if act != "none":
                z = s["z"].to(f8)
                if act == "relu":
                    d = torch.heaviside(z, torch.zeros((), dtype=f8, device=z.device))
                elif act == "gelu":
                    d = torch.special.ndtr(z) + z * (-(z ** 2) / 2).exp() * (0.5 / math.pi) ** 0.5
                elif act == "silu":
                    d = z.sigmoid() + z * z.sigmoid() * (-z).sigmoid()
                else:  # 0.5 z (1 + tanh u) = z sigmoid(2u)
                    c = (2 / math.pi) ** 0.5
                    u2, du2 = 2 * c * (z + 0.044715 * z ** 3), 2 * c * (1 + 0.134145 * z ** 2)
                    d = u2.sigmoid() + z * u2.sigmoid() * (-u2).sigmoid() * du2
                dz = dz * d
            out = (dz @ w, dz.T @ x)
            return out + (dz.sum(0),) if case["bias"] else out
        z = x @ w.T
        if s["bias"] is not None:
            z += s["bias"].to(f8)
        if act == "relu":
            y = z.clamp(min=0)
        elif act == "gelu":
            y = z * torch.special.ndtr(z)
        elif act == "silu":
            y = z * z.sigmoid()
        elif act == "gelu_tanh":
            y = z * (2 * (2 / math.pi) ** 0.5 * (z + 0.044715 * z ** 3)).sigmoid()
        else:
            y = z
        if s["res"] is not None:
            y = y + s["res"].to(f8)
        return (y, z) if case["z"] else (y,)
    B, Hkv, d, page = case["B"], case["Hkv"], case["d"], case["page"]
    if op == "kv4_append":
        out = []
        for x in (s["k"], s["v"]):
            y = x.to(f8)
            step = ((y.amax(-1) - y.amin(-1)) / 15).float().to(torch.bfloat16).to(f8)[..., None]
            low = y.amin(-1).to(torch.bfloat16).to(f8)[..., None]
            n = ((y - low) / torch.where(step > 0, step, torch.ones_like(step))).round().clamp(0, 15)
            out.append(low + torch.where(step > 0, n * step, torch.zeros_like(n)))
        return tuple(out)
    lens, Sq, Hq = lens_of(case), case["Sq"], case["Hq"]
    o = torch.zeros((B, Hq, Sq, d), dtype=f8, device="cuda")
    lse = torch.full((B, Hq, Sq), -math.inf, dtype=f8, device="cuda")
    for b, n in enumerate(lens):
        used = (n + page - 1) // page
        if not used:
            continue
        raw = s["cache"][s["table"][b, :used].long()].view(used, Hkv, page // 16, 16 * (d + 8))
        both = []
        for j in (0, 1):
            codes = raw[..., j * 8 * d:(j + 1) * 8 * d].reshape(used, Hkv, page, d // 2).to(torch.int32)
            pair = raw[..., 16 * d + 64 * j:16 * d + 64 * j + 64].contiguous().view(torch.bfloat16)
            pair = pair.view(used, Hkv, page, 2).to(f8)
            val = torch.empty((used, Hkv, page, d), dtype=f8, device="cuda")
            val[..., 0::2] = pair[..., :1] * (codes % 16) + pair[..., 1:]
            val[..., 1::2] = pair[..., :1] * (codes // 16) + pair[..., 1:]
            both.append(val.transpose(0, 1).reshape(Hkv, used * page, d)[:, :n])
        k, v = both
        for i in range(Sq):
            m = n - Sq + i + 1  # keys that query i sees
            if m < 1:
                continue
            qi = s["q"][b, :, i].to(f8).view(Hkv, Hq // Hkv, d)
            x = qi @ k[:, :m].transpose(1, 2) * d ** -0.5
            lse[b, :, i] = x.logsumexp(-1).reshape(-1)
            o[b, :, i] = (x.softmax(-1) @ v[:, :m]).reshape(Hq, d)
    return o, lse
