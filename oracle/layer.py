"""fp64 oracles of the layer operators around the ring (numpy; written from the definitions):
rotary positions, the linear layer and its gradients, the 4-bit cache and its attention.

Inputs are float64 arrays that hold the bf16 / fp16 / fp32 values exactly.
"""
from __future__ import annotations

import math
from fractions import Fraction

import numpy as np

# rounding of a value to a type is off by at most this fraction of it
HALF_STEP = {"bf16": 2.0**-8, "f16": 2.0**-11, "f32": 2.0**-24}


def shard_positions(S, P, balanced):
    """Global position of every stored row (load-balanced: shard r holds half-chunks r and 2P-1-r)."""
    if not balanced:
        return np.arange(S)
    c = S // P // 2
    return np.concatenate([np.concatenate([np.arange(r * c, (r + 1) * c),
                                           np.arange((2 * P - 1 - r) * c, (2 * P - r) * c)]) for r in range(P)])


def frequencies(rot, base=10000.0, scaling="plain", factor=1.0, original=0.0, fast=32.0, slow=1.0):
    """Radians per position of each pair."""
    out = []
    for i in range(rot // 2):
        f = base ** (-2.0 * i / rot)
        if scaling == "linear":
            f = f / factor
        elif scaling == "by_parts":
            pair = lambda turns: rot * math.log(original / (turns * 2 * math.pi)) / (2 * math.log(base))
            lo, hi = max(math.floor(pair(fast)), 0), min(math.ceil(pair(slow)), rot - 1)
            mix = min(1.0, max(0.0, (i - lo) / max(hi - lo, 0.001)))
            f = f * (1 - mix) + f / factor * mix
        out.append(f)
    return np.array(out)


def rotary(x, pos, freq, amplitude=1.0, interleaved=False, inverse=False):
    """x [B, H, S, d], pos [B or 1, S] (Python integers: no overflow), freq radians per position."""
    y = np.array(x, dtype=np.float64)
    n = len(freq)
    # the angle modulo a turn from exact integers: the frequency as a fraction with a 2^200 denominator
    one = 1 << 200
    ang = np.empty((len(pos), len(pos[0]), n))
    for i, f in enumerate(freq):
        m, e = math.frexp(f / (2 * math.pi))
        turns = int(m * 2**53) << (200 + e - 53)
        for b, row in enumerate(pos):
            ang[b, :, i] = [(int(p) * turns % one) / one * 2 * math.pi for p in row]
    if inverse:
        ang = -ang
    c, s = np.cos(ang)[:, None] * amplitude, np.sin(ang)[:, None] * amplitude
    a, b = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if interleaved else (slice(0, n), slice(n, 2 * n))
    x1, x2 = np.array(x[..., a]), np.array(x[..., b])
    y[..., a], y[..., b] = x1 * c - x2 * s, x2 * c + x1 * s
    return y


_erfc = np.vectorize(math.erfc, otypes=[np.float64])


def act(z, name):
    if name == "relu":
        return np.maximum(z, 0.0)
    if name == "gelu":
        return 0.5 * z * _erfc(-z / math.sqrt(2))  # (1 + erf loses the left tail)
    if name == "gelu_tanh":
        return 0.5 * z * (1 + np.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z**3)))
    if name == "silu":
        return z / (1 + np.exp(-z))
    return z


def act_slope(z, name):
    if name == "relu":
        return (z > 0).astype(np.float64)
    if name == "gelu":
        return 0.5 * _erfc(-z / math.sqrt(2)) + z * np.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if name == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        t = np.tanh(c * (z + 0.044715 * z**3))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z)
    if name == "silu":
        s = 1 / (1 + np.exp(-z))
        return s * (1 + z * (1 - s))
    return np.ones_like(z)


def linear(x, w, bias=None, residual=None, name="none"):
    """(y, z)"""
    z = x @ w.T + (0.0 if bias is None else bias)
    return act(z, name) + (0.0 if residual is None else residual), z


def linear_bwd(dy, x, w, z=None, name="none"):
    """(dx, dw, db, dz)"""
    dz = dy * act_slope(z, name) if name != "none" else dy
    return dz @ w, dz.T @ x, dz.sum(0), dz


def to_bf16(v):
    """float32 values rounded to bf16 (half to even), as float32."""
    u = np.ascontiguousarray(v, dtype=np.float32).view(np.uint32).astype(np.uint64)
    u = ((u + 0x7FFF + ((u >> 16) & 1)) >> 16).astype(np.uint32) << 16
    return u.astype(np.uint32).view(np.float32)


def _step(low, high):
    """(high - low) / 15 as the nearest bf16 number (half to even), from exact fractions."""
    exact = (Fraction(float(high)) - Fraction(float(low))) / 15
    near = int(to_bf16(np.float32([float(exact)])).view(np.uint32)[0]) >> 16
    value = lambda bits: Fraction(float(np.array([bits << 16], np.uint32).view(np.float32)[0]))
    bits = min((c for c in (near - 1, near, near + 1) if c >= 0), key=lambda c: (abs(value(c) - exact), c & 1))
    return float(value(bits))


kv4_step = np.vectorize(_step, otypes=[np.float64])


def kv4_quantise(x):
    """(codes uint8, scale, offset) of rows x [..., d], as the format defines them: the codes' steps in float32."""
    x = x.astype(np.float32)
    with np.errstate(all="ignore"):
        mn, mx = x.min(-1, keepdims=True), x.max(-1, keepdims=True)
        fine = np.isfinite(x).all(-1, keepdims=True)
        scale = kv4_step(np.where(fine, mn, 0), np.where(fine, mx, 0)).astype(np.float32)
        off = to_bf16(np.where(fine, mn, 0))
        f = np.where(scale < 1e37, np.float32(1), np.float32(0.0625))  # a distance may pass the largest float32
        c = np.clip(np.rint((x * f - off * f) / (scale * f)), 0, 15)
    c = np.where(fine & (scale > 0), c, 0).astype(np.uint8)
    nan = np.float32("nan")
    return c, np.where(fine, scale, nan), np.where(fine, off, nan)


def kv4_place(cache, table, page, b, h, pos, d):
    """(block bytes, row) of a position: a view of cache [n_pages, Hkv, page (d + 8)]."""
    pg = int(table[b, pos // page])
    at = pos % page
    n = 16 * (d + 8)
    return cache[pg, h, at // 16 * n:(at // 16 + 1) * n], at % 16


def kv4_write_row(cache, table, page, b, h, pos, kv, row):
    """Quantise one row into the cache (kv: 0 = K, 1 = V)."""
    d = len(row)
    blk, r = kv4_place(cache, table, page, b, h, pos, d)
    c, s, o = kv4_quantise(row)
    blk[kv * 8 * d + r * (d // 2):kv * 8 * d + (r + 1) * (d // 2)] = c[0::2] | (c[1::2] << 4)
    pair = (np.concatenate([s, o]).astype(np.float32).view(np.uint32) >> 16).astype(np.uint16)
    blk[16 * d + kv * 64 + r * 4:16 * d + kv * 64 + r * 4 + 4] = pair.view(np.uint8)


def kv4_row(cache, table, page, b, h, pos, kv, d):
    """(codes, scale, offset) of one row, float64."""
    blk, r = kv4_place(cache, table, page, b, h, pos, d)
    raw = blk[kv * 8 * d + r * (d // 2):kv * 8 * d + (r + 1) * (d // 2)]
    c = np.stack([raw & 15, raw >> 4], -1).reshape(d).astype(np.float64)
    pair = blk[16 * d + kv * 64 + r * 4:16 * d + kv * 64 + r * 4 + 4].copy().view(np.uint16).astype(np.uint32) << 16
    s, o = pair.astype(np.uint32).view(np.float32).astype(np.float64)
    return c, s, o


def kv4_attention(q, cache, table, lens, page, Hkv, scale):
    """q [B, Hq, S, d] -> (o, lse, tol_o, tol_lse): the tolerances are bounds on what the arithmetic of the
    kernel may be off by before the final rounding of o.

    Scores: q.c is summed in fp32 from exact products, at most d roundings (or truncations, 2^-23) of sum |q| c (c <= 15)
    and of sum |q|; so score j is off by at most
        e_j = scale * d * 2^-23 * sum |q| (15 s_j + |o_j|) + 2^-21 |x_j|,
    LSE by max e + 2^-20 (1 + |LSE|), each weight by the fraction 2 max e + 2^-20.  Output: the weight times s_j is rounded
    to fp16 (2^-11; 2^-25 of the largest such product where it is subnormal) and multiplies c - 8, as the difference of two
    products; the sums in fp32 add n 2^-23 of their terms' sizes, s (c + 8) and |o + 8 s|."""
    B, Hq, S, d = q.shape
    o = np.zeros((B, Hq, S, d))
    lse = np.full((B, Hq, S), -np.inf)
    tol_o, tol_lse = np.zeros((B, Hq, S, d)), np.zeros((B, Hq, S))
    for b in range(B):
        n = int(lens[b])
        if n <= 0:
            continue
        for h in range(Hkv):
            rows = [[kv4_row(cache, table, page, b, h, j, kv, d) for j in range(n)] for kv in (0, 1)]
            (kc, ks, ko), (vc, vs, vo) = ([np.array(a) for a in zip(*r)] for r in rows)
            k, v = kc * ks[:, None] + ko[:, None], vc * vs[:, None] + vo[:, None]
            for hq in range(h * (Hq // Hkv), (h + 1) * (Hq // Hkv)):
                for i in range(S):
                    m = n - S + i + 1
                    if m <= 0:
                        continue
                    x = k[:m] @ q[b, hq, i] * scale
                    top = x.max()
                    w = np.exp(x - top)
                    lse[b, hq, i] = top + math.log(w.sum())
                    w = w / w.sum()
                    o[b, hq, i] = w @ v[:m]
                    size = np.abs(q[b, hq, i]).sum()
                    e = scale * d * 2.0**-23 * size * (15 * np.abs(ks[:m]) + np.abs(ko[:m])) + 2.0**-21 * np.abs(x)
                    e = float(e.max())
                    tol_lse[b, hq, i] = e + 2.0**-20 * (1 + abs(lse[b, hq, i]))
                    tol_o[b, hq, i] = (2.0**-11 * (w @ (np.abs(vc[:m] - 8) * vs[:m, None])) + m * 15 * 2.0**-25 * (w * vs[:m]).max()
                                       + (2 * e + 2.0**-20) * (w @ np.abs(v[:m]) + np.abs(o[b, hq, i]))
                                       + (m + 32) * 2.0**-23 * (w @ (31 * vs[:m] + np.abs(vo[:m]))))
    return o, lse, tol_o, tol_lse
