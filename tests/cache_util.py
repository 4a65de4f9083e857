"""Shared by the tests of rotary positions, the paged cache and its attention: caches of several layouts, and the
definitions in 64 bits (NumPy on the CPU)."""
import numpy as np

import block_scaled_fp8_linear_amd as B
from gpu_util import device, torch

LAYOUTS = ("head_major", "token_major", "side_by_side", "padded")


def new_cache(layout, pages, page, heads, D, codes, fill=None):
    """A PagedKVCache whose bytes are random (``fill`` None) or ``fill`` everywhere, and the tensors that hold them."""
    t = torch()
    dev = device()
    dt = t.uint8 if codes else t.bfloat16
    G = -(-D // 128)

    def make(shape, dtype):
        if fill is not None:
            return t.full(shape, fill, dtype=dtype, device=dev)
        if dtype == t.uint8:   # finite codes
            u = t.randint(0, 127, shape, dtype=t.uint8, device=dev)
            return u | (t.randint(0, 2, shape, dtype=t.uint8, device=dev) << 7)
        return t.rand(shape, device=dev).to(dtype) + 0.25

    if layout == "head_major":
        base = [make((pages, heads, page, D), dt) for _ in "kv"]
        kv = [x.transpose(1, 2) for x in base]
        sbase = [make((pages, heads, G, page), t.float32) for _ in "kv"]
        sc = [x.permute(0, 3, 1, 2) for x in sbase]
    elif layout == "token_major":
        kv = base = [make((pages, page, heads, D), dt) for _ in "kv"]
        sc = sbase = [make((pages, page, heads, G), t.float32) for _ in "kv"]
    elif layout == "side_by_side":
        base = [make((pages, 2, page, heads, D), dt)]
        kv = [base[0][:, 0], base[0][:, 1]]
        sbase = [make((2, G, heads, pages, page), t.float32)]
        sc = [sbase[0][i].permute(2, 3, 1, 0) for i in range(2)]
    else:   # heads further apart than their channels, rows further than their heads
        base = [make((pages, page, heads + 1, D + 32), dt) for _ in "kv"]
        kv = [x[:, :, :heads, 16:16 + D] for x in base]
        sbase = [make((pages, page, heads, G + 1), t.float32) for _ in "kv"]
        sc = [x[..., :G] for x in sbase]
    if not codes:
        return B.PagedKVCache(*kv), base
    return B.PagedKVCache(*kv, *sc), base + sbase


def cache_values(c):
    """(k, v) as float64 [pages, page_size, heads, D]: the product of code and scale in F32, as it is read."""
    t = torch()
    out = []
    for x, s in ((c.k, c.k_scale), (c.v, c.v_scale)):
        if s is None:
            out.append(x.float().cpu().numpy().astype(np.float64))
            continue
        v = x.contiguous().view(t.float8_e4m3fn).float().cpu().numpy()
        per = np.repeat(s.cpu().numpy(), 128, axis=-1)[..., :c.head_dim]
        out.append((v * per).astype(np.float64))
    return out


def norm64(x, weight, eps):
    x = x.astype(np.float64)
    if weight is None:
        return x
    return x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * weight.astype(np.float64)


def rope64(x, positions, inv_freq, axes=None, pairing="half", scale=1.0, weight=None, eps=1e-6):
    """The definition in 64 bits: x [M, H, D], positions [A, M], inv_freq float32 [R / 2]."""
    y = norm64(x, weight, eps)
    if inv_freq is None:
        return y
    half = inv_freq.shape[0]
    axes = np.zeros(half, int) if axes is None else np.frombuffer(bytes(axes), np.uint8).astype(int)
    angle = positions.astype(np.float64)[axes].T * inv_freq.astype(np.float64)      # [M, half]
    c, s = np.cos(angle)[:, None] * scale, np.sin(angle)[:, None] * scale
    i = np.arange(half)
    a, b = (i, i + half) if pairing == "half" else (2 * i, 2 * i + 1)
    out = y.copy()
    out[..., a] = c * y[..., a] - s * y[..., b]
    out[..., b] = c * y[..., b] + s * y[..., a]
    return out


def rope_tolerance(want, x, scale=1.0, weight=None, eps=1e-6, bf16=False):
    """One rounding to F32 (2^-24 relative), one more to BF16 (2^-8); what F64 loses (some 40 roundings of 2^-53 on either
    side, and the angle's: both sides take the same product, which they reduce to within 2^-50) on a pair's magnitude."""
    pair = np.abs(norm64(x, weight, eps)).max(-1, keepdims=True) * max(1.0, abs(scale))
    tol = 2.0 ** -24 * np.abs(want) + 2.0 ** -44 * pair + 2.0 ** -149
    return tol + (2.0 ** -8 * np.abs(want) if bf16 else 0.0)


def to_f64(x):
    return x.float().cpu().numpy().astype(np.float64)


def make_table(g, lens, page, pages, columns=None, behind=-1):
    """Pages of each sequence in random order; entries behind its last page are ``behind``."""
    need = [-(-n // page) for n in lens]
    table = np.full((len(lens), columns or max(1, max(need))), behind, np.int32)
    perm = g.permutation(pages)[:sum(need)]
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = perm[at:at + n]
        at += n
    return table


def attention64(q, values, table, lens, page, window, scale, n_pages):
    """(out, lse, tolerance of out without its own rounding, tolerance of lse) in 64 bits.

    What F32 loses, per head row (u = 2^-24; an F32 sum of N terms in any order and rounding direction is off by at most
    2 N u of the sum of their magnitudes, which also covers what a matrix instruction does inside):
      a logit: its D products and scales, at most ds = 2 (3 D + 8) u scale sum |q k| (three terms of an F32 query);
      a weight: exp(2 ds) - 1 against the exact ones' (its own logit's and the maximum's, which cancels in the quotient
        but for its rounding), the exponent's rounding, 2 u times its size in base 2, and 4 u of the hardware's exp2;
      its split into two BF16 terms: 2^-16;
      the sums over n tokens, 2 n u of sum p |v|, once for the numerator and once for the denominator, and some 64
        roundings of rescaling and joining."""
    K, V = values
    B, H, D = q.shape
    kv = K.shape[2]
    G = H // kv
    u = 2.0 ** -24
    out, lse = np.zeros((B, H, D)), np.full((B, H), -np.inf)
    tol, tol_lse = np.zeros((B, H, D)), np.zeros((B, H))
    for b, n in enumerate(lens):
        n = min(max(int(n), 0), table.shape[1] * page)
        pos = np.arange(max(0, n - window) if window else 0, n)
        pg = table[b, pos // page] if n else np.zeros(0, int)
        ok = (pg >= 0) & (pg < n_pages)
        pos, pg = pos[ok], pg[ok]
        if len(pos) == 0:
            continue
        for h in range(kv):
            k, v = K[pg, pos % page, h], V[pg, pos % page, h]
            rows = slice(h * G, (h + 1) * G)
            s = scale * (q[b, rows] @ k.T)
            m = s.max(-1, keepdims=True)
            p = np.exp(s - m)
            z = p.sum(-1, keepdims=True)
            out[b, rows] = p @ v / z
            lse[b, rows] = (m + np.log(z))[:, 0]
            ds = 2 * (3 * D + 8) * u * abs(scale) * (np.abs(q[b, rows]) @ np.abs(k).T).max(-1)
            size = np.abs(s / np.log(2)).max(-1)
            rel = np.expm1(2 * ds) + (4 * size + 8) * u + 2.0 ** -16 + (4 * len(pos) + 64) * u
            tol[b, rows] = rel[:, None] * (p @ np.abs(v) / z)
            tol_lse[b, rows] = ds + (2 * len(pos) + 64 + 4 * size) * u
    return out, lse, tol, tol_lse
