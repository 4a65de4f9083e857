"""Cases whose attention shows in how many BF16 terms a query and a softmax weight enter their products, and the kernel's
arithmetic on them with any number of terms.

Keys and values have one channel that is 1: token i's are at channel i, so that its logit (the scale is 1) is channel i of the
query and its weight is channel i of the output; no sum of products has a second term that is not zero.  Tokens between
them have the last channel and a logit 400 below: a weight of zero in F32.  Queries in F32 are 300 and less, so that a
third term of theirs is up to 2^-9 of a logit.

What such an output may be off by, relative to it (u = 2^-24, logits at most 1 below the largest, n tokens that count):
  a weight: the logit's difference is exact; log2(e) and its product are two roundings of at most log2(e), 2 u of the
    weight; the hardware's exp2, 1 ulp, 2 u: 4 u;
  the sum: the same, and n additions;
  the quotient's rounding, u.
One wave: (4 + 4 + n + 1) u.  Where a maximum rises from tile to tile (at most n - 1 times, its differences at most 1 in
all: 2 u of the exponential and 1 u of the product each, 2 u together) and the parts of waves and of blocks are brought to a
common one (4 u and a product's 1 each), the weight has 3 (n - 1) + 2 + 10 u more, the sum the same and some 8 additions of
parts: (9 + n + 2 (3 (n - 1) + 12) + 8) u.
A weight in two terms has 2^-17 more (half a step of the second, which is at most 2^-8 of the first), in one 2^-8."""
import numpy as np

U = 2.0 ** -24
TOKENS = 6


def tolerance(split):
    n = TOKENS
    return (9 + n + (2 * (3 * (n - 1) + 12) + 8 if split else 0)) * U


def bf16(x):
    """Float32 values rounded to BF16 (nearest, ties to even), as float32."""
    b = np.ascontiguousarray(x, np.float32).view(np.uint32).astype(np.uint64)
    return ((b + 0x7FFF + ((b >> 16) & 1)) & 0xFFFF0000).astype(np.uint32).view(np.float32)


def in_terms(x, n):
    """What n BF16 terms hold of float32 values."""
    total, rest = np.zeros_like(x), x.copy()
    for _ in range(n):
        t = bf16(rest)
        total, rest = total + t, rest - t
    return total


def queries(g, B, H, D, f32):
    """[B, H, D] float32 (BF16 values unless f32)."""
    q = np.zeros((B, H, D), np.float32)
    top = 300.0 if f32 else 0.0
    q[..., :TOKENS] = top - g.uniform(0.0, 1.0, (B, H, TOKENS))
    q[..., D - 1] = top - 400.0
    return q if f32 else bf16(q)


def exact(q):
    """(out, lse) in 64 bits; what the tokens between add (e^-396) is left out."""
    s = q[..., :TOKENS].astype(np.float64)
    m = s.max(-1, keepdims=True)
    p = np.exp(s - m)
    z = p.sum(-1, keepdims=True)
    out = np.zeros(q.shape)
    out[..., :TOKENS] = p / z
    return out, (m + np.log(z))[..., 0]


def emulate(q, q_terms, weight_terms):
    """The kernel's arithmetic in F32, one wave, before the output's own rounding."""
    s = in_terms(q, q_terms)[..., :TOKENS]
    e = (s - s.max(-1, keepdims=True)) * np.float32(1.4426950408889634)
    p = np.exp2(e.astype(np.float64)).astype(np.float32)
    l = np.zeros(p.shape[:-1], np.float32)
    for i in range(TOKENS):
        l = l + p[..., i]
    out = np.zeros(q.shape, np.float32)
    out[..., :TOKENS] = in_terms(p, weight_terms) / l[..., None]
    return out


def within(got, want, out_bf16, terms, split):
    """Whether every output is within its tolerance (terms: of a weight, 3 hold all of its bits)."""
    rel = tolerance(split) + (0.0 if terms == 3 else 2.0 ** -17)
    if out_bf16:
        rel = rel + 2.0 ** -8 * (1 + rel)
    return bool((np.abs(got - want) <= rel * np.abs(want)).all())


def norm_bound(D, largest):
    """Of |got - want| / |want| over a batch of ordinary values with F32 queries and outputs, none of whose terms is lost.  The
    outputs' errors are the weights', which are independent from token to token, so that the norm shows a single weight's:
    its logit's D / 32 additions of the matrix instruction, each u of a partial sum of at most `largest` (and as much again
    for what the instruction drops inside), which grow as the square root of their number, and the exponent's two roundings
    of a difference of at most 2 `largest`, with 4 u for the exponential and the sums."""
    return (2 * (D / 32) ** 0.5 * largest + 4 * largest + 4) * U
