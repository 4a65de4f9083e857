"""Bounds shared by the tests of the products with an epilogue and by expert.

Codes that are decoded to BF16 (where a call's describe line says so):
an output is acc = sum over K blocks of P * (xs * sw), P an MFMA's sum of 128
exact products.  Whatever its order and rounding direction, an F32 sum of 128
terms is off by at most 127 * 2^-23 of the sum of their magnitudes; xs * sw and
its product with P add two roundings, the sum over the Kb blocks (in up to eight
parts, then the parts, or up to eight splits) Kb + 16 more of 2^-24 each.
Activations have slope below 1.13 and are evaluated within 16 * 2^-24 of |z|
(exp, erfc and division of a few units each; their arguments' roundings reach the
result times at most max |u sigma(u) (1 - sigma(u))| < 0.25), bias and residual
add a rounding each, a BF16 output half a step.
"""
import math

import numpy as np

U = 2.0 ** -24


def acc_bound(abs_sum, K, fp8_mfma=False):
    """fp8_mfma: the kernel that ran sums a block in the FP8 matrix instruction, whose internal sum is narrower than
    F32 (it feeds BF16 outputs only): the W8A8 arm's documented bound, 1e-3 of the sum of magnitudes."""
    if fp8_mfma:
        return 1e-3 * abs_sum
    return (127 * 2 + 2 + -(-K // 128) + 16) * U * abs_sum


_erfc = np.vectorize(math.erfc, otypes=[np.float64])


def act64(z, act):
    if act == "relu":
        return np.maximum(z, 0)
    if act == "silu":
        return z / (1 + np.exp(-z))
    if act == "gelu":
        return 0.5 * z * _erfc(-z / math.sqrt(2))
    if act == "gelu_tanh":
        u = 2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)
        return z / (1 + np.exp(-u))
    return z


def expect(acc, abs_sum, K, bias=None, act=None, residual=None, scale=1.0, bf16=False, fp8_mfma=False):
    """(float64 outputs, tolerance)."""
    z = acc + (bias if bias is not None else 0.0)
    zmag = np.abs(acc) + (np.abs(bias) if bias is not None else 0.0)
    with np.errstate(over="ignore"):
        v = act64(z, act)
    tol = 1.2 * acc_bound(abs_sum, K, fp8_mfma) + (20 if act not in (None, "none", "relu") else 2) * U * zmag
    if residual is not None:
        v = v + scale * residual
        tol = tol + 2 * U * (np.abs(v) + np.abs(scale * residual))
    return v, tol + (2.0 ** -8 * (np.abs(v) + tol) if bf16 else U * np.abs(v)) + 2.0 ** -126
