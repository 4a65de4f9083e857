"""The epilogue's activations over the whole range of their argument.

A product of zero codes is zero, so the argument of the activation is the bias itself, exactly.  Every routine that
applies an activation is reached: the few-row kernel, the tile kernel's whole and ragged strips, the sum of split tiles.
"""
import numpy as np
import pytest

import block_scaled_fp8_linear_amd as B
from fused_util import act64
from gpu_util import banner, device, torch

pytestmark = pytest.mark.gpu

F32, BF16 = "f32", "bf16"
# (tokens, columns, K, output): few rows; whole and ragged strips of 128 x 128 and 256 x 256 tiles; K split
PLACES = [(3, 700, 128, F32), (130, 700, 128, F32), (200, 640, 4096, F32), (3, 700, 128, BF16), (130, 700, 128, BF16),
          (1000, 8200, 512, BF16)]
ACTS = [None, "relu", "silu", "gelu", "gelu_tanh"]


def activate(values, M, N, K, out, act):
    """act(values) as a call gives it: [M, N] outputs whose columns repeat the values."""
    t = torch()
    v = np.resize(np.asarray(values, np.float32), N)
    w = B.BlockFP8Weight([(t.full((N, K), 0x38, dtype=t.uint8, device=device()),
                           t.ones((-(-N // 128), -(-K // 128)), device=device()))])
    xq = t.zeros((M, K), dtype=t.uint8, device=device())
    xs = t.ones((M, -(-K // 128)), device=device())
    banner(f"activation {act} M={M} N={N} K={K} {out}: {w.describe(B.ARM_W8A8_EPILOGUE, M)}")
    y = B.linear_w8a8_epilogue(w, xq, xs, bias=t.from_numpy(v).to(device()), activation=act,
                               out_dtype=t.float32 if out == F32 else t.bfloat16)
    y = y.double().cpu().numpy()
    assert np.array_equal(y, np.broadcast_to(y[0], y.shape), equal_nan=True)
    return v.astype(np.float64), y[0]


@pytest.mark.parametrize("M,N,K,out", PLACES)
@pytest.mark.parametrize("act", ACTS)
def test_infinities_and_huge_values(M, N, K, out, act):
    """v * Phi(v) and its like at +inf are +inf, and at -inf the formulas' -inf * 0, NaN (relu: zero); finite values of
    any size give themselves or zero."""
    big = float(np.float32(2.0 ** 127))
    v, y = activate([np.inf, -np.inf, 1e20, -1e20, big, -big, np.nan], M, N, K, out, act)
    at_minus = -np.inf if act is None else 0.0 if act == "relu" else np.nan
    want = np.where(v > 0, v, 0.0 if act is not None else v)
    want[np.isnan(v)] = np.nan
    want[v == -np.inf] = at_minus
    # (1e20 in BF16 is off by half a step; the powers of two and the rest are exact)
    assert np.array_equal(np.isnan(y), np.isnan(want))
    ok = ~np.isnan(want) & np.isfinite(want)
    assert np.array_equal(y[np.isinf(want)], want[np.isinf(want)])
    assert np.all(np.abs(y[ok] - want[ok]) <= (2.0 ** -8 if out == BF16 else 2.0 ** -24) * np.abs(want[ok]))


# How far an output may be off, relative to itself, in units of 2^-24.  The hardware's exp2 and reciprocal are within one
# unit in the last place, 2 units of 2^-24 here; every F32 operation adds one.
#  silu: exp2's argument carries its product's rounding and the constant's, 1.5 |v| 2^-24 of its natural exponent, and
#  exp2, the sum, the reciprocal and the product add 2 + 1 + 2 + 1.
#  gelu_tanh: the same with u, |u| <= 2 sqrt(2 / pi) (|v| + 0.045 |v|^3), whose own four roundings and constants make 4 |u|.
#  gelu: tail = |v| / 2 * t P(t) * exp2(-v^2 / (2 ln 2)).  exp2's argument has the square's and the product's rounding and
#  the constant's, 2.5 * v^2 / 2; t = 1 / (1 + p |v|) is off by 1 + 2 and acts on t P(t) with a slope below 3 (at v = 0),
#  the polynomial's own error is below 1, its evaluation below 4, exp2 and the products add 2 + 3.  The result is the
#  tail where v < 0 and at least as large as it where v >= 0.
def _units(v, act):
    a = np.abs(v)
    if act == "silu":
        return 6 + 1.5 * a
    if act == "gelu_tanh":
        return 6 + 5.5 * 2 * np.sqrt(2 / np.pi) * (a + 0.045 * a ** 3)
    return 19 + 1.25 * v ** 2


@pytest.mark.parametrize("M,N,K,out", [(3, 60000, 128, F32), (130, 60000, 128, F32), (200, 640, 4096, F32),
                                       (1000, 8200, 512, BF16)])
@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
def test_relative_error(M, N, K, out, act):
    """Outputs far below the argument, where the activation vanishes, are as accurate as those near it."""
    v = np.concatenate([np.linspace(-13, 13, N // 2), -np.logspace(-12, np.log10(80.0), N // 4), np.logspace(-12, 2, N // 4)])
    v, y = activate(v, M, N, K, out, act)
    want = act64(v, act)
    rel = _units(v, act) * 2.0 ** -24
    if out == BF16:
        rel = rel + 2.0 ** -8 * (1 + rel)
    # exp2 and the reciprocal know no denormals: what is below 2^-118 may be zero
    err = np.abs(y - want) - 2.0 ** -118
    bad = ~(err <= rel * np.abs(want))
    assert not bad.any(), (act, v[bad][:5], y[bad][:5], want[bad][:5])
