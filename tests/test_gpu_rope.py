"""Rotary positions against their definition in 64 bits."""
import numpy as np
import pytest

import block_scaled_fp8_linear_amd as B
from cache_util import rope64, rope_tolerance, to_f64
from gpu_util import banner, device, torch

pytestmark = pytest.mark.gpu


def _inputs(M, H, KV, D, R, axes, x, seed, far=200000):
    t = torch()
    g = np.random.default_rng(seed)
    dt = t.bfloat16 if x == "bf16" else t.float32
    qkv = t.from_numpy(g.standard_normal((M, H + 2 * KV, D)).astype(np.float32)).to(device()).to(dt)
    inv = (1e6 ** (-np.arange(0, R, 2) / max(R, 1))).astype(np.float32)
    pos = g.integers(-far, far, (axes, M))
    return qkv, inv, pos


def _check(got, want, x, bf16, what, **kw):
    err = np.abs(to_f64(got) - want)
    tol = rope_tolerance(want, x, bf16=bf16, **kw)
    assert (err <= tol).all(), (what, float((err / tol).max()))


# M, H, KV, D, R, axes, order, pairing, input, output, norm
CASES = [
    (1, 40, 8, 128, 128, 1, "blocks", "half", "bf16", "bf16", False),
    (1, 1, 1, 16, 16, 1, "blocks", "half", "f32", "f32", True),
    (5, 3, 2, 16, 2, 1, "blocks", "half", "f32", "f32", False),
    (7, 24, 4, 256, 64, 3, "turns", "half", "bf16", "bf16", True),
    (9, 5, 1, 256, 256, 4, "blocks", "half", "f32", "f32", True),
    (33, 7, 3, 80, 80, 2, "turns", "adjacent", "f32", "f32", False),
    (33, 7, 3, 80, 80, 2, "turns", "half", "f32", "f32", True),      # R / 2 = 40
    (4, 6, 2, 96, 20, 3, "blocks", "half", "bf16", "f32", True),     # R / 2 = 10: no multiple of a lane's channels
    (4, 6, 2, 96, 22, 3, "blocks", "adjacent", "bf16", "f32", True),  # ends inside a lane
    (3, 2, 1, 192, 192, 1, "blocks", "half", "bf16", "bf16", False),
    (6, 9, 5, 144, 144, 16, "blocks", "adjacent", "bf16", "bf16", True),
    (700, 12, 4, 64, 32, 1, "blocks", "half", "bf16", "bf16", False),
    (5000, 20, 4, 64, 64, 3, "blocks", "half", "f32", "bf16", True),  # more than one pass of heads per wave
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(v) for v in c))
def test_rope(case):
    M, H, KV, D, R, A, order, pairing, x, y, norm = case
    t = torch()
    banner(f"rope {case}")
    qkv, inv, pos = _inputs(M, H, KV, D, R, A, x, 5)
    g = np.random.default_rng(6)
    axes = None
    if A > 1:
        n = R // 2 // A
        axes = B.rope_axes([R // 2 - n * (A - 1)] + [n] * (A - 1), interleaved=order == "turns")
    w = [t.from_numpy((1 + 0.2 * g.standard_normal(D)).astype(np.float32)).to(device()).bfloat16() if norm else None
         for _ in "qk"]
    q, k = qkv[:, :H], qkv[:, H:H + KV]
    before = qkv.clone()
    ydt = t.bfloat16 if y == "bf16" else t.float32
    p = t.from_numpy(pos).to(device())
    yq, yk = B.rope(q, p[0] if A == 1 else p, t.from_numpy(inv).to(device()), k=k, axes=axes, pairing=pairing, scale=1.25,
                    q_weight=w[0], k_weight=w[1], eps=1e-5, out_dtype=ydt)
    assert yq.dtype == ydt and yq.shape == (M, H, D) and yk.shape == (M, KV, D)
    assert t.equal(before, qkv)
    for got, src, wt in ((yq, q, w[0]), (yk, k, w[1])):
        xs, ws = to_f64(src), None if wt is None else to_f64(wt)
        want = rope64(xs, pos, inv, axes, pairing, 1.25, ws, 1e-5)
        _check(got, want, xs, y == "bf16", case, scale=1.25, weight=ws, eps=1e-5)
    # queries alone give the same bits, also with 32-bit positions
    again, none = B.rope(q, (p[0] if A == 1 else p).int(), t.from_numpy(inv).to(device()), axes=axes, pairing=pairing,
                         scale=1.25, q_weight=w[0], eps=1e-5, out_dtype=ydt)
    assert none is None and t.equal(again, yq)


@pytest.mark.parametrize("pairing,R", [("half", 128), ("half", 20), ("adjacent", 128), ("half", 0)])
@pytest.mark.parametrize("x", ["bf16", "f32"])
def test_in_place_and_unaligned(pairing, R, x):
    """An output that is its input, and heads at addresses and strides that allow no wide access."""
    t = torch()
    M, H, KV, D = 37, 5, 2, 128
    qkv, inv, pos = _inputs(M, H, KV, D, R, 1, x, 11)
    p = t.from_numpy(pos[0]).to(device())
    f = t.from_numpy(inv).to(device()) if R else None
    weight = t.linspace(0.5, 1.5, D, device=device())
    args = dict(positions=p if R else None, inv_freq=f, pairing=pairing)
    want_q, want_k = B.rope(qkv[:, :H], args["positions"], f, k=qkv[:, H:H + KV], pairing=pairing, q_weight=weight)
    if R == 0:
        assert t.equal(want_k, qkv[:, H:H + KV])
    # odd pitch, odd first element
    wide = t.zeros(M, (H + 2 * KV) * D + 3, dtype=qkv.dtype, device=device())
    odd = wide[:, 1:1 + (H + 2 * KV) * D].unflatten(1, (H + 2 * KV, D))
    odd.copy_(qkv)
    keep = wide.clone()
    q, k = odd[:, :H], odd[:, H:H + KV]
    banner(f"rope in place {pairing} {R} {x}")
    gq, gk = B.rope(q, args["positions"], f, k=k, pairing=pairing, q_weight=weight, out=q, k_out=k)
    assert gq.data_ptr() == q.data_ptr() and t.equal(gq, want_q) and t.equal(gk, want_k)
    changed = odd.clone()
    assert t.equal(changed[:, H + KV:], qkv[:, H + KV:])      # the values behind are left alone
    odd.copy_(qkv)
    assert t.equal(wide, keep)                                # and so is everything around
    # the same heads head-major
    qt = qkv[:, :H].transpose(0, 1).contiguous().transpose(0, 1)
    gq, _ = B.rope(qt, args["positions"], f, pairing=pairing, q_weight=weight)
    assert t.equal(gq, want_q)


def test_far_positions():
    """Angles of positions up to 2^29 are exact products: nothing of them is lost."""
    t = torch()
    D, M = 64, 64
    g = np.random.default_rng(3)
    pos = np.concatenate([[0, 1, -1, 2 ** 29 - 1, -2 ** 29 + 1], g.integers(-2 ** 29, 2 ** 29, M - 5)])[None]
    inv = g.uniform(0.1, 1.0, D // 2).astype(np.float32)
    x = g.standard_normal((M, 2, D)).astype(np.float32)
    banner("rope far positions")
    y, _ = B.rope(t.from_numpy(x).to(device()), t.from_numpy(pos[0]).to(device()), t.from_numpy(inv).to(device()))
    want = rope64(x, pos, inv)
    _check(y, want, x, False, "far")
    # a turn keeps a pair's length: F32 roundings of both channels alone
    a, b = to_f64(y)[..., :D // 2], to_f64(y)[..., D // 2:]
    n = np.hypot(x[..., :D // 2].astype(np.float64), x[..., D // 2:].astype(np.float64))
    assert (np.abs(np.hypot(a, b) - n) <= 2.0 ** -23 * n).all()


def test_no_tokens_and_signs():
    t = torch()
    e = t.empty(0, 4, 64, device=device())
    inv = t.ones(32, device=device())
    y, k = B.rope(e, t.empty(0, dtype=t.int64, device=device()), inv, k=e)
    assert y.shape == (0, 4, 64) and k.shape == (0, 4, 64)
    # channels that do not turn are passed on, the sign of zero with them
    x = t.zeros(1, 1, 64, device=device())
    x[..., 33::2] = -0.0
    y, _ = B.rope(x, t.tensor([7], device=device()), t.ones(16, device=device()))
    assert t.equal(y.view(t.int32)[..., 32:], x.view(t.int32)[..., 32:])
