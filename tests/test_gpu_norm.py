"""bsf8_quant_norm against its formula in float64.

The kernel computes in F64 with two stated roundings (the stream h; the norm n,
F32), so what it writes is off the exact value by those roundings and by F64
noise: a sum of K terms in any order is within K 2^-53 relative of the exact
sum of squares, so 1/sqrt is within (K + 8) 2^-53, and the few products and
sums around it add some 2^-53 each of the terms they add.  The tolerances below
count exactly that.  The codes and scales are compared bit for bit with the
oracle's quantizer on the F32 norm the same call returns, and the second norm
is checked on the h the call stored.
"""
import numpy as np
import pytest

import block_scaled_fp8_linear_amd as B
import oracle as O
from gpu_util import banner, device, torch

pytestmark = pytest.mark.gpu

EPS = 1e-6


def _bf16(a):
    return O.f32_to_bf16(np.asarray(a, np.float32))


def _dev(a, dtype, pad=0, shift=0):
    """Array [M, K] on the device as float32 or bfloat16, rows ``pad`` elements longer than K, the base ``shift``
    elements into its allocation."""
    t = torch()
    a2 = np.atleast_2d(np.asarray(a, np.float32))
    M, K = a2.shape
    dt = t.bfloat16 if dtype == "bf16" else t.float32
    flat = t.full((M * (K + pad) + shift,), 7.0, dtype=dt, device=device())
    v = flat[shift:].view(M, K + pad)[:, :K]
    v.copy_(t.from_numpy(a2))
    return v if np.ndim(a) == 2 else v[0]


def _np(t_):
    return t_.float().cpu().numpy().astype(np.float64)


def _norm64(v, kind):
    """(mean, 1/sqrt) of float64 rows."""
    mean = v.mean(-1, keepdims=True) if kind == "layer" else np.zeros_like(v[:, :1])
    return mean, 1.0 / np.sqrt(((v - mean) ** 2).mean(-1, keepdims=True) + EPS)


def check(M, K, kind="rms", x="bf16", h="bf16", w="bf16", post=False, bias=False, gate="none", residual=True, top=0,
          plain="f32", pad=0, shift=0, token_major=False, inplace=False, alpha=0.75, gain=1.0, seed=0):
    t = torch()
    banner(f"quant_norm M={M} K={K} {kind} x={x} h={h} w={w} post={post} bias={bias} gate={gate} res={residual} "
           f"top={top} n={plain} pad={pad} shift={shift} tm={token_major} inplace={inplace}")
    g = np.random.default_rng(1000 + seed)
    R = M * top + 3 if top else M
    cast = lambda a, d: _bf16(a) if d == "bf16" else np.asarray(a, np.float32)
    xs_ = cast(gain * g.standard_normal((R, K)), x)
    res = cast(gain * 2 * g.standard_normal((M, K)), h)
    vec = lambda near: cast(near + 0.2 * g.standard_normal(K), w)
    wn, wp, bn, bp = vec(1.0), vec(1.0), vec(0.0), vec(0.0)
    gt = cast(0.5 + 0.2 * g.standard_normal((M, K) if gate == "token" else K), w) if gate != "none" else None
    kw = dict(kind=kind, eps=EPS, residual_scale=alpha)
    if top:
        slots = g.permutation(R)[:M * top].reshape(M, top).astype(np.int32)
        drop = g.random((M, top))
        slots[drop < 0.1] = -1
        slots[drop > 0.95] = R          # beyond the rows: nothing
        slots[M // 2] = -1              # a token without any row
        probs = g.random((M, top)).astype(np.float32)
        kw.update(slots=t.from_numpy(slots).to(device()), probs=t.from_numpy(probs).to(device()))
    xd = _dev(xs_, x, pad, shift)
    if residual:
        kw["residual"] = _dev(res, h, pad, shift)
    hd = _dev(np.zeros((M, K)), h, pad, shift)
    if inplace:
        hd = kw["residual"] if residual else xd
    if residual or h != x or inplace:
        kw["h"] = hd
    if post:
        kw["post_weight"] = _dev(wp, w, shift=shift)
        if bias:
            kw["post_bias"] = _dev(bp, w, shift=shift)
    if bias:
        kw["bias"] = _dev(bn, w, shift=shift)
    if gt is not None:
        kw["gate"] = _dev(gt, w, pad if gate == "token" else 0, shift)
    Kb = -(-K // 128)
    xq = t.full((M, K + pad), 0x5A, dtype=t.uint8, device=device())
    xs = t.full((M, Kb + pad) if token_major else (Kb, M + pad), -1.0, dtype=t.float32, device=device())
    nd = _dev(np.zeros((M, K)), plain, pad, shift)
    n2 = nd.as_strided((M, K + pad), (K + pad, 1)) if pad else nd
    q, s, hh, n = B.quant_norm(xd, _dev(wn, w, shift=shift), xq=xq[:, :K],
                               xs=xs[:, :Kb] if token_major else xs[:, :M].t(), out=nd, **kw)
    t.cuda.synchronize()
    assert q.data_ptr() == xq.data_ptr() and n is nd

    # ---- the stream
    f = np.float64
    if top:
        o, mag = np.zeros((M, K)), np.zeros((M, K))
        for j in range(top):
            ok = (slots[:, j] >= 0) & (slots[:, j] < R)
            term = np.where(ok, probs[:, j], 0.0).astype(f)[:, None] * xs_[np.where(ok, slots[:, j], 0)].astype(f)
            o += term
            mag += np.abs(term)
    else:
        o = xs_.astype(f)
        mag = np.abs(o)
    noise = 2.0 ** -52 * (K + 64)
    if post:
        mean, r = _norm64(o, kind)
        mag = (mag + np.abs(mean)) * r * np.abs(wp) + (np.abs(bp) if bias else 0)
        # with a row that is all one value up to rounding the statistics' own error shows: bounded by the row's largest
        o = (o - mean) * r * wp.astype(f) + (bp.astype(f) if bias else 0.0)
    if gt is not None:
        o, mag = o * gt.astype(f), mag * np.abs(gt)
    h64 = o + (alpha * res.astype(f) if residual else 0.0)
    mag = mag + (np.abs(alpha * res) if residual else 0.0)
    if hh is not None:
        stored = _np(hh)
        half = 2.0 ** -24 + (2.0 ** -8 if h == "bf16" else 0.0) * (1 + 2.0 ** -24)
        tol = half * np.abs(h64) + noise * mag + 2.0 ** -126
        assert np.all(np.abs(stored - h64) <= tol), np.max(np.abs(stored - h64) / tol)
    else:
        stored = (_bf16(h64.astype(np.float32)) if h == "bf16" else h64.astype(np.float32)).astype(f)

    # ---- the norm of the stored stream
    mean, r = _norm64(stored, kind)
    n64 = (stored - mean) * r * wn.astype(f) + (bn.astype(f) if bias else 0.0)
    mag = (np.abs(stored) + np.abs(mean)) * r * np.abs(wn) + (np.abs(bn) if bias else 0.0)
    got = _np(nd)
    half = 2.0 ** -24 + (2.0 ** -8 * (1 + 2.0 ** -24) if plain == "bf16" else 0.0)
    tol = half * np.abs(n64) + noise * mag + 2.0 ** -126
    assert np.all(np.abs(got - n64) <= tol), np.max(np.abs(got - n64) / tol)

    # ---- codes and scales of the F32 norm
    if plain == "f32":
        q_ref, s_ref = O.quant_act(nd.cpu().numpy().astype(np.float32))
        s_got = (xs[:, :Kb] if token_major else xs[:, :M].t()).cpu().numpy()
        assert np.array_equal(s_got.view(np.uint32), s_ref.view(np.uint32)), "scales differ"
        assert np.array_equal(xq[:, :K].cpu().numpy(), q_ref), "codes differ"
    if pad:
        assert bool((xq[:, K:] == 0x5A).all()) and bool((n2[:, K:].float() == 7.0).all())
        assert bool((xs[:, Kb:] == -1.0).all() if token_major else (xs[:, M:] == -1.0).all())
    return nd, xq, xs, hh


# every thread count and register depth: K up to 512 takes a wave, to 2048 .. 8192 one to four vectors of 256
# threads, beyond two or four of 1024; widths that end inside a vector, a scale group and a wave
@pytest.mark.parametrize("K", [1, 5, 127, 128, 512, 513, 2040, 2048, 2049, 4096, 5000, 5120, 6145, 7168, 8191, 8192,
                               8193, 16384, 17408, 32768])
@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_widths(K, kind):
    check(3, K, kind, post=K % 2 == 0, bias=kind == "layer", gate="row", seed=K)


@pytest.mark.parametrize("x,h,w", [(a, b, c) for a in ("bf16", "f32") for b in ("bf16", "f32") for c in ("bf16", "f32")])
@pytest.mark.parametrize("K", [384, 4096])
def test_types(x, h, w, K):
    check(9, K, "layer", x=x, h=h, w=w, post=True, bias=True, gate="token", seed=3)


@pytest.mark.parametrize("terms", [dict(residual=False), dict(residual=False, h="f32"), dict(gate="token"),
                                   dict(post=True), dict(post=True, bias=True, kind="layer"), dict(plain="bf16"),
                                   dict(residual=False, post=True, gate="row"), dict(token_major=True, pad=8),
                                   dict(pad=8), dict(pad=3), dict(shift=1), dict(shift=1, pad=5, x="f32", h="f32", w="f32"),
                                   dict(inplace=True), dict(inplace=True, residual=False), dict(gain=1e15), dict(gain=1e-20),
                                   dict(alpha=0.0), dict(alpha=-3.0)],
                         ids=lambda d: "-".join(f"{k}_{v}" for k, v in d.items()))
@pytest.mark.parametrize("M,K", [(1, 640), (6, 5000), (5, 200)])
def test_terms(terms, M, K):
    check(M, K, **terms)


@pytest.mark.parametrize("top", [1, 2, 8])
@pytest.mark.parametrize("M,K,x", [(1, 256, "bf16"), (17, 2048, "f32"), (40, 5120, "bf16"), (3, 9000, "bf16")])
def test_combine(M, K, x, top):
    check(M, K, x=x, top=top, post=top == 2, seed=top)


def test_many_rows():
    check(2051, 1408, post=True, gate="row")
    check(4099, 130, kind="layer", bias=True)


def test_zero_and_equal_rows():
    """Rows of zeros (rms: eps alone; the quantizer's amax floor) and rows of one value (layer: variance zero)."""
    t = torch()
    banner("quant_norm zero rows")
    x = t.zeros((4, 640), dtype=t.float32, device=device())
    x[2:] = 3.5
    w = t.ones(640, dtype=t.float32, device=device())
    xq, xs, h, n = B.quant_norm(x, w, kind="layer", out_dtype=t.float32)
    assert h is None and bool((n == 0).all()) and bool((xq == 0).all())
    assert bool((xs == np.float32(1e-10) / np.float32(448.0)).all())
    xq, xs, h, n = B.quant_norm(x, w, kind="rms", out_dtype=t.float32)
    assert bool((n[:2] == 0).all())
    assert np.allclose(n[2:].cpu().numpy(), 3.5 / np.sqrt(3.5 ** 2 + EPS), rtol=2.0 ** -23, atol=0)


def test_both_roundings():
    """The stream and the norm are rounded to F32 and then to BF16: 1 + 2^-8 + 2^-40 is 1 + 2^-8 in F32, the midpoint
    of 1 and 1 + 2^-7, and so 1 in BF16 (one rounding from F64 would give 1 + 2^-7)."""
    t = torch()
    banner("quant_norm roundings")
    K = 256
    one = t.ones((2, K), device=device())
    w = t.ones(K, device=device())
    x = t.zeros((2, K), device=device()).bfloat16()
    _, _, h, n = B.quant_norm(x, w, residual=one.bfloat16(), residual_scale=1 + 2.0 ** -8 + 2.0 ** -40, eps=1e-300,
                              out_dtype=t.bfloat16)
    assert bool((h == 1.0).all())
    # the rms norm of ones is 1 up to 2^-40, times the weight (1 + 2^-8), plus a bias that F32 rounds away
    wd = t.full((K,), 1 + 2.0 ** -8, device=device())
    for bias, want in ((2.0 ** -30, 1.0), (2.0 ** -22, 1 + 2.0 ** -7)):
        n = B.quant_norm(one, wd, bias=t.full((K,), bias, device=device()), eps=1e-300, quantize=False,
                         out_dtype=t.bfloat16)[3]
        assert bool((n == want).all()), bias


def test_fused_equals_its_parts():
    """One call gives what the same steps in separate calls give, bit for bit: the stream first, then its norm."""
    t = torch()
    banner("quant_norm fused against parts")
    g = t.Generator(device=device())
    g.manual_seed(5)
    M, K = 33, 4000
    rnd = lambda *s: t.randn(*s, generator=g, device=device())
    x, res = rnd(M, K).bfloat16(), rnd(M, K).bfloat16()
    w, wp, gt = rnd(K), rnd(K), rnd(K)
    xq, xs, h, _ = B.quant_norm(x, w, residual=res, gate=gt, post_weight=wp)
    xq2, xs2, h2, n2 = B.quant_norm(h, w, out_dtype=t.float32)
    assert h2 is None and t.equal(xq, xq2) and t.equal(xs, xs2)
    xq3, xs3 = B.quant_act(n2)
    assert t.equal(xq, xq3) and t.equal(xs, xs3)
    none = B.quant_norm(h, w, quantize=False, out_dtype=t.float32)
    assert none[0] is None and none[1] is None and t.equal(none[3], n2)


def test_empty():
    t = torch()
    w = t.ones(64, device=device())
    xq, xs, h, n = B.quant_norm(t.empty((0, 64), device=device()), w, out_dtype=t.float32)
    assert xq.shape == (0, 64) and n.shape == (0, 64)
    # experts that got no row at all: the sum is zero
    sl = t.full((2, 3), -1, dtype=t.int32, device=device())
    res = t.ones((2, 64), device=device())
    banner("quant_norm without expert rows")
    xq, xs, h, n = B.quant_norm(t.empty((0, 64), device=device()), w, slots=sl, probs=t.ones((2, 3), device=device()),
                                residual=res, residual_scale=2.0)
    assert bool((h == 2.0).all())


def test_graph_and_another_stream():
    t = torch()
    banner("quant_norm captured")
    M, K = 12, 5120
    x, res = t.randn(M, K, device=device()).bfloat16(), t.randn(M, K, device=device())
    w = t.randn(K, device=device())
    out = [t.empty((M, K), dtype=t.uint8, device=device()), B.scales_kmajor(M, K // 128, device()),
           t.empty((M, K), device=device()), t.empty((M, K), device=device())]

    def go():
        B.quant_norm(x, w, residual=res, post_weight=w, xq=out[0], xs=out[1], h=out[2], out=out[3])

    go()
    t.cuda.synchronize()
    ref = [v.clone() for v in out]
    side = t.cuda.Stream()
    side.wait_stream(t.cuda.current_stream())
    with t.cuda.stream(side):
        for v in out:
            v.zero_()
        go()
    side.synchronize()
    assert all(t.equal(a, b) for a, b in zip(out, ref))
    graph = t.cuda.CUDAGraph()
    with t.cuda.graph(graph):
        go()
    for _ in range(3):
        for v in out:
            v.zero_()
        x2 = x.clone()
        t.cuda.synchronize()
        graph.replay()
        t.cuda.synchronize()
        assert all(t.equal(a, b) for a, b in zip(out, ref)) and t.equal(x, x2)
