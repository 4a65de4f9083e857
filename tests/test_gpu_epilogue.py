"""bsf8_linear_w8a8_epilogue against the product in float64 with its bias, activation and residual."""
import numpy as np
import pytest

import block_scaled_fp8_linear_amd as B
import oracle as O
import synth
from fused_util import acc_bound, expect
from gpu_util import banner, device, member_to_device, oracle_members, raw_member_to_device, sample_rows, sample_tokens, to_np, torch

pytestmark = pytest.mark.gpu


def _real(a, dtype):
    t = torch()
    return t.from_numpy(np.asarray(a, np.float32)).to(device()).to(t.bfloat16 if dtype == "bf16" else t.float32)


def check(M, rows, K, act=None, bias="bf16", residual=None, y="bf16", f32_scales=False, token_major=False, pad=0, shift=0,
          inplace=False, full=True, seed=0):
    t = torch()
    N = sum(rows)
    ms = [synth.random_code_weight(700 + seed, f"epi_W{i}", r, K) for i, r in enumerate(rows)]
    om = oracle_members(ms)
    w = B.BlockFP8Weight([raw_member_to_device(c, s) if f32_scales else member_to_device(m) for m, (c, s) in zip(ms, om)])
    banner(f"epilogue M={M} rows={rows} K={K} act={act} bias={bias} res={residual} y={y} pad={pad} shift={shift} "
           f"inplace={inplace}: {w.describe(B.ARM_W8A8_EPILOGUE, M)}")
    g = np.random.default_rng(seed)
    q, s = O.quant_act(synth.gaussian_activations(701 + seed, f"epi_X{M}x{K}", M, K) * np.float32(0.02))
    Kb = s.shape[1]
    # NaN codes beyond K and around the tensor: none may reach a product
    buf = t.full((M * (K + pad) + shift,), 0x7F, dtype=t.uint8, device=device())
    xq = buf[shift:].view(M, K + pad)[:, :K]
    xq.copy_(t.from_numpy(q))
    if token_major:
        xs = t.from_numpy(s).to(device())
    else:
        xs = B.scales_kmajor(M, Kb, device())
        xs.copy_(t.from_numpy(s))
    b = np.asarray(g.standard_normal(N), np.float32)
    r = np.asarray(3 * g.standard_normal((M, N)), np.float32)
    kw = {}
    if bias:
        kw["bias"] = _real(b, bias)
        b = to_np(kw["bias"]).astype(np.float64)
    yt = t.bfloat16 if y == "bf16" else t.float32
    out = t.full((M, N + pad), 5.0, dtype=yt, device=device())
    if residual:
        if inplace:
            out[:, :N].copy_(_real(r, residual))
            kw["residual"] = out[:, :N]
        else:
            wide = t.zeros((M, N + pad), dtype=t.bfloat16 if residual == "bf16" else t.float32, device=device())
            wide[:, :N].copy_(_real(r, residual))
            kw["residual"] = wide[:, :N]
        r = to_np(kw["residual"].contiguous()).astype(np.float64)
        kw["residual_scale"] = 0.3
    B.linear_w8a8_epilogue(w, xq, xs, activation=act, out_dtype=yt, out=out[:, :N], **kw)
    t.cuda.synchronize()
    got = to_np(out)
    if pad:
        assert np.all(got[:, N:] == 5.0)
    cols = list(range(N)) if full else sample_rows(N, rows, 64)
    tok = np.arange(M) if full else sample_tokens(M)
    acc = O.linear_w8a8_rows(q[tok], s[tok], om, cols)
    mag = O.abs_bound_w8a8_rows(q[tok], s[tok], om, cols)
    want, tol = expect(acc, mag, K, b[cols] if bias else None, act, r[np.ix_(tok, cols)] if residual else None,
                       float(np.float32(0.3)), y == "bf16", "f8f6f4" in w.describe(B.ARM_W8A8_EPILOGUE, M) and y == "bf16")
    err = np.abs(got[np.ix_(tok, cols)] - want)
    assert not np.isnan(err).any() and np.all(err <= tol), f"worst err/tol {np.max(err / tol):.3g}"
    return out


# few rows, one to three 16-row tiles, the tile kernel and its splits; N and K that end inside tiles and blocks
@pytest.mark.parametrize("M", [1, 2, 15, 16, 17, 33, 48, 49, 64, 65, 100, 129, 257, 300])
@pytest.mark.parametrize("rows,K", [((256,), 512), ((1000,), 1408), ((300,), 1000)])
def test_sizes(M, rows, K):
    check(M, rows, K, act="silu", residual="bf16", seed=M)


@pytest.mark.parametrize("act", [None, "none", "relu", "silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("M", [3, 70])
def test_activations(act, M):
    check(M, (384,), 640, act=act, y="f32")
    check(M, (384,), 640, act=act, y="bf16", bias=None, residual="f32")


@pytest.mark.parametrize("terms", [dict(bias=None), dict(bias="f32"), dict(residual="f32"), dict(residual="bf16", y="f32"),
                                   dict(residual="f32", y="f32", inplace=True), dict(residual="bf16", inplace=True),
                                   dict(f32_scales=True), dict(token_major=True), dict(pad=16, residual="bf16"),
                                   dict(pad=3, residual="f32", y="f32", act="gelu"), dict(shift=1), dict(shift=5, pad=1)],
                         ids=lambda d: "-".join(f"{k}_{v}" for k, v in d.items()))
@pytest.mark.parametrize("M,rows,K", [(1, (512,), 2048), (40, (200, 130, 77), 1136), (150, (300, 256), 768),
                                      (200, (131,), 333)])
def test_terms(M, rows, K, terms):
    check(M, rows, K, **terms)


def test_small_k():
    for K in (1, 15, 16, 17, 32, 127, 128, 129):
        check(5, (40,), K, act="gelu", residual="f32", y="f32", seed=K)
        check(130, (40,), K, act="gelu", residual="f32", y="f32", seed=K)


@pytest.mark.parametrize("M,rows,K", [(1, (5120,), 5120), (512, (6144, 1000, 1000), 5120), (1024, (5120,), 17408),
                                      (16, (17408,), 5120)])
def test_projections(M, rows, K):
    """The repository's projection shapes, sampled as its parity tests sample them."""
    check(M, rows, K, act="gelu_tanh", residual="bf16", full=False)


def test_per_tensor_weight():
    t = torch()
    g = np.random.default_rng(7)
    N, K, M = 200, 640, 60
    codes = synth.random_code_weight(702, "epi_pt", N, K).codes
    w = B.BlockFP8Weight([(t.from_numpy(codes).to(device()), t.tensor(0.01, device=device()))], block=(0, 0))
    q, s = O.quant_act(synth.gaussian_activations(702, "epi_ptx", M, K))
    banner("epilogue per tensor")
    for m in (5, M):
        y = B.linear_w8a8_epilogue(w, t.from_numpy(q[:m]).to(device()), t.from_numpy(s[:m]).to(device()), activation="relu",
                                   out_dtype=t.float32)
        x64 = O.dequantize_act(q[:m], s[:m])
        w64 = O.e4m3_decode(codes).astype(np.float64) * float(np.float32(0.01))
        want, tol = expect(x64 @ w64.T, np.abs(x64) @ np.abs(w64).T, K, act="relu")
        assert np.all(np.abs(to_np(y) - want) <= tol)


def test_near_the_plain_product():
    """Without bias, activation and residual: the plain product's call within both calls' bounds."""
    t = torch()
    m = synth.random_code_weight(703, "epi_plain", 1000, 1408)
    w = B.BlockFP8Weight([member_to_device(m)])
    banner("epilogue against linear_w8a8")
    for M in (1, 40, 200):
        q, s = O.quant_act(synth.gaussian_activations(703, f"epi_p{M}", M, 1408))
        xq, xs = t.from_numpy(q).to(device()), t.from_numpy(s).to(device())
        a = to_np(B.linear_w8a8_epilogue(w, xq, xs, out_dtype=t.float32))
        b = to_np(B.linear_w8a8(w, xq, xs, out_dtype=t.float32))
        mag = O.abs_bound_w8a8(q, s, oracle_members([m]))
        # linear_w8a8 promises 1e-3 of the sum of magnitudes (its FP8 matrix instruction)
        assert np.all(np.abs(a - b) <= expect(a * 0, mag, 1408)[1] + acc_bound(mag, 1408, fp8_mfma=True))


def test_graph_and_another_stream():
    t = torch()
    m = synth.random_code_weight(704, "epi_graph", 640, 2048)
    w = B.BlockFP8Weight([member_to_device(m)])
    cases = []
    for M in (1, 40, 64, 300):
        xq, xs = B.quant_act(t.randn(M, 2048, device=device()))
        cases.append((xq, xs, t.randn(M, 640, device=device()).bfloat16(), t.empty((M, 640), dtype=t.bfloat16, device=device()),
                      w.workspace(B.ARM_W8A8_EPILOGUE, M)))
    bias = t.randn(640, device=device())

    def go():
        for xq, xs, r, y, ws in cases:
            B.linear_w8a8_epilogue(w, xq, xs, bias=bias, activation="silu", residual=r, out=y, workspace=ws)

    banner("epilogue captured")
    go()
    t.cuda.synchronize()
    ref = [c[3].clone() for c in cases]
    side = t.cuda.Stream()
    side.wait_stream(t.cuda.current_stream())
    with t.cuda.stream(side):
        for c in cases:
            c[3].zero_()
        go()
    side.synchronize()
    assert all(t.equal(c[3], r) for c, r in zip(cases, ref))
    graph = t.cuda.CUDAGraph()
    with t.cuda.graph(graph):
        go()
    for _ in range(3):
        for c in cases:
            c[3].zero_()
            if c[4][0] is not None:
                c[4][0].fill_(0xFF)
        t.cuda.synchronize()
        graph.replay()
        t.cuda.synchronize()
        assert all(t.equal(c[3], r) for c, r in zip(cases, ref))
