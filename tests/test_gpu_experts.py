"""bsf8_linear_w8a8_experts against each expert's product in float64, and the operators of a routed layer in a row."""
import numpy as np
import pytest

import block_scaled_fp8_linear_amd as B
import oracle as O
import synth
from fused_util import acc_bound, expect
from gpu_util import banner, device, to_np, torch
from test_gpu_route import plan_ref

pytestmark = pytest.mark.gpu


def experts(E, rows, K, seed=0, f32_scales=False):
    """(handle, per expert the oracle's members)."""
    t = torch()
    ms = [[synth.random_code_weight(800 + seed, f"ex_{i}_{e}", r, K) for e in range(E)] for i, r in enumerate(rows)]
    members = []
    for mi in ms:
        w = t.from_numpy(np.stack([m.codes for m in mi])).to(device())
        if f32_scales:
            s = t.from_numpy(np.stack([m.scale_f32() for m in mi])).to(device())
        else:
            s = t.from_numpy(np.stack([m.scale_bits for m in mi]).view(np.int16)).to(device()).view(t.bfloat16)
        members.append((w, s))
    return B.ExpertsFP8Weight(members), [[(mi[e].codes, mi[e].scale_f32()) for mi in ms] for e in range(E)]


def codes(M, K, seed, pad=0, shift=0, token_major=False):
    t = torch()
    q, s = O.quant_act(synth.gaussian_activations(801 + seed, f"ex_X{M}x{K}", M, K))
    buf = t.full((M * (K + pad) + shift,), 0x7F, dtype=t.uint8, device=device())
    xq = buf[shift:].view(M, K + pad)[:, :K]
    xq.copy_(t.from_numpy(q))
    xs = t.empty(s.shape, device=device()) if token_major else B.scales_kmajor(M, s.shape[1], device())
    xs.copy_(t.from_numpy(s))
    return q, s, xq, xs


def verify(got, q, s, om, offsets, rows, N, K, bf16, keep=5.0, fp8_mfma=False):
    """Every row of [R, >= N] outputs: its expert's product, zeros for a row without a token, ``keep`` elsewhere."""
    R = got.shape[0]
    seen = np.zeros(R, bool)
    for e in range(len(om)):
        lo, hi = int(np.clip(offsets[e], 0, R)), int(np.clip(offsets[e + 1], 0, R))
        if hi <= lo:
            continue
        seen[lo:hi] = True
        tok = np.arange(lo, hi) if rows is None else rows[lo:hi]
        ok = (tok >= 0) & (tok < q.shape[0])
        assert np.all(got[lo:hi][~ok][:, :N] == 0.0)
        if ok.any():
            acc = O.linear_w8a8(q[tok[ok]], s[tok[ok]], om[e])
            want, tol = expect(acc, O.abs_bound_w8a8(q[tok[ok]], s[tok[ok]], om[e]), K, bf16=bf16, fp8_mfma=fp8_mfma)
            err = np.abs(got[lo:hi][ok][:, :N] - want)
            assert not np.isnan(err).any() and np.all(err <= tol), (e, float(np.max(err / tol)))
    assert np.all(got[~seen] == keep)
    assert np.all(got[:, N:] == keep)


def check(counts, rows, K, gather=True, M=None, y="bf16", f32_scales=False, token_major=False, pad=0, shift=0, extra=0,
          bad_rows=False, seed=0):
    t = torch()
    E, N = len(counts), sum(rows)
    used = int(sum(counts))
    R = used + extra
    M = M if M is not None else (max(1, R // 2) if gather else R)
    w, om = experts(E, rows, K, seed, f32_scales)
    banner(f"experts counts={list(counts)[:12]} rows={rows} K={K} M={M} R={R} gather={gather} {y} pad={pad} shift={shift}: "
           f"{w.describe(R)}")
    q, s, xq, xs = codes(M, K, seed, pad, shift, token_major)
    g = np.random.default_rng(seed)
    offsets = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    idx = None
    if gather:
        idx = g.integers(0, M, R).astype(np.int32)
        if bad_rows:
            idx[::3] = -1
            idx[1::7] = M
            idx[2::11] = 2 ** 31 - 1
    out = t.full((R, N + pad), 5.0, dtype=t.bfloat16 if y == "bf16" else t.float32, device=device())
    B.linear_w8a8_experts(w, xq, xs, t.from_numpy(offsets).to(device()),
                          rows=t.from_numpy(idx).to(device()) if gather else None, out_dtype=out.dtype, out=out[:, :N])
    t.cuda.synchronize()
    verify(to_np(out), q, s, om, offsets, idx, N, K, y == "bf16", fp8_mfma=y == "bf16" and "f8f6f4" in w.describe(R))   # (F32 outputs never use it)


# run lengths around the tiles, experts without rows at both ends and between, one expert, more than 64 experts
COUNTS = [(1,), (0, 1, 0), (16, 17, 0, 15, 1), (0, 0, 63, 64, 65, 0), (5,) * 9, (129, 0, 1, 127, 128), (300, 2, 257), (0, 0, 0)]


@pytest.mark.parametrize("counts", COUNTS, ids=lambda c: "_".join(map(str, c)))
@pytest.mark.parametrize("rows,K,gather", [((256,), 512, True), ((200, 77), 1136, True), ((300,), 1000, False)])
def test_runs(counts, rows, K, gather):
    check(counts, rows, K, gather, extra=3, seed=len(counts))


@pytest.mark.parametrize("terms", [dict(y="f32"), dict(f32_scales=True), dict(token_major=True), dict(pad=16), dict(pad=3, y="f32"),
                                   dict(shift=1), dict(bad_rows=True), dict(extra=40), dict(M=1), dict(gather=False)],
                         ids=lambda d: "-".join(f"{k}_{v}" for k, v in d.items()))
@pytest.mark.parametrize("counts,rows,K", [((3, 0, 20, 1), (128, 128), 768), ((150, 260, 0, 31), (300,), 640),
                                           ((40, 70), (131,), 333)])
def test_terms(counts, rows, K, terms):
    check(counts, rows, K, **terms)


def test_many_experts():
    g = np.random.default_rng(3)
    check(g.integers(0, 4, 150), (64,), 256, seed=5)
    c = np.zeros(200, int)
    c[[0, 63, 64, 127, 128, 199]] = (3, 20, 1, 130, 17, 40)
    check(c, (64,), 256, seed=6)


def test_small_k():
    for K in (1, 16, 17, 127, 129):
        check((3, 0, 30), (40,), K, y="f32", seed=K)


def test_offsets_stay_in_bounds():
    """Offsets that leave [0, R] count as clamped; where they descend, runs may overlap and their rows get either
    expert's product, but nothing outside y is written."""
    t = torch()
    w, om = experts(4, (130,), 256)
    R = 50
    q, s, xq, xs = codes(R, 256, 0)
    for off in ([-5, 10, 10, 30, 99], [60, 70, 80, 90, 100], [0, 20, 10, 10, 50], [2 ** 31 - 1, -2 ** 31, 5, 6, 7]):
        banner(f"experts offsets {off}")
        buf = t.full((R + 20, 130), 5.0, dtype=t.float32, device=device())
        out = buf[10:10 + R]
        B.linear_w8a8_experts(w, xq, xs, t.tensor(off, dtype=t.int32, device=device()), out_dtype=t.float32, out=out)
        t.cuda.synchronize()
        if all(a <= b for a, b in zip(off, off[1:])):
            verify(to_np(out), q, s, om, np.array(off, np.int64), None, 130, 256, False)
        assert bool((buf[:10] == 5.0).all()) and bool((buf[10 + R:] == 5.0).all())


def test_no_rows():
    t = torch()
    w, _ = experts(2, (64,), 256)
    off = t.zeros(3, dtype=t.int32, device=device())
    y = B.linear_w8a8_experts(w, t.empty((0, 256), dtype=t.uint8, device=device()), t.empty((0, 2), device=device()), off)
    assert y.shape == (0, 64)


def _routed(t, M, top, E, H, F, seed):
    """Weights and inputs of a routed gated layer."""
    g = t.Generator(device=device())
    g.manual_seed(seed)
    wgu, omgu = experts(E, (F, F), H, seed)
    wd, omd = experts(E, (H,), F, seed + 1)
    x = t.randn(M, H, generator=g, device=device()).bfloat16()
    ids = t.randint(0, E, (M, top), generator=g, device=device(), dtype=t.int32)
    probs = t.rand(M, top, generator=g, device=device())
    return wgu, omgu, wd, omd, x, ids, probs


@pytest.mark.parametrize("M,top,E,H,F", [(1, 2, 4, 256, 128), (50, 2, 4, 256, 192), (300, 3, 5, 384, 256)])
def test_routed_layer(M, top, E, H, F):
    """quant_norm -> expert_plan -> gate/up by expert -> quant_glu -> down by expert -> quant_norm with the combine,
    each step against its reference on the step's own inputs, eager and replayed from a graph with other choices."""
    t = torch()
    wgu, omgu, wd, omd, x, ids, probs = _routed(t, M, top, E, H, F, 3)
    norm = t.rand(H, device=device()) + 0.5
    R = M * top
    d = device()
    gu = t.full((R, 2 * F), 0.0, device=d)
    dn = t.full((R, H), 0.0, device=d)
    rows = t.zeros(R, dtype=t.int32, device=d)
    keep = {}

    def layer():
        xq, xs, _, n = B.quant_norm(x, norm, out_dtype=t.float32)
        off, _, slots = B.expert_plan(ids, E, rows=rows)
        B.linear_w8a8_experts(wgu, xq, xs, off, rows=rows, out_dtype=t.float32, out=gu)
        hq, hs = B.quant_glu(gu)
        B.linear_w8a8_experts(wd, hq, hs, off, out_dtype=t.float32, out=dn)
        yq, ys, h, n2 = B.quant_norm(dn, norm, slots=slots, probs=probs, residual=x, h=t.empty_like(x), out_dtype=t.float32)
        keep.update(xq=xq, xs=xs, off=off, slots=slots, hq=hq, hs=hs, yq=yq, ys=ys, h=h, n2=n2)

    def examine():
        off, rr, rs = plan_ref(ids.cpu().numpy(), E)
        assert np.array_equal(keep["off"].cpu().numpy(), off) and np.array_equal(keep["slots"].cpu().numpy(), rs)
        q, s = keep["xq"].cpu().numpy(), keep["xs"].cpu().numpy()
        verify(to_np(gu), q, s, omgu, off, rr, 2 * F, H, False)
        hq, hs = O.glu_quant(gu.cpu().numpy(), F)
        assert np.array_equal(keep["hq"].cpu().numpy(), hq) and np.array_equal(keep["hs"].cpu().numpy(), hs)
        verify(to_np(dn), hq, hs, omd, off, None, H, F, False)
        o = np.einsum("mj,mjk->mk", probs.cpu().numpy().astype(np.float64), dn.cpu().numpy().astype(np.float64)[rs])
        mag = np.einsum("mj,mjk->mk", probs.cpu().numpy().astype(np.float64), np.abs(dn.cpu().numpy().astype(np.float64)[rs]))
        h64 = o + to_np(x)
        tol = 2.0 ** -8 * (1 + 2.0 ** -15) * np.abs(h64) + 2.0 ** -50 * (mag + np.abs(to_np(x)))
        assert np.all(np.abs(to_np(keep["h"]) - h64) <= tol)
        yq, ys = O.quant_act(keep["n2"].cpu().numpy())
        assert np.array_equal(keep["yq"].cpu().numpy(), yq) and np.array_equal(keep["ys"].cpu().numpy(), ys)

    banner(f"routed layer M={M} top={top} E={E}")
    layer()
    t.cuda.synchronize()
    examine()
    graph = t.cuda.CUDAGraph()
    with t.cuda.graph(graph):
        layer()
    for rep in range(3):
        g = np.random.default_rng(rep)
        # one replay with everything on one expert
        ids.copy_(t.from_numpy(np.full((M, top), E - 1) if rep == 1 else g.integers(0, E, (M, top))).to(t.int32))
        x.copy_(t.randn(M, H, device=d))
        t.cuda.synchronize()
        graph.replay()
        t.cuda.synchronize()
        examine()


def test_dense_layer():
    """quant_norm -> up with bias and GELU -> quant_act -> down with bias and residual, in the stream's own buffer."""
    t = torch()
    H, F, M = 384, 512, 70
    up, down = synth.random_code_weight(810, "dl_up", F, H), synth.random_code_weight(810, "dl_down", H, F)
    mk = lambda m: B.BlockFP8Weight([(t.from_numpy(m.codes).to(device()),
                                      t.from_numpy(m.scale_bits.view(np.int16)).to(device()).view(t.bfloat16))])
    wu, wd = mk(up), mk(down)
    x = t.randn(M, H, device=device())
    res = t.randn(M, H, device=device())
    norm, bu, bd = t.rand(H, device=device()) + 0.5, t.randn(F, device=device()), t.randn(H, device=device())
    banner("dense layer")
    xq, xs, h, _ = B.quant_norm(x, norm, residual=res)
    u = B.linear_w8a8_epilogue(wu, xq, xs, bias=bu, activation="gelu_tanh", out_dtype=t.float32)
    uq, us = B.quant_act(u)
    before = to_np(h).astype(np.float64)
    y = B.linear_w8a8_epilogue(wd, uq, us, bias=bd, residual=h, out_dtype=t.float32, out=h)
    q, s = xq.cpu().numpy(), xs.cpu().numpy()
    om = [(up.codes, up.scale_f32())]
    want, tol = expect(O.linear_w8a8(q, s, om), O.abs_bound_w8a8(q, s, om), H, to_np(bu).astype(np.float64), "gelu_tanh")
    assert np.all(np.abs(to_np(u) - want) <= tol)
    q, s = O.quant_act(u.cpu().numpy())
    om = [(down.codes, down.scale_f32())]
    want, tol = expect(O.linear_w8a8(q, s, om), O.abs_bound_w8a8(q, s, om), F, to_np(bd).astype(np.float64), None, before)
    assert np.all(np.abs(to_np(y) - want) <= tol)
