"""Calls of the operators around the products that lie off the usual paths: mixed types, experts' sums on rows without
alignment, the most experts, members of a row each, runs that do not start at row 0, outputs of more than 2^31 elements."""
import numpy as np
import pytest

import block_scaled_fp8_linear_amd as B
import oracle as O
import test_gpu_epilogue as epilogue
import test_gpu_experts as experts
import test_gpu_norm as norm
from fused_util import expect
from gpu_util import banner, device, to_np, torch
from test_gpu_route import plan_ref

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,K", [(5, 130), (9, 1001), (4, 5001), (3, 17408), (2, 32768)])
@pytest.mark.parametrize("terms", [dict(), dict(pad=3), dict(shift=1, x="f32", h="f32", w="f32"), dict(post=True, bias=True, gate="token")],
                         ids=lambda d: "-".join(d) or "plain")
def test_experts_sum_on_the_general_kernel(M, K, terms):
    for kind in ("rms", "layer"):
        norm.check(M, K, kind, top=3, seed=K, **terms)


@pytest.mark.parametrize("K", [640, 1001])
@pytest.mark.parametrize("types", ["wpg", "wPg", "Wpg", "wpG", "WPg", "wPG"])
def test_vectors_of_mixed_types(K, types):
    """Norm weights, post weights and gates of different types (capitals: F32) give what their F32 copies give: the
    stream within the roundings of two F64 evaluations, the codes those of the norm the call returns."""
    t = torch()
    banner(f"quant_norm mixed types {types} K={K}")
    g = t.Generator(device=device())
    g.manual_seed(K)
    M = 7
    rnd = lambda *s: t.randn(*s, generator=g, device=device())
    x, res = rnd(M, K), rnd(M, K)
    w, p, gate = (v if c.isupper() else v.bfloat16() for c, v in zip(types, (rnd(K), rnd(K), rnd(M, K))))
    q, s, h, n = B.quant_norm(x, w, residual=res, post_weight=p, gate=gate, out_dtype=t.float32)
    q2, s2, h2, n2 = B.quant_norm(x, w.float(), residual=res, post_weight=p.float(), gate=gate.float(), out_dtype=t.float32)
    # F32 outputs of one formula, each a rounding of an F64 value with noise some 2^-40 of the terms
    f = lambda v: v.double()
    assert bool(((f(h) - f(h2)).abs() <= 2.0 ** -23 * f(h2).abs() + 2.0 ** -39).all())
    assert bool(((f(n) - f(n2)).abs() <= 2.0 ** -21 * (f(n2).abs() + f(h2).abs())).all())
    yq, ys = O.quant_act(n.cpu().numpy())
    assert np.array_equal(q.cpu().numpy(), yq) and np.array_equal(s.cpu().numpy(), ys)


@pytest.mark.parametrize("M", [1, 16, 64, 65, 130])
def test_eight_members_of_few_rows(M):
    epilogue.check(M, (1, 2, 3, 1, 129, 1, 31, 33), 272, act="gelu", residual="bf16")
    epilogue.check(M, (1,), 16, act="silu", residual="f32", y="f32")


@pytest.mark.parametrize("y", ["bf16", "f32"])
def test_the_most_experts(y):
    t = torch()
    E, N, K, R, M = 65535, 8, 48, 70000, 999
    g = np.random.default_rng(12)
    w = g.integers(0, 0x78, (E, N, K)).astype(np.uint8) | (g.integers(0, 2, (E, N, K)) << 7).astype(np.uint8)
    s = g.uniform(0.5, 2, (E, 1, 1)).astype(np.float32)
    we = B.ExpertsFP8Weight([(t.from_numpy(w).to(device()), t.from_numpy(s).to(device()))])
    xq, xs = B.quant_act(t.from_numpy(g.standard_normal((M, K)).astype(np.float32)).to(device()))
    ids = g.integers(-1, E, (R, 1)).astype(np.int32)
    ids[:3000] = E - 1
    banner(f"{E} experts {y}: {we.describe(R)}")
    off, rows, slots = B.expert_plan(t.from_numpy(ids).to(device()), E, rows=t.zeros(R, dtype=t.int32, device=device()))
    ro, rr, rs = plan_ref(ids, E)
    assert np.array_equal(off.cpu().numpy(), ro) and np.array_equal(slots.cpu().numpy(), rs)
    out = t.full((R, N), 5.0, dtype=t.bfloat16 if y == "bf16" else t.float32, device=device())
    B.linear_w8a8_experts(we, xq, xs, off, rows=rows % M, out_dtype=out.dtype, out=out)
    got = to_np(out)
    used = rr.size
    x64 = O.dequantize_act(xq.cpu().numpy(), xs.cpu().numpy())[rr % M]
    w64 = (O.e4m3_decode(w).astype(np.float64) * s)[np.sort(ids[ids >= 0], kind="stable")]
    acc = np.matmul(w64, x64[:, :, None])[:, :, 0]
    mag = np.matmul(np.abs(w64), np.abs(x64)[:, :, None])[:, :, 0]
    want, tol = expect(acc, mag, K, bf16=y == "bf16", fp8_mfma=y == "bf16")
    assert np.all(np.abs(got[:used] - want) <= tol) and np.all(got[used:] == 5.0)


@pytest.mark.parametrize("y", ["bf16", "f32"])
@pytest.mark.parametrize("off", [[7, 9, 9, 40], [100, 500, 600, 1990]])
def test_runs_that_start_late_and_end_early(off, y):
    t = torch()
    R, K, rows = 2000, 400, (1000, 200)
    w, om = experts.experts(3, rows, K)
    q, s, xq, xs = experts.codes(R, K, 0)
    dt = t.bfloat16 if y == "bf16" else t.float32
    banner(f"offsets {off} {y}: {w.describe(R)}")
    out = t.full((R, sum(rows)), 5.0, dtype=dt, device=device())
    B.linear_w8a8_experts(w, xq, xs, t.tensor(off, dtype=t.int32, device=device()), out_dtype=dt, out=out)
    experts.verify(to_np(out), q, s, om, np.array(off), None, sum(rows), K, y == "bf16", fp8_mfma=y == "bf16")


@pytest.mark.parametrize("y", ["bf16", "f32"])
def test_outputs_beyond_32_bits(y):
    """Tokens that repeat: every repetition gives the first ones' bits, wherever its rows lie."""
    t = torch()
    M, N, K, n = 131072 + 77, 16500, 128, 997
    dt = t.bfloat16 if y == "bf16" else t.float32
    g = t.Generator(device=device())
    g.manual_seed(9)
    codes = t.randint(0, 0x78, (N, K), dtype=t.uint8, device=device(), generator=g)
    scales = t.rand((-(-N // 128), 1), device=device(), generator=g) + 0.5
    xq0, xs0 = B.quant_act(t.randn((n, K), device=device(), generator=g), xs=t.empty((n, 1), device=device()))
    idx = t.arange(M, device=device()) % n
    xq, xs = xq0[idx], xs0[idx]
    res = t.randn((n, N), device=device(), generator=g).to(dt)
    assert M * N > 2 ** 31
    w = B.BlockFP8Weight([(codes, scales)])
    banner(f"{M} x {N} outputs {y}: {w.describe(B.ARM_W8A8_EPILOGUE, M)}")

    def repeats(out):
        for i in range(0, M, n):
            here = out[i:i + n]
            if not t.equal(here, out[:here.shape[0]]):
                return False
        return True

    out = t.empty((M, N), dtype=dt, device=device())
    for i in range(0, M, n):
        out[i:i + n] = res[:min(n, M - i)]
    B.linear_w8a8_epilogue(w, xq, xs, activation="relu", residual=out, out_dtype=dt, out=out)
    q, s = xq0.cpu().numpy(), xs0.cpu().numpy()
    om = [(codes.cpu().numpy(), scales.cpu().numpy())]
    cols = [0, 1, 127, 128, 8191, 16384, 16499]
    acc, mag = O.linear_w8a8_rows(q, s, om, cols), O.abs_bound_w8a8_rows(q, s, om, cols)
    want, tol = expect(acc, mag, K, act="relu", residual=to_np(res)[:, cols].astype(np.float64), bf16=y == "bf16",
                       fp8_mfma=y == "bf16")
    assert np.all(np.abs(to_np(out[:n][:, cols]) - want) <= tol) and repeats(out)
    we = B.ExpertsFP8Weight([(codes[None].repeat(3, 1, 1), scales[None].repeat(3, 1, 1))])
    out.fill_(5.0)
    off = t.tensor([0, 40000, 40000, M], dtype=t.int32, device=device())
    banner(f"{M} x {N} outputs of experts {y}: {we.describe(M)}")
    B.linear_w8a8_experts(we, xq0, xs0, off, rows=idx.int(), out_dtype=dt, out=out)
    want, tol = expect(acc, mag, K, bf16=y == "bf16", fp8_mfma=y == "bf16")
    assert np.all(np.abs(to_np(out[:n][:, cols]) - want) <= tol) and repeats(out)


@pytest.mark.parametrize("K", [640, 5120, 1001, 17408])
def test_dropped_choices_hold_anything(K):
    """Router weights of choices without a row, and rows that no choice names, may be NaN or infinite."""
    t = torch()
    banner(f"quant_norm dropped choices K={K}")
    M, top, R = 6, 5, 40
    g = t.Generator(device=device())
    g.manual_seed(K)
    x = t.randn((R, K), generator=g, device=device()).bfloat16()
    slots = t.randperm(R, generator=g, device=device())[:M * top].view(M, top).int()
    probs = t.rand((M, top), generator=g, device=device())
    slots[:, 1], slots[2], slots[0, 4] = -1, R, -2 ** 31
    dropped = (slots < 0) | (slots >= R)
    w, res = t.rand(K, device=device()) + 0.5, t.randn((M, K), generator=g, device=device())
    call = lambda p, v: B.quant_norm(v, w, slots=slots, probs=p, residual=res, out_dtype=t.float32)
    want = call(probs.masked_fill(dropped, 0.0), x)
    named = t.zeros(R, dtype=t.bool, device=device())
    named[slots[~dropped].long()] = True
    for bad in (float("nan"), float("inf")):
        got = call(probs.masked_fill(dropped, bad), x.masked_fill(~named[:, None], bad))
        assert all(t.equal(a, b) for a, b in zip(got, want))
    assert t.equal(want[2][2], res[2])


@pytest.mark.parametrize("K", [65536, 65664, 70001, 131072, 131088])
def test_the_longest_sums(K):
    """K whose blocks outnumber a wave's scales held at a time, and beyond what the tile kernel takes."""
    for M in (2, 70):
        epilogue.check(M, (40,), K, act="relu", residual="f32", y="f32", seed=1)
        epilogue.check(M, (40,), K, act="relu", seed=1)
    experts.check((1, 0, 40), (33,), K, y="f32", seed=1)
