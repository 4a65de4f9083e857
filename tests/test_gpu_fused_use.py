"""quant_norm, expert_plan, linear_w8a8_epilogue and linear_w8a8_experts as programs use them: several calls at once,
graphs that share a stream, and the largest sizes."""
import numpy as np
import pytest

import block_scaled_fp8_linear_amd as B
import oracle as O
import synth
from fused_util import expect
from gpu_util import banner, device, member_to_device, oracle_members, to_np, torch
from test_gpu_route import plan_ref

pytestmark = pytest.mark.gpu


def test_two_graphs_of_one_stream_at_once():
    """Both split K and were captured on one stream; replayed together on two streams, each with its own workspace."""
    t = torch()
    m = synth.random_code_weight(820, "two_graphs", 640, 4096)
    w = B.BlockFP8Weight([member_to_device(m)])
    banner("two graphs")
    graphs, outs, wants = [], [], []
    for seed, M in ((0, 200), (1, 300)):
        assert w.workspace_size(B.ARM_W8A8_EPILOGUE, M) > 0
        xq, xs = B.quant_act(t.randn(M, 4096, device=device()))
        y = t.empty((M, 640), device=device())
        call = lambda: B.linear_w8a8_epilogue(w, xq, xs, activation="gelu", out_dtype=t.float32, out=y)
        call()
        wants.append(y.clone())
        graph = t.cuda.CUDAGraph()
        with t.cuda.graph(graph):
            call()
        graphs.append((graph, xq, xs))
        outs.append(y)
    streams = [t.cuda.Stream(), t.cuda.Stream()]
    for _ in range(4):
        for y in outs:
            y.zero_()
        t.cuda.synchronize()
        for _ in range(5):
            for (graph, _, _), st in zip(graphs, streams):
                with t.cuda.stream(st):
                    graph.replay()
        t.cuda.synchronize()
        assert all(t.equal(y, want) for y, want in zip(outs, wants))


def test_calls_on_two_streams_at_once():
    t = torch()
    E, H, F, M, top = 6, 512, 256, 90, 2
    ws = t.randint(0, 0x7E, (E, F, H), dtype=t.uint8, device=device())
    w = B.ExpertsFP8Weight([(ws, t.full((E, F // 128, H // 128), 0.01, device=device()))])
    norm = t.rand(H, device=device()) + 0.5
    sets = [(t.randn(M, H, device=device()), t.randint(0, E, (M, top), device=device(), dtype=t.int32)) for _ in range(2)]

    def go(x, ids):
        xq, xs, h, _ = B.quant_norm(x, norm, residual=x, h=t.empty_like(x))
        off, rows, slots = B.expert_plan(ids, E)
        y = B.linear_w8a8_experts(w, xq, xs, off, rows=rows)
        z = B.quant_norm(y, norm[:F], slots=slots, probs=t.ones((M, top), device=device()), out_dtype=t.float32)[3]
        return xq, xs, h, off, rows, slots, y, z

    banner("two streams")
    wants = [go(*s) for s in sets]
    t.cuda.synchronize()
    streams = [t.cuda.Stream(), t.cuda.Stream()]
    for _ in range(5):
        got = []
        for s, st in zip(sets, streams):
            with t.cuda.stream(st):
                got.append(go(*s))
        t.cuda.synchronize()
        for a, b in zip(got, wants):
            assert all(t.equal(p, q) for p, q in zip(a, b))


@pytest.mark.parametrize("M,K", [((1 << 22) + 5, 8), ((1 << 24) + 70, 5)])
def test_norm_of_more_rows_than_one_launch(M, K):
    """Rows that repeat: every repetition of the first ones gives their bits."""
    t = torch()
    banner(f"quant_norm M={M} K={K}")
    n = 977
    x0 = t.randn(n, K, device=device()).bfloat16()
    weight = t.rand(K, device=device()) + 0.5
    idx = t.arange(M, device=device()) % n
    want = B.quant_norm(x0, weight, residual=x0, h=t.empty_like(x0), out_dtype=t.bfloat16)
    x = x0[idx]
    got = B.quant_norm(x, weight, residual=x, h=t.empty_like(x), out_dtype=t.bfloat16)
    t.cuda.synchronize()
    for a, b in zip(got, want):
        assert t.equal(a, b[idx])


def test_plan_of_the_most_choices():
    t = torch()
    n = 2 ** 31 - 1
    banner(f"expert_plan {n} choices")
    ids = t.zeros((n, 1), dtype=t.int32, device=device())
    ids[5] = 1
    ids[n - 1] = 1
    ids[n - 2] = -1
    off, rows, slots = B.expert_plan(ids, 2)
    t.cuda.synchronize()
    assert off.tolist() == [0, n - 3, n - 1]
    assert rows[n - 3:n - 1].tolist() == [5, n - 1]
    assert [int(slots[i, 0]) for i in (0, 4, 5, 6, n - 3, n - 2, n - 1)] == [0, 4, n - 3, 5, n - 4, -1, n - 2]
    assert int(rows[4]) == 4 and int(rows[5]) == 6 and int(rows[n - 4]) == n - 3
    part = t.arange(6, n - 2, device=device(), dtype=t.int32)
    assert t.equal(rows[5:n - 3], part)


def _far_tokens(M, K, pitch):
    """Quantized activations whose rows lie ``pitch`` bytes apart."""
    t = torch()
    q, s = O.quant_act(synth.gaussian_activations(821, "far", M, K))
    buf = t.full((M * pitch,), 0x7F, dtype=t.uint8, device=device())
    xq = buf.view(M, pitch)[:, :K]
    xq.copy_(t.from_numpy(q))
    return q, s, xq, t.from_numpy(s).to(device())


def test_tokens_beyond_32_bits():
    t = torch()
    M, K, N = 300, 512, 200
    q, s, xq, xs = _far_tokens(M, K, 1 << 23)
    m = synth.random_code_weight(821, "far_w", N, K)
    om = oracle_members([m])
    banner("tokens 2.5 GB apart")
    want, tol = expect(O.linear_w8a8(q, s, om), O.abs_bound_w8a8(q, s, om), K, act="silu")
    w = B.BlockFP8Weight([member_to_device(m)])
    assert np.all(np.abs(to_np(B.linear_w8a8_epilogue(w, xq, xs, activation="silu", out_dtype=t.float32)) - want) <= tol)
    codes, scales = member_to_device(m)
    we = B.ExpertsFP8Weight([(codes[None].contiguous(), scales[None].contiguous())])
    want, tol = expect(O.linear_w8a8(q, s, om), O.abs_bound_w8a8(q, s, om), K)
    y = B.linear_w8a8_experts(we, xq, xs, t.tensor([0, M], dtype=t.int32, device=device()), out_dtype=t.float32)
    assert np.all(np.abs(to_np(y) - want) <= tol)


@pytest.mark.parametrize("R", [3, 700])
@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_experts_beyond_32_bits(R, out):
    """Five experts of 512 MiB each; the last one's product, on the last of its weight rows."""
    t = torch()
    E, N, K = 5, 16384, 32768
    g = t.Generator(device=device())
    g.manual_seed(5)
    w = t.randint(0, 0x7E, (E, N, K), dtype=t.uint8, device=device(), generator=g)
    w |= t.randint(0, 2, (E, N, 1), dtype=t.uint8, device=device(), generator=g) << 7
    s = t.rand((E, N // 128, K // 128), device=device(), generator=g) + 0.5
    we = B.ExpertsFP8Weight([(w, s)])
    xq, xs = B.quant_act(t.randn((R, K), device=device(), generator=g))
    off = t.tensor([0, 0, 0, 0, 0, R], dtype=t.int32, device=device())
    banner(f"experts of 2.5 GiB R={R} {out}: {we.describe(R)}")
    dt = t.bfloat16 if out == "bf16" else t.float32
    y = to_np(B.linear_w8a8_experts(we, xq, xs, off, out_dtype=dt))[:, -40:]
    q, sa = xq.cpu().numpy(), xs.cpu().numpy()
    om = [(w[4, -128:].cpu().numpy(), s[4, -1:].cpu().numpy())]
    acc, mag = O.linear_w8a8(q, sa, om)[:, -40:], O.abs_bound_w8a8(q, sa, om)[:, -40:]
    want, tol = expect(acc, mag, K, bf16=out == "bf16", fp8_mfma=out == "bf16" and "f8f6f4" in we.describe(R))
    assert np.all(np.abs(y - want) <= tol)


def test_offsets_of_many_experts_that_descend():
    """Runs that overlap a hundredfold: nothing outside y is written, and the call ends."""
    t = torch()
    E, R, K, N = 200, 500, 256, 130
    w = B.ExpertsFP8Weight([(t.zeros((E, N, K), dtype=t.uint8, device=device()), t.ones((E, 2, 2), device=device()))])
    xq, xs = B.quant_act(t.randn(R, K, device=device()))
    off = t.tensor([0, 2 ** 31 - 1] * 100 + [5], dtype=t.int32, device=device())
    for dt in (t.bfloat16, t.float32):
        banner(f"descending offsets {dt}")
        buf = t.full((R + 20, N), 5.0, dtype=dt, device=device())
        B.linear_w8a8_experts(w, xq, xs, off, out_dtype=dt, out=buf[10:10 + R])
        t.cuda.synchronize()
        assert bool((buf[:10] == 5.0).all()) and bool((buf[10 + R:] == 5.0).all())


@pytest.mark.parametrize("M", [1, 20, 64, 130, 300])
@pytest.mark.parametrize("act", [None, "relu", "silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_nan_codes_reach_their_outputs_only(M, act, out):
    """A NaN code of a weight row makes that column NaN, one of a token that row, whatever the activation."""
    t = torch()
    N, K = 260, 2048
    m = synth.random_code_weight(822, "nan_w", N, K)
    codes, scales = member_to_device(m)
    codes = codes.clone()
    codes[137, 300] = 0x7F
    codes[259, K - 1] = 0xFF
    w = B.BlockFP8Weight([(codes, scales)])
    xq, xs = B.quant_act(t.randn(M, K, device=device()))
    banner(f"NaN codes M={M} {act} {out}")
    dt = t.bfloat16 if out == "bf16" else t.float32
    args = dict(bias=t.randn(N, device=device()), activation=act, residual=t.randn(M, N, device=device()), out_dtype=dt)
    want = t.zeros((M, N), dtype=t.bool, device=device())
    want[:, [137, 259]] = True
    assert t.equal(B.linear_w8a8_epilogue(w, xq, xs, **args).isnan(), want)
    xq[M // 2, 5] = 0xFF
    want[M // 2] = True
    assert t.equal(B.linear_w8a8_epilogue(w, xq, xs, **args).isnan(), want)


@pytest.mark.parametrize("counts", [(1, 0, 2), (3, 20, 40), (200, 0, 300), (1500, 1500, 1500)])
@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_nan_codes_by_expert(counts, out):
    """NaN codes of one expert's weight row and of token 0, which every fifth row gathers; rows without a token are
    zero all the same."""
    t = torch()
    E, N, K = len(counts), 260, 1024
    g = t.Generator(device=device())
    g.manual_seed(6)
    w = t.randint(0, 0x70, (E, N, K), dtype=t.uint8, device=device(), generator=g)
    w[2, 100, 1000] = 0x7F
    we = B.ExpertsFP8Weight([(w, t.full((E, 3, 8), 0.01, device=device()))])
    R, M = sum(counts), 50
    xq, xs = B.quant_act(t.randn((M, K), device=device(), generator=g))
    xq[0] = 0xFF
    rows = t.randint(1, M, (R,), device=device(), generator=g, dtype=t.int32)
    rows[::5] = 0
    rows[1::7] = -1
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    banner(f"NaN codes by expert {counts} {out}: {we.describe(R)}")
    dt = t.bfloat16 if out == "bf16" else t.float32
    y = B.linear_w8a8_experts(we, xq, xs, t.from_numpy(off).to(device()), rows=rows, out_dtype=dt)
    want = (rows == 0)[:, None].repeat(1, N)
    want[off[2]:, 100] = True
    want &= (rows >= 0)[:, None]
    assert t.equal(y.isnan(), want)
    assert bool((y[rows < 0] == 0).all())


@pytest.mark.parametrize("K", [40, 129, 1024, 2047, 5120, 12000, 16400, 20001])
@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_norm_in_place(K, kind):
    """The new stream written over the old one, or over the block's output: the bits of the call that does not."""
    t = torch()
    M = 37
    x = t.randn(M, K, device=device()).bfloat16()
    r = t.randn(M, K + 8, device=device()).bfloat16()[:, :K]
    weight, post = t.rand(K, device=device()) + 0.5, t.rand(K, device=device()) + 0.5
    banner(f"quant_norm in place K={K} {kind}")
    call = lambda **kw: B.quant_norm(kw.pop("x", x), weight, kind=kind, post_weight=post, **kw)
    q, s, h, _ = call(residual=r)
    old = r.clone()
    pitched = t.zeros((M, K + 8), dtype=t.bfloat16, device=device())[:, :K]
    pitched.copy_(old)
    got = call(residual=pitched, h=pitched)
    assert got[2].data_ptr() == pitched.data_ptr()
    assert t.equal(got[0], q) and t.equal(got[1], s) and t.equal(pitched, h)
    over = x.clone()
    got = call(x=over, residual=r, h=over)
    assert t.equal(got[0], q) and t.equal(got[1], s) and t.equal(over, h) and t.equal(r, old)


@pytest.mark.parametrize("K", [5, 100, 1024, 5120, 20000])
def test_norm_of_constant_rows(K):
    """Rows of zeros and of one value: a norm of exactly zero (layer norm, zeros) gives codes zero and the floor's scale."""
    t = torch()
    banner(f"quant_norm constant rows K={K}")
    for value in (0.0, 3.0, -2.0 ** -100):
        x = t.full((3, K), value, device=device())
        for kind in ("rms", "layer"):
            q, s, _, n = B.quant_norm(x, t.ones(K, device=device()), kind=kind, out_dtype=t.float32)
            want = 0.0 if kind == "layer" else value / (value * value + 1e-6) ** 0.5
            # the layer norm's mean of K equal values is off by at most K roundings, times 1 / sqrt(eps)
            tol = 2.0 ** -24 * abs(want) + (K * 2.0 ** -53 * abs(value) * 1000 if kind == "layer" else 0.0) + 2.0 ** -149
            assert bool(((n.double() - want).abs() <= tol).all())
            yq, ys = O.quant_act(n.cpu().numpy())
            assert np.array_equal(q.cpu().numpy(), yq) and np.array_equal(s.cpu().numpy(), ys)


@pytest.mark.parametrize("top", [1, 2, 3, 5, 6, 7, 9, 10, 12, 17, 33, 100, 1000, 65537, 1 << 20, (1 << 20) + 1])
def test_plan_divides_by_any_top(top):
    t = torch()
    M = max(2, 3_000_000 // top)
    banner(f"expert_plan M={M} top={top}")
    g = np.random.default_rng(top)
    ids = g.integers(-1, 5, (M, top)).astype(np.int32)
    off, rows, slots = B.expert_plan(t.from_numpy(ids).to(device()), 5)
    ro, rr, rs = plan_ref(ids, 5)
    assert np.array_equal(off.cpu().numpy(), ro) and np.array_equal(slots.cpu().numpy(), rs)
    assert np.array_equal(rows.cpu().numpy()[:ro[-1]], rr[:ro[-1]])
