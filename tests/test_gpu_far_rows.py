"""Activation rows tens of megabytes apart: few tokens, whose codes span less than 2 GiB, in a tile of 128 or 256 rows
whose last ones lie past 4 GiB."""
import numpy as np
import pytest

import block_scaled_fp8_linear_amd as B
import oracle as O
import synth
from fused_util import expect
from gpu_util import banner, device, member_to_device, oracle_members, sample_rows, to_np, torch

pytestmark = pytest.mark.gpu


def far(M, K, pitch):
    """Codes [M, K] whose rows lie ``pitch`` bytes apart; the buffer ends with the last one."""
    t = torch()
    q, s = O.quant_act(synth.gaussian_activations(830, "far", M, K))
    buf = t.full(((M - 1) * pitch + K,), 0x7F, dtype=t.uint8, device=device())
    xq = buf.as_strided((M, K), (pitch, 1))
    xq.copy_(t.from_numpy(q))
    return q, s, xq, t.from_numpy(s).to(device())


@pytest.mark.parametrize("M,pitch,N", [(66, 32_000_000, 33000), (100, 21_000_000, 33000), (70, 30_000_000, 300),
                                       (127, 16_800_000, 33000)])
@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_epilogue(M, pitch, N, out):
    t = torch()
    K = 256
    q, s, xq, xs = far(M, K, pitch)
    m = synth.random_code_weight(830, f"far_w{N}", N, K)
    om = oracle_members([m])
    w = B.BlockFP8Weight([member_to_device(m)])
    banner(f"epilogue M={M} pitch={pitch} N={N} {out}")
    y = to_np(B.linear_w8a8_epilogue(w, xq, xs, activation="silu", out_dtype=t.float32 if out == "f32" else t.bfloat16))
    cols = sample_rows(N, [N], 64)
    want, tol = expect(O.linear_w8a8_rows(q, s, om, cols), O.abs_bound_w8a8_rows(q, s, om, cols), K, act="silu",
                       bf16=out == "bf16", fp8_mfma=out == "bf16")
    assert np.all(np.abs(y[:, cols] - want) <= tol)


@pytest.mark.parametrize("M,pitch,N", [(50, 40_000_000, 300), (100, 21_000_000, 33000)])
def test_plain_product(M, pitch, N):
    t = torch()
    K = 256
    q, s, xq, xs = far(M, K, pitch)
    m = synth.random_code_weight(830, f"far_w{N}", N, K)
    om = oracle_members([m])
    w = B.BlockFP8Weight([member_to_device(m)])
    banner(f"linear_w8a8 M={M} pitch={pitch} N={N}")
    y = to_np(B.linear_w8a8(w, xq, xs, out_dtype=t.float32))
    cols = sample_rows(N, [N], 64)
    ok, worst = O.within_bound(y[:, cols], O.linear_w8a8_rows(q, s, om, cols), O.abs_bound_w8a8_rows(q, s, om, cols))
    assert ok, worst


# the farthest rows the dense product takes, the last of a tile's 128 ending at 4 GiB; one row at any pitch
@pytest.mark.parametrize("M,ldx", [(30, 16_909_312), (1, 1_000_000_000)])
def test_dense_within_the_limit(M, ldx):
    t = torch()
    K, N = 256, 300
    buf = t.full(((M - 1) * ldx + K,), float("nan"), dtype=t.bfloat16, device=device())
    x = buf.as_strided((M, K), (ldx, 1))
    x.copy_(t.randn(M, K, device=device()))
    wd = t.randn(N, K, device=device()).bfloat16()
    banner(f"linear_dense ldx={ldx}")
    y = B.linear_dense(wd, x).double().cpu()
    a, b = x.double().cpu(), wd.double().cpu()
    # K exact products summed in F32, in any order
    assert bool(((y - a @ b.T).abs() <= 2.0 ** -23 * K * (a.abs() @ b.abs().T)).all())
