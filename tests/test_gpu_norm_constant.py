"""The layer norm of rows that are one value: v - mean is exactly zero, whatever the value, the width and eps.

The sum of K equal F32 values is exact in F64, and so is its quotient by K, the value itself; what is left of a mean off
by its last place would be multiplied by 1 / sqrt(eps) and, the quantizer's scale having a floor, fill the codes.
"""
import numpy as np
import pytest

import block_scaled_fp8_linear_amd as B
from gpu_util import banner, device, torch

pytestmark = pytest.mark.gpu

VALUES = [1000.25, 12345.5, -0.1, 3.0, 1e-30, 7.7e8, 2.0 ** 100 / 3]


# a shift by one element, or a width that is no multiple of 8, takes the general kernel
@pytest.mark.parametrize("K", [8, 200, 1000, 1408, 5000, 5120, 7168, 16384, 20000, 5, 1001, 5121])
@pytest.mark.parametrize("shift", [0, 1])
@pytest.mark.parametrize("eps", [1e-5, 1e-12])
def test_next_norm(K, shift, eps):
    t = torch()
    banner(f"layer norm of constant rows K={K} shift={shift} eps={eps}")
    x = t.tensor(VALUES, device=device())[:, None].expand(len(VALUES), K).contiguous()
    flat = t.zeros(x.numel() + shift, device=device())
    xd = flat[shift:].view(x.shape)
    xd.copy_(x)
    w = t.linspace(0.5, 2.0, K, device=device())
    xq, xs, _, n = B.quant_norm(xd, w, kind="layer", eps=eps, out_dtype=t.float32)
    assert bool((n == 0).all()), n.abs().max()
    assert bool((xq == 0).all()) and bool((xs == np.float32(1e-10) / np.float32(448.0)).all())
    bias = t.linspace(-3.0, 3.0, K, device=device())
    assert t.equal(B.quant_norm(xd, w, bias=bias, kind="layer", eps=eps, out_dtype=t.float32)[3], bias.expand_as(x))


@pytest.mark.parametrize("K", [200, 1000, 5120, 16384, 1001])
@pytest.mark.parametrize("shift", [0, 1])
def test_norm_of_the_output(K, shift):
    """The norm after a block: its bias alone is left, and the stream is that times the gate plus the residual."""
    t = torch()
    banner(f"layer norm of a constant output K={K} shift={shift}")
    x = t.tensor(VALUES, device=device())[:, None].expand(len(VALUES), K).contiguous()
    flat = t.zeros(x.numel() + shift, device=device())
    xd = flat[shift:].view(x.shape)
    xd.copy_(x)
    w = t.ones(K, device=device())
    pb = t.linspace(-3.0, 3.0, K, device=device())
    res = t.randn(x.shape, device=device())
    h = B.quant_norm(xd, w, kind="layer", eps=1e-5, post_weight=w, post_bias=pb, residual=res, residual_scale=0.0)[2]
    assert t.equal(h, pb.expand_as(x))
