"""Refusals of the operators around the products, before any launch (no GPU needed)."""
import ctypes

import pytest

import block_scaled_fp8_linear_amd as B

FAKE = 1 << 40
name = B.status_name


def _norm(**kw):
    a = B.NormArgs(4, 256, 0, 1e-6, 1.0)
    a.x, a.x_dtype, a.ldx = FAKE, B.DT_BF16, 256
    a.weight, a.weight_dtype = FAKE, B.DT_F32
    a.h_dtype = B.DT_BF16
    a.xq, a.ldq, a.xs, a.xs_sm, a.xs_sk = FAKE, 256, FAKE, 2, 1
    for k, v in kw.items():
        setattr(a, k, v)
    return name(B.lib().bsf8_quant_norm(ctypes.byref(a), None))


def test_quant_norm_refusals():
    assert name(B.lib().bsf8_quant_norm(None, None)) == "INVALID_ARG"
    assert _norm(M=0) == "OK" and _norm(K=0) == "OK"
    for bad in (dict(M=-1), dict(K=-1), dict(kind=2), dict(eps=0.0), dict(eps=float("nan")), dict(eps=float("inf")),
                dict(residual_scale=float("nan")), dict(x_dtype=B.DT_F16), dict(h_dtype=B.DT_F16),
                dict(weight_dtype=B.DT_U8), dict(x=None), dict(weight=None), dict(ldx=255), dict(ldq=255),
                dict(xq=None), dict(xs=None), dict(xq=None, xs=None), dict(xs_sm=1, xs_sk=3),
                dict(residual=FAKE, ldr=256), dict(residual=FAKE, ldr=255, h=FAKE, ldh=256),
                dict(residual=FAKE, ldr=256, h=FAKE, ldh=255), dict(n=FAKE, n_dtype=B.DT_F16, ldn=256),
                dict(n=FAKE, n_dtype=B.DT_F32, ldn=200), dict(gate=FAKE, gate_dtype=B.DT_F32, ldg=100),
                dict(gate=FAKE, gate_dtype=B.DT_F16), dict(post_bias=FAKE), dict(post_weight=FAKE, post_dtype=B.DT_U8),
                dict(slots=FAKE), dict(probs=FAKE), dict(slots=FAKE, probs=FAKE, top=0, x_rows=4),
                dict(slots=FAKE, probs=FAKE, top=2, x_rows=-1)):
        assert _norm(**bad) == "INVALID_ARG", bad
    for bad in (dict(x=FAKE + 1), dict(weight=FAKE + 2), dict(xs=FAKE + 2), dict(residual=FAKE + 1, ldr=256, h=FAKE, ldh=256),
                dict(slots=FAKE + 2, probs=FAKE, top=2, x_rows=4), dict(bias=FAKE + 1)):
        assert _norm(**bad) == "ALIGNMENT", bad
    assert _norm(K=32769, ldx=32769, ldq=32769, xs_sm=257) == "UNSUPPORTED"
    assert _norm(slots=FAKE, probs=FAKE, top=2, x_rows=1 << 31) == "UNSUPPORTED"


def test_expert_plan_refusals():
    L = B.lib()
    call = lambda ids=FAKE, b=4, M=4, top=2, E=8, off=FAKE, rows=FAKE, slots=FAKE: name(
        L.bsf8_expert_plan(ids, b, M, top, E, off, rows, slots, None))
    for bad in (dict(ids=None), dict(b=2), dict(M=-1), dict(top=0), dict(E=0), dict(off=None), dict(rows=None),
                dict(slots=None)):
        assert call(**bad) == "INVALID_ARG", bad
    for bad in (dict(ids=FAKE + 2), dict(ids=FAKE + 4, b=8), dict(off=FAKE + 1), dict(rows=FAKE + 2), dict(slots=FAKE + 2)):
        assert call(**bad) == "ALIGNMENT", bad
    assert call(M=1 << 30, top=2) == "UNSUPPORTED" and call(E=65536) == "UNSUPPORTED"


def test_binding_refuses_host_tensors():
    import torch
    x, w = torch.zeros((4, 256)), torch.ones(256)
    with pytest.raises(ValueError, match="GPU tensor"):
        B.quant_norm(x, w)
    with pytest.raises(ValueError, match="GPU tensor"):
        B.expert_plan(torch.zeros((4, 2), dtype=torch.int32), 4)
