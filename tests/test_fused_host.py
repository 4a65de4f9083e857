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


def _weight(rows=(128,), K=256):
    members = [dict(weight=dict(dtype="F8_E4M3", shape=(r, K), addr=FAKE),
                    scale_inv=dict(dtype="BF16", shape=(-(-r // 128), -(-K // 128)), addr=FAKE)) for r in rows]
    arr, keep = B._members_array(members)
    h = ctypes.c_void_p()
    assert B.lib().bsf8_weight_create(ctypes.byref(B._decl()), arr, len(rows), ctypes.byref(h)) == 0
    return h


def test_epilogue_refusals():
    L, h = B.lib(), _weight()

    def call(w=h, xq=FAKE, ldq=256, xs=FAKE, sm=2, sk=1, M=4, y=FAKE, dt=B.DT_BF16, ldy=128, e=True, **kw):
        ep = B.Epilogue()
        for k, v in kw.items():
            setattr(ep, k, v)
        return name(L.bsf8_linear_w8a8_epilogue(w, xq, ldq, xs, sm, sk, M, ctypes.byref(ep) if e else None, y, dt, ldy, None, 0, None))

    try:
        assert call(M=0) == "OK"
        for bad in (dict(w=None), dict(e=False), dict(M=-1), dict(dt=B.DT_F16), dict(xq=None), dict(xs=None), dict(y=None),
                    dict(ldq=255), dict(ldy=127), dict(sm=1, sk=3), dict(activation=5), dict(activation=-1),
                    dict(bias=FAKE, bias_dtype=B.DT_F16), dict(residual=FAKE, residual_dtype=B.DT_U8, ldr=128),
                    dict(residual=FAKE, residual_dtype=B.DT_F32, ldr=127)):
            assert call(**bad) == "INVALID_ARG", bad
        for bad in (dict(xs=FAKE + 2), dict(y=FAKE + 1), dict(bias=FAKE + 2, bias_dtype=B.DT_F32),
                    dict(residual=FAKE + 1, residual_dtype=B.DT_BF16, ldr=128)):
            assert call(**bad) == "ALIGNMENT", bad
        assert call(M=1 << 31) == "UNSUPPORTED"
        b = ctypes.c_size_t()
        assert L.bsf8_workspace_size(h, B.ARM_W8A8_EPILOGUE, 8, ctypes.byref(b)) == 0
        assert "arm=w8a8-epilogue" in L.bsf8_describe(h, B.ARM_W8A8_EPILOGUE, 8).decode()
    finally:
        L.bsf8_weight_destroy(h)


def _experts(members, block=(128, 128), n=None):
    arr, keep = B._members_array(members)
    h = ctypes.c_void_p()
    st = B.lib().bsf8_experts_create(ctypes.byref(B._decl("fp8", block)), arr, len(members) if n is None else n, ctypes.byref(h))
    return name(st), h


def _member(E=3, N=300, K=256, grid=None, wd="F8_E4M3", sd="BF16", leaf="scale_inv", addr=FAKE, shape=None):
    return {"weight": dict(dtype=wd, shape=shape or (E, N, K), addr=addr),
            leaf: dict(dtype=sd, shape=grid if grid is not None else (E, -(-N // 128), -(-K // 128)), addr=addr)}


def test_experts_create():
    ok, h = _experts([_member(), _member(N=77)])
    assert ok == "OK"
    L = B.lib()
    e, n, k = ctypes.c_int64(), ctypes.c_int64(), ctypes.c_int64()
    assert L.bsf8_experts_geometry(h, ctypes.byref(e), ctypes.byref(n), ctypes.byref(k)) == 0
    assert (e.value, n.value, k.value) == (3, 377, 256)
    assert "E=3 N=377 K=256" in L.bsf8_experts_describe(h, 10).decode()
    assert name(L.bsf8_experts_geometry(None, None, None, None)) == "INVALID_ARG"
    L.bsf8_experts_destroy(h)
    L.bsf8_experts_destroy(None)
    for want, members, kw in [
            ("GROUP", [], {}), ("GROUP", [_member()] * 9, {}), ("DECL", [_member()], dict(block=(64, 64))),
            ("DECL", [_member()], dict(block=(0, 0))), ("WEIGHT_E5M2", [_member(wd="F8_E5M2")], {}),
            ("WEIGHT_DTYPE", [_member(wd="BF16")], {}), ("WEIGHT_RANK", [_member(shape=(300, 256))], {}),
            ("WEIGHT_RANK", [_member(shape=(1, 3, 300, 256))], {}), ("WEIGHT_EMPTY", [_member(N=0)], {}),
            ("WEIGHT_EMPTY", [_member(E=0)], {}), ("SCALE_RANK", [_member(grid=(3, 2))], {}),
            ("SCALE_RANK", [_member(grid=(3,))], {}), ("SCALE_GRID", [_member(grid=(3, 4, 2))], {}),
            ("SCALE_GRID", [_member(grid=(2, 3, 2))], {}), ("SCALE_TRANSPOSED", [_member(grid=(3, 2, 3))], {}),
            ("SCALE_DTYPE", [_member(sd="F16")], {}), ("SCALE_GRID", [_member(leaf="scale")], {}),
            ("SCALE_MISSING", [dict(weight=_member()["weight"])], {}), ("GROUP", [_member(), _member(E=4)], {}),
            ("GROUP", [_member(), _member(K=384)], {}), ("GROUP", [_member(), _member(sd="F32")], {}),
            ("ALIGNMENT", [_member(addr=FAKE + 8)], {}), ("INVALID_ARG", [_member(addr=0)], {}),
            ("UNSUPPORTED", [_member(E=65536)], {})]:
        got, h = _experts(members, **kw)
        assert got == want and not h.value, (want, got)


def test_experts_refusals():
    L = B.lib()
    ok, h = _experts([_member()])
    assert ok == "OK"

    def call(w=h, xq=FAKE, ldq=256, xs=FAKE, sm=2, sk=1, M=4, off=FAKE, rows=FAKE, R=8, y=FAKE, dt=B.DT_BF16, ldy=300):
        return name(L.bsf8_linear_w8a8_experts(w, xq, ldq, xs, sm, sk, M, off, rows, R, y, dt, ldy, None))

    try:
        assert call(R=0) == "OK"
        for bad in (dict(w=None), dict(M=-1), dict(R=-1), dict(dt=B.DT_F16), dict(M=0), dict(xq=None), dict(xs=None),
                    dict(off=None), dict(y=None), dict(rows=None), dict(ldq=255), dict(ldy=299), dict(sm=1, sk=2)):
            assert call(**bad) == "INVALID_ARG", bad
        for bad in (dict(off=FAKE + 2), dict(rows=FAKE + 1), dict(y=FAKE + 1), dict(xs=FAKE + 3)):
            assert call(**bad) == "ALIGNMENT", bad
        assert call(R=1 << 31) == "UNSUPPORTED"
    finally:
        L.bsf8_experts_destroy(h)


def test_binding_refuses_host_tensors():
    import torch
    x, w = torch.zeros((4, 256)), torch.ones(256)
    with pytest.raises(ValueError, match="GPU tensor"):
        B.quant_norm(x, w)
    with pytest.raises(ValueError, match="GPU tensor"):
        B.expert_plan(torch.zeros((4, 2), dtype=torch.int32), 4)


def test_sizes_beyond_one_launch_and_workspaces():
    """Refused before any launch: more blocks than a launch holds, a workspace that is missing or too small."""
    L = B.lib()
    ok, h = _experts([_member(K=24)])
    assert ok == "OK"
    try:
        assert name(L.bsf8_linear_w8a8_experts(h, FAKE, 24, FAKE, 1, 1, 2 ** 30 - 1, FAKE, FAKE, 2 ** 30 - 1, FAKE,
                                               B.DT_F32, 300, None)) == "UNSUPPORTED"
    finally:
        L.bsf8_experts_destroy(h)

    def weight(N, K):
        arr, keep = B._members_array([{k: dict(d, shape=d["shape"][1:]) for k, d in _member(E=1, N=N, K=K).items()}])
        w = ctypes.c_void_p()
        assert L.bsf8_weight_create(ctypes.byref(B._decl("fp8", (128, 128))), arr, 1, ctypes.byref(w)) == 0
        return w

    def call(w, M, K, N, ws, nbytes):
        return name(L.bsf8_linear_w8a8_epilogue(w, FAKE, K, FAKE, -(-K // 128), 1, M, ctypes.byref(B.Epilogue()), FAKE,
                                                B.DT_F32, N, ws, nbytes, None))

    w = weight(300, 24)
    assert call(w, 2 ** 30 - 1, 24, 300, None, 0) == "UNSUPPORTED"
    L.bsf8_weight_destroy(w)
    w = weight(640, 4096)
    need = ctypes.c_size_t()
    assert L.bsf8_workspace_size(w, B.ARM_W8A8_EPILOGUE, 200, ctypes.byref(need)) == 0 and need.value > 0
    assert call(w, 200, 4096, 640, None, 0) == "WORKSPACE"
    assert call(w, 200, 4096, 640, FAKE, need.value - 1) == "WORKSPACE"
    assert call(w, 200, 4096, 640, FAKE + 128, need.value) == "ALIGNMENT"
    assert L.bsf8_workspace_size(w, B.ARM_W8A8_EPILOGUE, 64, ctypes.byref(need)) == 0 and need.value == 0
    L.bsf8_weight_destroy(w)
