"""describe lines of the calls with an epilogue and by expert, against the plans they name (no GPU needed)."""
import ctypes
import re

import pytest

import block_scaled_fp8_linear_amd as B
from test_fused_host import _experts, _member


def _describe(rows, K, M):
    members = [{k: dict(d, shape=d["shape"][1:]) for k, d in _member(E=1, N=n, K=K).items()} for n in rows]
    arr, _keep = B._members_array(members)
    w = ctypes.c_void_p()
    assert B.lib().bsf8_weight_create(ctypes.byref(B._decl()), arr, len(rows), ctypes.byref(w)) == 0
    try:
        need = ctypes.c_size_t()
        assert B.lib().bsf8_workspace_size(w, B.ARM_W8A8_EPILOGUE, M, ctypes.byref(need)) == 0
        return B.lib().bsf8_describe(w, B.ARM_W8A8_EPILOGUE, M).decode(), need.value
    finally:
        B.lib().bsf8_weight_destroy(w)


# (the plans of 256 compute units, which the library assumes where there is no device)
@pytest.mark.parametrize("M,rows,K", [(1024, (5120,), 17408), (300, (9000, 5001), 2048), (200, (640,), 4096),
                                      (1000, (6144, 1000, 1000), 512), (1000, (17408,), 1152)])
def test_epilogue_names_both_plans(M, rows, K):
    text, need = _describe(rows, K, M)
    bf16, f32 = text.split(" | bf16 outputs: ")[1].split(" | f32 outputs: ")
    assert "f8f6f4" in bf16 and "f8f6f4" not in f32 and "mfma_f32_16x16x32_bf16" in f32
    ws = []
    for part in (bf16, f32):
        T, splits, tiles = (int(re.search(key + r"=(\d+)", part).group(1)) for key in ("tile", "split_k", "split_row_tiles"))
        assert (splits > 1) == (tiles > 0) and tiles <= sum(-(-n // T) for n in rows)
        ws.append(splits * M * tiles * T * 4 if splits > 1 else 0)
    assert "tile=128x128" in f32
    assert max(ws) == need   # the workspace covers the larger of the plans the line names


def test_few_tokens_name_the_few_row_kernel():
    text, need = _describe((640,), 4096, 64)
    assert "w8a8_rows" in text and "outputs:" not in text and need == 0


def test_experts_name_both_kernels():
    ok, h = _experts([_member(E=4, N=3000, K=400)])
    assert ok == "OK"
    text = B.lib().bsf8_experts_describe(h, 4000).decode()
    B.lib().bsf8_experts_destroy(h)
    bf16, f32 = text.split(" | bf16 outputs: ")[1].split(" | f32 outputs: ")
    assert "tile=256x256" in bf16 and "tile=128x128" in f32
