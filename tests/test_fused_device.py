"""Which device is current while the library is asked, with the device calls recorded in place of made (no GPU needed)."""
import types

import pytest

import block_scaled_fp8_linear_amd as B


@pytest.mark.parametrize("current,owner", [(0, 1), (1, 0), (1, 1)])
def test_workspace_is_asked_on_the_weights_device(monkeypatch, current, owner):
    """The plan behind a workspace goes by the current device's compute units, and the call runs on the weight's."""
    import torch
    state = [current]

    class Guard:
        def __init__(self, idx):
            self.idx = idx

        def __enter__(self):
            self.old, state[0] = state[0], self.idx

        def __exit__(self, *exc):
            state[0] = self.old

    seen = []

    def size(handle, arm, M, out):
        seen.append(state[0])
        return 0

    monkeypatch.setattr(torch.cuda, "device", Guard)
    monkeypatch.setattr(B, "_CURRENT", (lambda: state[0], lambda idx: 0))
    monkeypatch.setattr(B, "lib", lambda: types.SimpleNamespace(bsf8_workspace_size=size))
    w = B.BlockFP8Weight.__new__(B.BlockFP8Weight)
    w._h, w.device = None, types.SimpleNamespace(index=owner)
    assert w.workspace_size(B.ARM_W8A8_EPILOGUE, 200) == 0
    assert seen == [owner] and state == [current]


@pytest.mark.parametrize("shape,strides,given", [(100, None, 101), (0, None, 1), (None, None, 256), ((8, 64), (128, 1), 512)])
def test_a_workspace_shorter_than_it_says_is_refused(monkeypatch, shape, strides, given):
    """The library is told the bytes of the workspace, so they must be there."""
    import torch
    called = []
    w = types.SimpleNamespace(device=types.SimpleNamespace(index=-1), K=256, n_total=64, handle=None)
    xq, xs = torch.zeros((4, 256), dtype=torch.uint8), torch.zeros((4, 2))
    out = torch.zeros((4, 64), dtype=torch.bfloat16)
    monkeypatch.setattr(B, "_CURRENT", (lambda: -1, lambda idx: 0))
    monkeypatch.setattr(B, "lib", lambda: types.SimpleNamespace(bsf8_linear_w8a8_epilogue=lambda *a: called.append(a) or 0))
    ws = None if shape is None else torch.zeros(shape, dtype=torch.uint8)
    if strides:
        ws = torch.zeros(1024, dtype=torch.uint8).as_strided(shape, strides)
    with pytest.raises(ValueError, match="workspace"):
        B.linear_w8a8_epilogue(w, xq, xs, out=out, workspace=(ws, given))
    assert not called
    B.linear_w8a8_epilogue(w, xq, xs, out=out, workspace=(torch.zeros(512, dtype=torch.uint8), 512))
    B.linear_w8a8_epilogue(w, xq, xs, out=out, workspace=(None, 0))
    assert len(called) == 2
