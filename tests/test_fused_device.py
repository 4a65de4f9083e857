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
