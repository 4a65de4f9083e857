"""bsf8_expert_plan against a stable sort on the CPU, value for value."""
import numpy as np
import pytest

import block_scaled_fp8_linear_amd as B
from gpu_util import banner, device, torch

pytestmark = pytest.mark.gpu


def plan_ref(ids, E):
    M, top = ids.shape
    flat = ids.reshape(-1).astype(np.int64)
    ok = (flat >= 0) & (flat < E)
    order = np.argsort(np.where(ok, flat, E), kind="stable")[:int(ok.sum())]
    slots = np.full(flat.shape, -1, np.int32)
    slots[order] = np.arange(order.size)
    offsets = np.concatenate([[0], np.cumsum(np.bincount(flat[ok], minlength=E))])
    return offsets, order // top, slots.reshape(M, top)


def check(ids, E, dtype="int32", shift=0):
    t = torch()
    M, top = ids.shape
    banner(f"expert_plan M={M} top={top} E={E} {dtype} shift={shift}")
    dt = t.int64 if dtype == "int64" else t.int32
    buf = t.zeros(M * top + shift, dtype=dt, device=device())
    d = buf[shift:].view(M, top)
    d.copy_(t.from_numpy(ids.astype(np.int64)))
    rows = t.full((M * top,), -7, dtype=t.int32, device=device())
    off, r, sl = B.expert_plan(d, E, rows=rows)
    ro, rr, rs = plan_ref(ids, E)
    assert np.array_equal(off.cpu().numpy(), ro)
    assert np.array_equal(sl.cpu().numpy(), rs)
    got = r.cpu().numpy()
    assert np.array_equal(got[:rr.size], rr) and np.all(got[rr.size:] == -7)


@pytest.mark.parametrize("dtype", ["int32", "int64"])
@pytest.mark.parametrize("M,top,E", [(1, 1, 1), (1, 8, 64), (3, 2, 5), (64, 8, 64), (257, 1, 300), (1023, 4, 7),
                                     (4096, 4, 32), (8195, 8, 128)])
def test_plan(M, top, E, dtype):
    g = np.random.default_rng(M + top + E)
    check(g.integers(-1, E + 1, (M, top)), E, dtype)


@pytest.mark.parametrize("shift", [1, 2, 3])
@pytest.mark.parametrize("dtype", ["int32", "int64"])
def test_unaligned(dtype, shift):
    check(np.random.default_rng(shift).integers(0, 9, (501, 3)), 9, dtype, shift)


def test_one_sided():
    """Every choice one expert (the first, the last); none with an expert; the same expert twice in a token;
    numbers at the ends of the type."""
    check(np.zeros((700, 2), int), 4)
    check(np.full((700, 2), 3), 4)
    check(np.full((700, 2), -1), 4)
    check(np.full((5, 2), 2 ** 31 - 1), 4)
    check(np.array([[2 ** 62, 1], [-2 ** 62, 2 ** 32], [3, 2 ** 32 + 3]]), 4, "int64")


def test_no_tokens():
    t = torch()
    off, r, sl = B.expert_plan(t.empty((0, 2), dtype=t.int32, device=device()), 6)
    assert off.cpu().tolist() == [0] * 7 and r.numel() == 0 and sl.shape == (0, 2)


def test_graph():
    t = torch()
    ids = t.from_numpy(np.random.default_rng(1).integers(0, 16, (100, 4)).astype(np.int32)).to(device())
    out = [t.zeros(17, dtype=t.int32, device=device()), t.zeros(400, dtype=t.int32, device=device()),
           t.zeros((100, 4), dtype=t.int32, device=device())]
    banner("expert_plan captured")
    B.expert_plan(ids, 16, *out)
    graph = t.cuda.CUDAGraph()
    with t.cuda.graph(graph):
        B.expert_plan(ids, 16, *out)
    for rep in range(3):
        ids.copy_(t.from_numpy(np.random.default_rng(rep).integers(-1, 16, (100, 4)).astype(np.int32)))
        ro, rr, rs = plan_ref(ids.cpu().numpy(), 16)
        t.cuda.synchronize()
        graph.replay()
        t.cuda.synchronize()
        assert np.array_equal(out[0].cpu().numpy(), ro) and np.array_equal(out[2].cpu().numpy(), rs)
        assert np.array_equal(out[1].cpu().numpy()[:rr.size], rr)
