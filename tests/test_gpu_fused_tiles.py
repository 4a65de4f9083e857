"""The tile kernel's instances with an epilogue and for the experts' runs, value by value.

Which kernel takes a call goes by modelled times, so every case first asks describe() whether it is the one meant.
"""
import numpy as np
import pytest

import block_scaled_fp8_linear_amd as B
import test_gpu_epilogue as epilogue
import test_gpu_experts as experts
from gpu_util import banner, device, to_np, torch

pytestmark = pytest.mark.gpu


def expert_kernel(E, rows, K, R, y):
    """The tile of a call of R rows, 0 for the few-row kernel."""
    t = torch()
    members = [(t.zeros((E, n, K), dtype=t.uint8, device=device()),
                t.ones((E, -(-n // 128), -(-K // 128)), dtype=t.bfloat16, device=device())) for n in rows]
    text = B.ExpertsFP8Weight(members).describe(R)
    part = text.split("bf16 outputs: ")[1].split(" | f32 outputs: ")[0 if y == "bf16" else 1]
    return int(part.split("tile=")[1].split("x")[0]) if "tile=" in part else 0


def check_experts(tile, counts, rows, K, y="bf16", extra=3, **terms):
    assert expert_kernel(len(counts), rows, K, sum(counts) + extra, y) == tile
    experts.check(counts, rows, K, y=y, extra=extra, **terms)


# runs that end inside a wave's rows, leave one, two or three of the four column waves without rows, or fill tiles
# exactly; experts without rows; K that ends inside a block; columns that end inside a strip
RUNS = {128: ((129, 0, 1, 255, 256, 31, 97, 65), (1000, 520), 1136),
        256: ((700, 0, 257, 513, 1, 770), (3000, 1200), 400)}
TERMS = [dict(), dict(bad_rows=True), dict(pad=16), dict(pad=3), dict(token_major=True), dict(f32_scales=True),
         dict(extra=40, bad_rows=True, pad=3), dict(gather=False), dict(M=1)]


def _ids(d):
    return "-".join(f"{k}_{v}" for k, v in d.items()) or "plain"


@pytest.mark.parametrize("terms", TERMS, ids=_ids)
@pytest.mark.parametrize("tile,y", [(128, "bf16"), (128, "f32"), (256, "bf16")])
def test_runs_of_tiles(tile, y, terms):
    counts, rows, K = RUNS[tile]
    check_experts(tile, counts, rows, K, y, seed=len(terms), **terms)


@pytest.mark.parametrize("tile,y,rows,K", [(128, "bf16", (2048,), 400), (128, "f32", (2048,), 400), (256, "bf16", (512,), 400)])
def test_more_than_64_experts(tile, y, rows, K):
    g = np.random.default_rng(11)
    c = np.zeros(70, int)
    c[[0, 3, 63, 64, 69]] = (300, 130, 1, 420, 200) if tile == 128 else (2500, 130, 1, 2300, 200)
    c[5:12] = g.integers(1, 300, 7)
    if tile == 128:
        c[20:60:3] = g.integers(100, 400, 14)
    else:
        c[20:60] = g.integers(100, 200, 40)
    check_experts(tile, tuple(int(v) for v in c), rows, K, y)


@pytest.mark.parametrize("tile,y", [(128, "bf16"), (128, "f32"), (256, "bf16")])
def test_offsets_stay_in_bounds(tile, y):
    """Offsets outside [0, R] count as the nearer end; where they descend nothing outside y is written."""
    t = torch()
    R, K = 2000, 400
    rows = (3000, 1200) if tile == 256 else (1000, 200)
    N = sum(rows)
    assert expert_kernel(4, rows, K, R, y) == tile
    w, om = experts.experts(4, rows, K)
    q, s, xq, xs = experts.codes(R, K, 0)
    dt = t.bfloat16 if y == "bf16" else t.float32
    for off in ([-5, 310, 310, 1030, 99999], [2060, 2070, 2080, 2090, 2100], [0, 900, 300, 300, 1900],
                [2 ** 31 - 1, -2 ** 31, 5, 6, 7]):
        banner(f"experts tile={tile} {y} offsets {off}")
        buf = t.full((R + 20, N), 5.0, dtype=dt, device=device())
        out = buf[10:10 + R]
        B.linear_w8a8_experts(w, xq, xs, t.tensor(off, dtype=t.int32, device=device()), out_dtype=dt, out=out)
        t.cuda.synchronize()
        if all(a <= b for a, b in zip(off, off[1:])):
            experts.verify(to_np(out), q, s, om, np.array(off, np.int64), None, N, K, y == "bf16", fp8_mfma=y == "bf16")
        assert bool((buf[:10] == 5.0).all()) and bool((buf[10 + R:] == 5.0).all())


def epilogue_plan(rows, K, M, y):
    """(tile, split_k, split row tiles, row tiles) of a call, from its describe line."""
    t = torch()
    w = B.BlockFP8Weight([(t.zeros((n, K), dtype=t.uint8, device=device()),
                           t.ones((-(-n // 128), -(-K // 128)), dtype=t.bfloat16, device=device())) for n in rows])
    text = w.describe(B.ARM_W8A8_EPILOGUE, M)
    part = text.split("bf16 outputs: ")[1].split(" | f32 outputs: ")[0 if y == "bf16" else 1]
    num = lambda key: int(part.split(key + "=")[1].split()[0].split("x")[0])
    T = num("tile")
    return T, num("split_k"), num("split_row_tiles"), sum(-(-n // T) for n in rows)


def check_epilogue(tile, split, M, rows, K, y="bf16", **terms):
    """split: "none" (whole tiles only), "some" or "all" of the row tiles."""
    T, s, n, total = epilogue_plan(rows, K, M, y)
    assert T == tile and (n == 0, 0 < n < total, n == total) == (split == "none", split == "some", split == "all"), (T, s, n)
    epilogue.check(M, rows, K, y=y, full=False, **terms)


STORES = [dict(), dict(residual="bf16"), dict(residual="f32"), dict(residual="bf16", inplace=True), dict(pad=16, residual="f32"),
          dict(pad=3, residual="bf16"), dict(pad=3, residual="f32", bias="f32"), dict(bias=None), dict(bias="f32"),
          dict(f32_scales=True, token_major=True)]


@pytest.mark.parametrize("terms", STORES, ids=_ids)
@pytest.mark.parametrize("K", [512, 1136])
def test_store_of_whole_256_tiles(terms, K):
    """Members that end inside a tile and a strip, tokens that end inside a wave's."""
    check_epilogue(256, "none", 1000, (6144, 1000, 1000), K, act="gelu_tanh", seed=K, **terms)


@pytest.mark.parametrize("act", [None, "relu", "silu", "gelu"])
def test_activations_of_256_tiles(act):
    check_epilogue(256, "none", 1000, (8192,), 512, act=act, residual="bf16")


@pytest.mark.parametrize("terms", [dict(), dict(residual="f32"), dict(residual="f32", inplace=True),
                                   dict(residual="bf16", pad=16), dict(residual="bf16", pad=3), dict(bias=None)], ids=_ids)
def test_store_of_exact_tiles(terms):
    check_epilogue(128, "none", 300, (9000, 5001), 1152, "f32", act="silu", **terms)


@pytest.mark.parametrize("tile,split,M,rows,K,y", [(256, "some", 1000, (17408,), 1152, "bf16"),
                                                   (128, "some", 300, (9000, 5001), 2048, "f32"),
                                                   (256, "all", 1024, (5120,), 17408, "bf16")])
def test_whole_and_split_tiles_of_one_call(tile, split, M, rows, K, y):
    check_epilogue(tile, split, M, rows, K, y, act="gelu", residual="bf16")
