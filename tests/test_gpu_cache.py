"""The paged cache: what is written is what the activation quantizer (the oracle's) makes of the rotated rows, what is read
back is code times scale, and everything else stays as it was."""
import numpy as np
import pytest

import block_scaled_fp8_linear_amd as B
import oracle as O
from cache_util import LAYOUTS, cache_values, new_cache
from gpu_util import banner, device, torch

pytestmark = pytest.mark.gpu


def _bits(x):
    t = torch()
    x = x.contiguous()
    return x.view({1: t.uint8, 2: t.int16, 4: t.int32}[x.element_size()])


def _expected(cache, tensors, f32, slots, which):
    """The cache's tensor (and scales) with the float32 rows [M, heads, D] put at their slots, on the CPU."""
    t = torch()
    x = getattr(cache, which).cpu().clone()
    s = getattr(cache, which + "_scale")
    s = None if s is None else s.cpu().clone()
    rows = f32.cpu().numpy()
    for m, slot in enumerate(slots):
        if not 0 <= slot < cache.n_pages * cache.page_size:
            continue
        p, r = divmod(int(slot), cache.page_size)
        if s is None:
            x[p, r] = f32[m].cpu().to(t.bfloat16)
            continue
        q, sc = O.quant_act(rows[m])
        x[p, r] = t.from_numpy(q)
        s[p, r] = t.from_numpy(sc)
    return x, s


def _write_and_check(cache, held, k, v, slots, f32_k, f32_v, **kw):
    t = torch()
    want = [_expected(cache, held, f, slots.tolist(), w) for f, w in ((f32_k, "k"), (f32_v, "v"))]
    around = [h.clone() for h in held]
    out = B.cache_write(cache, k, v, slots, **kw)
    for (x, s), w in zip(want, "kv"):
        assert t.equal(_bits(getattr(cache, w)).cpu(), _bits(x)), w
        if s is not None:
            assert t.equal(_bits(getattr(cache, w + "_scale")).cpu(), _bits(s)), w + "_scale"
    # what lies between the rows of a padded layout is untouched: put the old rows back and compare all of the memory
    after = [h.clone() for h in held]
    return out, around, after


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("codes", [True, False])
@pytest.mark.parametrize("M,heads,D,page,x", [(1, 1, 16, 1, "f32"), (19, 8, 128, 16, "bf16"), (40, 3, 80, 7, "f32"),
                                              (11, 4, 256, 24, "bf16"), (6, 5, 192, 64, "f32"), (30, 24, 64, 5, "bf16"),
                                              (900, 2, 128, 32, "bf16")])
def test_write(layout, codes, M, heads, D, page, x):
    t = torch()
    g = np.random.default_rng(M + D)
    pages = -(-M // page) + 2
    cache, held = new_cache(layout, pages, page, heads, D, codes)
    dt = t.bfloat16 if x == "bf16" else t.float32
    kv = t.from_numpy(g.standard_normal((M, 2 * heads, D)).astype(np.float32) * 3).to(device()).to(dt)
    kv[0, 0] = 0                     # a row of zeros: scale 1e-10 / 448
    kv[0, 0, 1] = -0.0
    slots = g.permutation(pages * page)[:M]
    if M > 2:
        slots[1], slots[2] = -1, pages * page + (0 if M % 2 else 2 ** 33)
    slots = t.from_numpy(slots).to(device())
    if not bool((slots > 2 ** 31).any()) and M % 3:
        slots = slots.int()
    banner(f"cache_write {layout} codes={codes} M={M} heads={heads} D={D} page={page} {x}")
    _, around, after = _write_and_check(cache, held, kv[:, :heads], kv[:, heads:], slots, kv[:, :heads].float(),
                                        kv[:, heads:].float())
    if layout == "padded":
        for a, b in zip(around, after):
            if a.dim() == 4 and a.shape[3] == D + 32:
                assert t.equal(_bits(a[:, :, heads:]), _bits(b[:, :, heads:]))
                assert t.equal(_bits(a[..., :16]), _bits(b[..., :16])) and t.equal(_bits(a[..., 16 + D:]), _bits(b[..., 16 + D:]))


@pytest.mark.parametrize("codes", [True, False])
@pytest.mark.parametrize("pairing,R,axes,norm,D", [("half", 128, 1, False, 128), ("half", 64, 3, True, 256),
                                                   ("adjacent", 80, 2, True, 80), ("half", 20, 1, False, 96),
                                                   ("half", 0, 1, True, 64), ("adjacent", 34, 1, False, 64)])
def test_write_rotates(codes, pairing, R, axes, norm, D):
    """Keys are stored as rope's float32 output quantizes, values as they are, queries come back as rope gives them."""
    t = torch()
    g = np.random.default_rng(R + D)
    M, H, KV, page = 29, 6, 3, 16
    cache, held = new_cache("head_major", 4, page, KV, D, codes)
    qkv = t.from_numpy(g.standard_normal((M, H + 2 * KV, D)).astype(np.float32)).to(device()).bfloat16()
    q, k, v = qkv[:, :H], qkv[:, H:H + KV], qkv[:, H + KV:]
    inv = t.from_numpy((1e4 ** (-np.arange(0, R, 2) / max(R, 1))).astype(np.float32)).to(device()) if R else None
    pos = t.from_numpy(g.integers(0, 10 ** 5, (axes, M))).to(device()) if R else None
    n = R // 2 // axes
    kw = dict(pairing=pairing, eps=1e-5, scale=0.75)
    kw["axes"] = B.rope_axes([R // 2 - n * (axes - 1)] + [n] * (axes - 1)) if axes > 1 else None
    w = [1 + 0.1 * t.randn(D, device=device()) if norm else None for _ in "qk"]
    slots = t.from_numpy(g.permutation(4 * page)[:M]).to(device())
    slots[3] = -7
    f32_q, f32_k = B.rope(q, pos, inv, k=k, q_weight=w[0], k_weight=w[1], out_dtype=t.float32, **kw)
    banner(f"cache_write rotated codes={codes} {pairing} R={R} axes={axes} norm={norm} D={D}")
    out, _, _ = _write_and_check(cache, held, k, v, slots, f32_k, v.float(), positions=pos, inv_freq=inv, k_weight=w[1],
                                 q=q, q_weight=w[0], **kw)
    assert out.dtype == t.bfloat16 and t.equal(_bits(out), _bits(f32_q.bfloat16()))
    out, _, _ = _write_and_check(cache, held, k, v, slots, f32_k, v.float(), positions=pos, inv_freq=inv, k_weight=w[1],
                                 **kw)
    assert out is None


def _table(g, lens, page, pages):
    need = [-(-n // page) for n in lens]
    table = np.full((len(lens), max(1, max(need))), -1, np.int32)
    perm = g.permutation(pages)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = perm[at:at + n]
        at += n
    return table


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("codes", [True, False])
@pytest.mark.parametrize("y", ["bf16", "f32"])
@pytest.mark.parametrize("lens,heads,D,page", [([1], 1, 16, 1), ([0, 5, 0, 0, 37, 1, 0], 3, 80, 7), ([64, 64], 8, 128, 16),
                                               ([100, 3, 250], 5, 256, 24), ([9] * 70, 2, 192, 3), ([700], 6, 64, 64)])
def test_read(layout, codes, y, lens, heads, D, page):
    t = torch()
    g = np.random.default_rng(sum(lens))
    pages = sum(-(-n // page) for n in lens) + 2
    cache, _ = new_cache(layout, pages, page, heads, D, codes)
    table = _table(g, lens, page, pages)
    ends = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    R = int(ends[-1]) + 3                       # rows behind the last sequence
    dt = t.bfloat16 if y == "bf16" else t.float32
    out = [t.full((R, heads, D + 8), 7.0, dtype=dt, device=device())[..., :D] for _ in "kv"]
    banner(f"cache_read {layout} codes={codes} {y} lens={lens[:8]} heads={heads} D={D} page={page}")
    B.cache_read(cache, t.from_numpy(table).to(device()), t.from_numpy(ends).to(device()), R, k_out=out[0], v_out=out[1])
    for got, vals in zip(out, cache_values(cache)):
        want = np.full((R, heads, D), 7.0)
        for b, n in enumerate(lens):
            pos = np.arange(n)
            want[ends[b]:ends[b + 1]] = vals[table[b, pos // page], pos % page]
        want = t.from_numpy(want.astype(np.float32)).to(dt)
        assert t.equal(_bits(got).cpu(), _bits(want))


def test_read_starts_bad_pages_and_bounds():
    """First positions other than 0, pages that are none, positions past the table, offsets outside [0, R]."""
    t = torch()
    cache, _ = new_cache("token_major", 6, 8, 2, 32, True)
    table = np.array([[0, 6, 2], [-1, 5, 4], [3, 1, -2147483648]], np.int32)
    starts = np.array([5, 12, -3], np.int32)
    ends = np.array([-4, 20, 27, 99], np.int32)
    R = 40
    vals = cache_values(cache)
    banner("cache_read bad pages")
    k, v = B.cache_read(cache, t.from_numpy(table).to(device()), t.from_numpy(ends).to(device()), R,
                        starts=t.from_numpy(starts).to(device()), out_dtype=t.float32)
    for got, val in ((k, vals[0]), (v, vals[1])):
        got = got.cpu().numpy()
        lo = np.clip(ends, 0, R)
        for b in range(3):
            for r in range(lo[b], lo[b + 1]):
                pos = starts[b] + r - lo[b]
                page = table[b, pos // 8] if 0 <= pos < 24 else -1
                want = val[page, pos % 8] if 0 <= page < 6 else 0.0
                assert (got[r] == want).all(), (b, r)


def test_written_then_read():
    """A round trip: every value comes back within half an E4M3 step of its group (2^-4 relative, 2^-10 of the scale)."""
    t = torch()
    g = np.random.default_rng(8)
    M, heads, D, page = 300, 4, 160, 16
    cache = B.PagedKVCache.new(M // page + 2, page, heads, D, device=device())
    assert cache.k.dtype == t.uint8 and cache.k_scale.shape == (M // page + 2, page, heads, 2)
    kv = t.from_numpy(g.standard_normal((M, 2, heads, D)).astype(np.float32)).to(device())
    table = t.from_numpy(g.permutation(M // page + 2).astype(np.int32)[None]).to(device())
    pos = t.arange(M, device=device())
    slots = table[0].long()[pos // page] * page + pos % page
    banner("cache round trip")
    assert B.cache_write(cache, kv[:, 0], kv[:, 1], slots) is None
    k, v = B.cache_read(cache, table, t.tensor([0, M], dtype=t.int32, device=device()), M, out_dtype=t.float32)
    for got, x in ((k, kv[:, 0]), (v, kv[:, 1])):
        amax = t.nn.functional.pad(x, (0, 96)).unflatten(-1, (2, 128)).abs().amax(-1)
        scale = (amax / 448).repeat_interleave(128, -1)[..., :D]
        # the scale's and the quotient's F32 roundings besides
        assert bool(((got - x).abs() <= x.abs() * (2.0 ** -4 + 2.0 ** -21) + scale * (2.0 ** -10 + 2.0 ** -21)).all())
    b = B.PagedKVCache.new(2, 8, 1, 16, dtype=t.bfloat16, device=device())
    assert b.k_scale is None and b.k.dtype == t.bfloat16


def test_nothing_to_do():
    t = torch()
    cache, held = new_cache("head_major", 2, 4, 2, 32, True)
    before = [h.clone() for h in held]
    e = t.empty(0, 2, 32, device=device())
    assert B.cache_write(cache, e, e, t.empty(0, dtype=t.int64, device=device())) is None
    x = t.randn(3, 2, 32, device=device())
    B.cache_write(cache, x, x, t.full((3,), -1, dtype=t.int32, device=device()))
    k, v = B.cache_read(cache, t.zeros(0, 1, dtype=t.int32, device=device()), t.zeros(1, dtype=t.int32, device=device()), 0)
    assert k.shape == (0, 2, 32)
    t.cuda.synchronize()
    for a, b in zip(before, held):
        assert t.equal(_bits(a), _bits(b))
