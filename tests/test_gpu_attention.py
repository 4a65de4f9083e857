"""Attention of one token over a paged cache against its definition in 64 bits."""
import numpy as np
import pytest

import block_scaled_fp8_linear_amd as B
from cache_util import LAYOUTS, attention64, cache_values, make_table, new_cache, to_f64
from gpu_util import banner, device, torch

pytestmark = pytest.mark.gpu


def _spoil(cache, table, lens):
    """Everything that is no sequence's row holds NaN (codes 0x7f, scales too)."""
    t = torch()
    used = np.zeros((cache.n_pages, cache.page_size), bool)
    for b, n in enumerate(lens):
        pos = np.arange(max(n, 0))
        pg = table[b, pos // cache.page_size] if n > 0 else np.zeros(0, int)
        ok = (pg >= 0) & (pg < cache.n_pages)
        used[pg[ok], (pos % cache.page_size)[ok]] = True
    free = t.from_numpy(~used).to(device())[..., None, None]
    for x in (cache.k, cache.v):
        x.copy_(t.where(free, t.full_like(x, 0x7F) if x.dtype == t.uint8 else t.full_like(x, float("nan")), x))
    for x in (cache.k_scale, cache.v_scale):
        if x is not None:
            x.copy_(t.where(free, t.full_like(x, float("nan")), x))


def _check(out, lse, q, cache, values, table, lens, window, scale):
    t = torch()
    want, wl, tol, tl = attention64(to_f64(q), values, table, lens, cache.page_size, window, scale, cache.n_pages)
    got = to_f64(out)
    tol = tol + (2.0 ** -8 if out.dtype == t.bfloat16 else 2.0 ** -24) * (np.abs(want) + tol) + 1e-37
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (np.argwhere(bad)[:5], float(np.nanmax(np.abs(got - want) / tol)), got[bad][:5], want[bad][:5])
    if lse is not None:
        got = to_f64(lse)
        none = np.isneginf(wl)
        assert (np.isneginf(got) == none).all()
        with np.errstate(invalid="ignore"):
            assert (np.abs(got - wl)[~none] <= (tl + 2.0 ** -23 * np.abs(wl))[~none]).all()


def _run(lens, heads, kv, D, page, codes, layout="head_major", q_dt="bf16", out_dt=None, window=0, spoil=True, seed=0,
         columns=None, scale=None):
    t = torch()
    g = np.random.default_rng(seed + sum(lens) + D)
    pages = sum(-(-max(n, 0) // page) for n in lens) + 3
    cache, _ = new_cache(layout, pages, page, kv, D, codes)
    if codes:   # scales of a plausible size: values up to 448 / 200
        for s in (cache.k_scale, cache.v_scale):
            s.mul_(0.01)
    else:
        for x in (cache.k, cache.v):
            x.copy_(t.randn_like(x, dtype=t.float32).bfloat16())
    table = make_table(g, [max(n, 0) for n in lens], page, pages, columns)
    values = cache_values(cache)
    if spoil:
        _spoil(cache, table, lens)
    dt = {"bf16": t.bfloat16, "f32": t.float32}
    q = t.from_numpy((1.5 * g.standard_normal((len(lens), heads, D))).astype(np.float32)).to(device()).to(dt[q_dt])
    banner(f"paged_attention lens={lens[:10]} heads={heads}/{kv} D={D} page={page} codes={codes} {layout} {q_dt}->{out_dt} "
           f"window={window} columns={table.shape[1]}")
    out, lse = B.paged_attention(q, cache, t.from_numpy(table).to(device()),
                                 t.tensor(lens, dtype=t.int32, device=device()), window=window, lse=True,
                                 scale=scale, out_dtype=dt.get(out_dt))
    t.cuda.synchronize()
    assert out.dtype == dt[out_dt or q_dt]
    _check(out, lse, q, cache, values, table, lens, window, D ** -0.5 if scale is None else scale)


EDGES = [0, 1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 400]


@pytest.mark.parametrize("codes", [True, False])
@pytest.mark.parametrize("q_dt,out_dt", [("bf16", None), ("f32", None), ("bf16", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("heads,kv,D,page", [(4, 2, 128, 16), (3, 3, 64, 32), (10, 2, 256, 16), (5, 1, 80, 24)])
def test_lengths(codes, q_dt, out_dt, heads, kv, D, page):
    """Every length around the edges of a tile, in one batch and alone."""
    _run(EDGES, heads, kv, D, page, codes, q_dt=q_dt, out_dt=out_dt)
    for n in (0, 1, 33, 129):
        _run([n], heads, kv, D, page, codes, q_dt=q_dt, out_dt=out_dt)


@pytest.mark.parametrize("codes", [True, False])
@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("page", [1, 3, 7, 8, 16, 24, 48, 64, 128, 1000])
def test_pages_and_layouts(codes, layout, page):
    _run([5, 700, 1, 130, 0, 64], 8, 2, 96, page, codes, layout=layout)


@pytest.mark.parametrize("codes", [True, False])
@pytest.mark.parametrize("D", [16, 32, 48, 64, 112, 128, 144, 160, 192, 240, 256])
@pytest.mark.parametrize("G", [1, 7, 16, 17, 40])
def test_head_dims_and_groups(codes, D, G):
    _run([200, 33, 1], 2 * G, 2, D, 16, codes)
    _run([70], 3 * G, 3, D, 5, codes, q_dt="f32")


@pytest.mark.parametrize("codes", [True, False])
@pytest.mark.parametrize("window", [1, 2, 31, 32, 100, 128, 129, 1000, 10 ** 9])
@pytest.mark.parametrize("page", [16, 7])
def test_window(codes, window, page):
    _run([0, 1, 32, 100, 128, 129, 500, 1025], 6, 2, 128, page, codes, window=window)


@pytest.mark.parametrize("codes", [True, False])
@pytest.mark.parametrize("lens,heads,kv,D,page", [([20000], 8, 1, 128, 16), ([30001], 4, 4, 64, 64), ([9000, 3, 17000], 10, 2, 256, 32),
                                                  ([5000] + [1] * 300, 4, 2, 128, 16), (list(range(1, 1200, 3)), 5, 5, 80, 16),
                                                  ([40000], 20, 1, 192, 128), ([4099] * 9, 32, 8, 128, 13)])
def test_long_and_ragged(codes, lens, heads, kv, D, page):
    """Items that lie in many blocks, blocks that hold many items, more than 64 sequences."""
    _run(lens, heads, kv, D, page, codes)
    if len(lens) < 10:
        _run(lens, heads, kv, D, page, codes, q_dt="f32", window=3000)


def test_wide_table_and_clamped_lengths():
    """A table far wider than the lengths, and lengths outside [0, pages * page_size]."""
    _run([40, 0, 300], 4, 2, 128, 16, True, columns=5000)
    t = torch()
    g = np.random.default_rng(1)
    cache, _ = new_cache("head_major", 9, 16, 2, 64, False)
    table = g.permutation(9)[:8].reshape(2, 4).astype(np.int32)
    q = t.randn(2, 4, 64, device=device())
    for lens in ([1000, -5], [2 ** 31 - 1, -2 ** 31], [64, 65]):
        out, lse = B.paged_attention(q, cache, t.from_numpy(table).to(device()), t.tensor(lens, dtype=t.int32, device=device()),
                                     lse=True)
        _check(out, lse, q, cache, cache_values(cache), table, lens, 0, 0.125)


@pytest.mark.parametrize("codes", [True, False])
@pytest.mark.parametrize("page", [16, 10])
def test_bad_pages(codes, page):
    """Positions on pages outside the cache are left out; a sequence of nothing else has zeros and -inf."""
    t = torch()
    g = np.random.default_rng(2)
    lens = [300, 45, 161, 20]
    cache, _ = new_cache("token_major", 60, page, 2, 64, codes)
    if codes:
        cache.k_scale.mul_(0.01), cache.v_scale.mul_(0.01)
    table = make_table(g, lens, page, 60)
    table[0, ::3] = -1
    table[0, 1] = 60
    table[2, 4] = 2 ** 31 - 1
    table[3] = -2 ** 31
    values = cache_values(cache)
    q = t.randn(4, 6, 64, device=device())
    banner(f"paged_attention bad pages codes={codes} page={page}")
    out, lse = B.paged_attention(q, cache, t.from_numpy(table).to(device()), t.tensor(lens, dtype=t.int32, device=device()), lse=True)
    _check(out, lse, q, cache, values, table, lens, 0, 0.125)
    assert not out[3].any() and bool(t.isneginf(lse[3]).all())


def test_strided_queries_and_outputs():
    """Queries inside a projection's output, at any element alignment; outputs with gaps that stay as they were."""
    t = torch()
    g = np.random.default_rng(3)
    lens = [90, 250, 0, 14]
    cache, _ = new_cache("head_major", 30, 16, 2, 96, True)
    cache.k_scale.mul_(0.01), cache.v_scale.mul_(0.01)
    table = make_table(g, lens, 16, 30)
    wide = np.full((4, 40), 77, np.int32)
    wide[:, 3:3 + table.shape[1]] = table
    tab = t.from_numpy(wide).to(device())[:, 3:3 + table.shape[1]]
    ln = t.tensor(lens, dtype=t.int32, device=device())
    for dt in (t.bfloat16, t.float32):
        rows = t.randn(4, 8 * 96 + 5, device=device()).to(dt)
        q = rows[:, 3:3 + 6 * 96].unflatten(1, (6, 96))
        banner(f"paged_attention strided {dt}")
        want, wl = B.paged_attention(q.contiguous(), cache, tab, ln, lse=True)
        _check(want, wl, q, cache, cache_values(cache), table, lens, 0, 96 ** -0.5)
        hold = t.full((4, 7, 101), 5.0, dtype=dt, device=device())
        out = hold[:, 1:, 2:98]
        got = B.paged_attention(q, cache, tab, ln, out=out)
        assert got.data_ptr() == out.data_ptr() and t.equal(got, want)
        out.fill_(5.0)
        assert bool((hold == 5.0).all())


@pytest.mark.parametrize("codes", [True, False])
def test_large_logits_and_scales(codes):
    """Logits of hundreds, a maximum that rises late, a scale of zero and a negative one."""
    _run([600, 40], 4, 2, 64, 16, codes, scale=3.0)
    _run([600, 40], 4, 2, 64, 16, codes, scale=0.0)
    _run([600, 40], 4, 2, 64, 16, codes, scale=-0.3, q_dt="f32")


def test_a_scale_beyond_f32():
    """Weights of one and zero: the value of the largest logit."""
    t = torch()
    cache, _ = new_cache("head_major", 50, 16, 1, 64, False)
    cache.k.normal_(), cache.v.normal_()
    table = t.arange(50, dtype=t.int32, device=device())[None]
    q = t.zeros(1, 2, 64, device=device())
    q[0, 0, 0], q[0, 1, 0] = 1.0, -1.0
    cache.k[30, 5, 0, 0], cache.k[7, 2, 0, 0] = 100.0, -100.0
    banner("paged_attention of a scale of 1e300")
    for n in (400, 800):   # (the first head's largest logit is among the tokens of the second alone)
        out = B.paged_attention(q, cache, table, t.tensor([n], dtype=t.int32, device=device()), scale=1e300)
        assert t.equal(out[0, 1], cache.v[7, 2, 0].float())
        assert n == 400 or t.equal(out[0, 0], cache.v[30, 5, 0].float())
        assert bool(out.isfinite().all())
    t = torch()
    cache, _ = new_cache("head_major", 20, 16, 1, 64, False)
    n = 310
    cache.k.zero_()
    ramp = t.arange(320, device=device(), dtype=t.float32).view(20, 16, 1)
    cache.k[..., 0] = ramp.bfloat16()
    q = t.zeros(1, 2, 64, device=device())
    q[0, 0, 0], q[0, 1, 0] = 1.0, -1.0
    table = np.arange(20, dtype=np.int32)[None]
    out, lse = B.paged_attention(q, cache, t.from_numpy(table).to(device()), t.tensor([n], dtype=t.int32, device=device()), scale=1.0, lse=True)
    _check(out, lse, q, cache, cache_values(cache), table, [n], 0, 1.0)


def test_same_result_every_time():
    """The sums' order goes by lengths alone, never by timing."""
    t = torch()
    g = np.random.default_rng(4)
    lens = [7000, 12, 3000, 0, 999]
    cache, _ = new_cache("head_major", 720, 16, 4, 128, True)
    cache.k_scale.mul_(0.01), cache.v_scale.mul_(0.01)
    tab = t.from_numpy(make_table(g, lens, 16, 720)).to(device())
    ln = t.tensor(lens, dtype=t.int32, device=device())
    q = t.randn(5, 16, 128, device=device()).bfloat16()
    banner("paged_attention repeated")
    first = B.paged_attention(q, cache, tab, ln)
    for _ in range(20):
        assert t.equal(first, B.paged_attention(q, cache, tab, ln))


@pytest.mark.parametrize("lens", [[40, 300], [5000, 12]])
@pytest.mark.parametrize("codes", [True, False])
def test_nan_is_not_hidden(lens, codes):
    """A query or a cached row of NaN gives NaN to the heads that meet it, in one block or joined, and to no other."""
    t = torch()
    g = np.random.default_rng(5)
    pages = sum(-(-n // 16) for n in lens) + 1
    cache, _ = new_cache("head_major", pages, 16, 2, 64, codes)
    if codes:
        cache.k_scale.mul_(0.01), cache.v_scale.mul_(0.01)
    table = make_table(g, lens, 16, pages)
    tab, ln = t.from_numpy(table).to(device()), t.tensor(lens, dtype=t.int32, device=device())
    q = t.randn(2, 4, 64, device=device())
    want, wl = B.paged_attention(q, cache, tab, ln, lse=True)
    banner(f"paged_attention NaN lens={lens} codes={codes}")
    bad = q.clone()
    bad[0, 1, 3] = float("nan")
    out, lse = B.paged_attention(bad, cache, tab, ln, lse=True)
    assert bool(out[0, 1].isnan().all()) and bool(lse[0, 1].isnan())
    keep = t.ones(2, 4, dtype=t.bool, device=device())
    keep[0, 1] = False
    assert t.equal(out[keep], want[keep]) and t.equal(lse[keep], wl[keep])
    row = lens[0] // 2
    page = int(table[0, row // 16])
    for x in (cache.k, cache.v):
        old = x.clone()
        x[page, row % 16, 1, 5] = 0x7F if codes else float("nan")
        out, lse = B.paged_attention(q, cache, tab, ln, lse=True)
        hit = out[0, 2:].isnan()
        assert bool(hit.all()) if x is cache.k else bool(hit[:, 5].all()) and int(hit.sum()) == 2
        assert t.equal(out[0, :2], want[0, :2]) and t.equal(out[1], want[1])
        x.copy_(old)


def test_no_sequences():
    t = torch()
    cache, _ = new_cache("head_major", 2, 16, 1, 64, False)
    e = t.empty(0, 3, 64, device=device())
    out, lse = B.paged_attention(e, cache, t.empty(0, 4, dtype=t.int32, device=device()), t.empty(0, dtype=t.int32, device=device()), lse=True)
    assert out.shape == (0, 3, 64) and lse.shape == (0, 3)


def _small_scale(q_exp, k_exp, scale, q_dt, codes, lens, page=16, D=64):
    """Queries of about 2^q_exp over keys of about 2^k_exp."""
    t = torch()
    g = np.random.default_rng(sum(lens) + page)
    pages = sum(-(-n // page) for n in lens) + 2
    cache, _ = new_cache("head_major", pages, page, 2, D, codes)
    if codes:   # codes of about 2^4, and scales to match
        cache.k_scale.mul_(2.0 ** (k_exp - 4)), cache.v_scale.mul_(0.01)
    else:
        cache.k.copy_((t.randn_like(cache.k, dtype=t.float32) * 2.0 ** k_exp).bfloat16()), cache.v.normal_()
    table = make_table(g, lens, page, pages)
    q = t.from_numpy((2.0 ** q_exp * g.standard_normal((len(lens), 6, D))).astype(np.float32)).to(device())
    q = q.bfloat16() if q_dt == "bf16" else q
    banner(f"paged_attention scale {scale} of 2^{q_exp} x 2^{k_exp} {q_dt} codes={codes} lens={lens} page={page} D={D}")
    out, lse = B.paged_attention(q, cache, t.from_numpy(table).to(device()), t.tensor(lens, dtype=t.int32, device=device()),
                                 scale=scale, lse=True, out_dtype=t.float32)
    _check(out, lse, q, cache, cache_values(cache), table, lens, 0, scale)
    return out


@pytest.mark.parametrize("q_dt", ["bf16", "f32"])
@pytest.mark.parametrize("codes", [True, False])
@pytest.mark.parametrize("lens", [[40, 300, 0, 1], [5000, 12]])
def test_small_scales(q_dt, codes, lens):
    """A scale far below the smallest that a model has counts as it is: logits of about one and of some tens from queries and keys
    of 10^18 (2^60), on either side of 2^-100, where queries are taken down by 2^64, and of either sign; a scale of zero, and
    others whose logits are zero, whatever the products, weigh all tokens alike."""
    for q_exp, k_exp, scale in ((60, 60, 2.0 ** -123), (60, 60, -3e-37), (60, 60, 2.0 ** -119), (30, 70, 0.11 * 2.0 ** -100),
                                (70, 33, 0.5 * 2.0 ** -103), (50, 50, 0.68 * 2.0 ** -100), (50, 50, 0.70 * 2.0 ** -100),
                                (50, 50, 1e-31), (60, 60, 0.0), (60, 60, -0.0), (60, 60, 1e-45), (60, 60, -5e-324), (60, 60, 1e-300)):
        _small_scale(q_exp, k_exp, scale, q_dt, codes, lens)


@pytest.mark.parametrize("D,page", [(128, 7), (128, 16), (80, 16), (256, 32), (256, 5)])
def test_small_scales_of_every_width(D, page):
    for q_dt in ("bf16", "f32"):
        for codes in (True, False):
            for scale in (0.0, 2.0 ** -123):
                _small_scale(60, 59, scale, q_dt, codes, [200, 33], page, D)


def test_nan_meets_a_scale_of_zero():
    t = torch()
    cache, _ = new_cache("head_major", 4, 16, 1, 64, False)
    for dt in (t.bfloat16, t.float32):
        q = t.randn(1, 4, 64, device=device()).to(dt)
        q[0, 2, 7] = float("nan")
        banner(f"paged_attention NaN at scale 0 {dt}")
        out = B.paged_attention(q, cache, t.arange(4, dtype=t.int32, device=device())[None],
                                t.tensor([50], dtype=t.int32, device=device()), scale=0.0)
        assert bool(out[0, 2].isnan().all()) and bool(out[0, [0, 1, 3]].isfinite().all())


@pytest.mark.parametrize("q_dt", ["bf16", "f32"])
@pytest.mark.parametrize("layout", ["token_major", "side_by_side", "padded"])
@pytest.mark.parametrize("D", [64, 128, 144, 256])
def test_layouts_of_codes(D, layout, q_dt):
    """Pages of whole halves whose scales lie apart (token-major) or next to each other, in one scale group and in two."""
    for page in (16, 48):
        _run([5, 700, 1, 130, 0, 64], 8, 2, D, page, True, layout=layout, q_dt=q_dt)
    _run([3000, 17], 8, 2, D, 16, True, layout=layout, q_dt=q_dt, window=2500)


@pytest.mark.parametrize("n", [310, 4000])
@pytest.mark.parametrize("codes", [True, False])
@pytest.mark.parametrize("q_dt", ["bf16", "f32"])
def test_a_maximum_that_rises_late(n, codes, q_dt):
    """Logits that rise along the sequence for one head, so that every tile rescales what was before it, and fall for the other."""
    t = torch()
    pages = n // 16 + 1
    cache, _ = new_cache("head_major", pages, 16, 1, 64, codes)
    cache.k.zero_()
    ramp = t.arange(pages * 16, device=device(), dtype=t.float32).view(pages, 16, 1)
    if codes:
        cache.v_scale.mul_(0.01)
        cache.k[..., 0] = 0x38                            # the code of 1
        cache.k_scale.copy_(ramp[..., None])
    else:
        cache.k[..., 0] = ramp.bfloat16()
    q = t.zeros(1, 2, 64, device=device())
    q[0, 0, 0], q[0, 1, 0] = 1.0, -1.0
    q = q.bfloat16() if q_dt == "bf16" else q
    table = np.random.default_rng(n).permutation(pages).astype(np.int32)[None]
    if n > 1000:   # along the sequence, not along the pages
        table = np.arange(pages, dtype=np.int32)[None]
    banner(f"paged_attention ramp n={n} codes={codes} {q_dt}")
    out, lse = B.paged_attention(q, cache, t.from_numpy(table).to(device()), t.tensor([n], dtype=t.int32, device=device()), scale=0.5,
                                 lse=True)
    _check(out, lse, q, cache, cache_values(cache), table, [n], 0, 0.5)
