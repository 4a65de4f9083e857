"""The precision of paged_attention: F32 queries in three BF16 terms, softmax weights in three where queries or outputs are F32
and in two otherwise.  test_attention_terms_host.py shows that these tolerances see a term that is lost."""
import numpy as np
import pytest

import attention_terms as A
import block_scaled_fp8_linear_amd as B
from cache_util import attention64, cache_values, make_table, new_cache, to_f64
from gpu_util import banner, device, torch

pytestmark = pytest.mark.gpu


def _one_hot(lens, D, page, kv, codes, at):
    """A cache of one-hot keys and values: each sequence's token at position at[i] has channel i, the others the last one."""
    t = torch()
    g = np.random.default_rng(D + page)
    pages = sum(-(-n // page) for n in lens) + 1
    cache, _ = new_cache("head_major", pages, page, kv, D, codes, fill=0)
    table = make_table(g, lens, page, pages)
    for x in (cache.k_scale, cache.v_scale):
        if x is not None:
            x.fill_(1.0)
    one = 0x38 if codes else 1.0
    for b, n in enumerate(lens):
        channel = np.full(n, D - 1)
        channel[at] = np.arange(len(at))
        pos = np.arange(n)
        pg, row = t.from_numpy(table[b, pos // page]).long().to(device()), t.from_numpy(pos % page).to(device())
        for x in (cache.k, cache.v):
            x[pg, row, :, t.from_numpy(channel).to(device())] = one
    return cache, table


@pytest.mark.parametrize("q_dt,out_dt", [("f32", "f32"), ("f32", "bf16"), ("bf16", "f32"), ("bf16", "bf16")])
@pytest.mark.parametrize("codes", [True, False])
@pytest.mark.parametrize("D,page", [(64, 16), (128, 16), (128, 7), (80, 32), (256, 16), (256, 24)])
@pytest.mark.parametrize("split", [False, True])
def test_terms(q_dt, out_dt, codes, D, page, split):
    """One wave holds all tokens that count, or they lie in many blocks."""
    t = torch()
    g = np.random.default_rng(D + split)
    kv, heads = 2, 32
    lens = [9000, 7001] if split else [A.TOKENS + 9 + i for i in range(6)]
    at = sorted(g.choice(7000, A.TOKENS, replace=False)) if split else list(range(A.TOKENS))
    cache, table = _one_hot(lens, D, page, kv, codes, at)
    q = A.queries(g, len(lens), heads, D, q_dt == "f32")
    dt = {"bf16": t.bfloat16, "f32": t.float32}
    banner(f"paged_attention terms {q_dt}->{out_dt} codes={codes} D={D} page={page} split={split}")
    out, lse = B.paged_attention(t.from_numpy(q).to(device()).to(dt[q_dt]), cache, t.from_numpy(table).to(device()),
                                 t.tensor(lens, dtype=t.int32, device=device()), scale=1.0, lse=True, out_dtype=dt[out_dt])
    want, wl = A.exact(q)
    got = to_f64(out)
    assert A.within(got, want, out_dt == "bf16", 2 if q_dt == out_dt == "bf16" else 3, split), \
        float(np.abs(got / np.where(want > 0, want, 1) - (want > 0)).max())
    # the log of a sum of at most n, 2 ulp, and the result's rounding
    assert (np.abs(to_f64(lse) - wl) <= A.tolerance(split) + 4 * A.U * np.log(A.TOKENS) + A.U * np.abs(wl)).all()


@pytest.mark.parametrize("codes", [True, False])
@pytest.mark.parametrize("D,lens,window", [(256, [5000, 700, 3, 1200, 31, 4000, 2500], 2048), (128, [6000, 40, 900], 0), (64, [3000, 129], 0)])
def test_norm_of_the_error(codes, D, lens, window):
    """Ordinary values: the error of a batch with F32 queries and outputs against its norm."""
    t = torch()
    g = np.random.default_rng(D)
    kv, heads, page = 2, 12, 24
    pages = sum(-(-n // page) for n in lens) + 1
    cache, _ = new_cache("head_major", pages, page, kv, D, codes)
    if codes:   # codes up to 448, most of them small: values up to some 4
        cache.k_scale.fill_(0.01), cache.v_scale.fill_(0.01)
    else:
        cache.k.normal_(), cache.v.normal_()
    table = make_table(g, lens, page, pages)
    q = t.from_numpy((2.0 * g.standard_normal((len(lens), heads, D))).astype(np.float32)).to(device())
    banner(f"paged_attention norm of the error codes={codes} D={D}")
    out = B.paged_attention(q, cache, t.from_numpy(table).to(device()), t.tensor(lens, dtype=t.int32, device=device()), window=window)
    values = cache_values(cache)
    want = attention64(to_f64(q), values, table, lens, page, window, D ** -0.5, pages)[0]
    # logits of a row: normal, of the deviation below; 5 of them are beyond none of some 10^5
    largest = 5 * 2.0 * np.sqrt((values[0] ** 2).mean())
    assert np.linalg.norm(to_f64(out) - want) <= A.norm_bound(D, largest) * np.linalg.norm(want)
