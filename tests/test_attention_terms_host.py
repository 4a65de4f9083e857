"""The tolerances of test_gpu_attention_terms.py see a lost term: the kernel's arithmetic with all terms is within them, with
one term less of a query or of a weight it is not (CPU only)."""
import numpy as np
import pytest

import attention_terms as A


def test_terms():
    x = np.random.default_rng(1).standard_normal(10000).astype(np.float32)
    assert np.array_equal(A.in_terms(x, 3), x)
    assert np.abs(A.in_terms(x, 2) / x - 1).max() <= 2.0 ** -17 < np.abs(A.in_terms(x, 1) / x - 1).max() <= 2.0 ** -8


@pytest.mark.parametrize("split", [False, True])
def test_a_lost_term_shows(split):
    g = np.random.default_rng(2)
    q = A.queries(g, 8, 64, 64, True)
    want, _ = A.exact(q)
    assert A.within(A.emulate(q, 3, 3), want, False, 3, split)
    for terms in ((2, 3), (1, 3), (3, 2), (3, 1)):
        assert not A.within(A.emulate(q, *terms), want, False, 3, split), terms
    q = A.queries(g, 8, 64, 64, False)
    want, _ = A.exact(q)
    assert A.within(A.emulate(q, 1, 3), want, False, 3, split)       # BF16 queries, F32 outputs
    assert not A.within(A.emulate(q, 1, 2), want, False, 3, split)
    assert A.within(A.bf16(A.emulate(q, 1, 2)), want, True, 2, split)
    assert not A.within(A.bf16(A.emulate(q, 1, 1)), want, True, 2, split)


def test_the_norm_of_a_batch_shows_a_second_term():
    """The bound of test_norm_of_the_error against logits and weights that keep one term."""
    g = np.random.default_rng(3)
    D, n = 256, 2000
    q = (2.0 * g.standard_normal((4, D))).astype(np.float32)
    k, v = A.bf16(g.standard_normal((n, D)).astype(np.float32)).astype(np.float64), A.bf16(g.standard_normal((n, D)).astype(np.float32)).astype(np.float64)

    def attention(q, terms):
        s = q.astype(np.float64) @ k.T / D ** 0.5
        p = np.exp(s - s.max(-1, keepdims=True))
        return A.in_terms(p.astype(np.float32), terms).astype(np.float64) @ v / p.sum(-1, keepdims=True)

    want, bound = attention(q, 3), A.norm_bound(D, np.abs(q.astype(np.float64) @ k.T / D ** 0.5).max())
    for other in (attention(A.in_terms(q, 1), 3), attention(q, 1)):
        assert np.linalg.norm(other - want) > 100 * bound * np.linalg.norm(want)
