"""The oracle of the text model's attention and of its paged cache, pinned by values worked by hand, by properties and by
differences."""
import numpy as np
import pytest

from oracle import lm


def test_attention_by_hand():
    """Two keys, two queries: the first sees one key, the second both with weights 1/4 and 3/4."""
    q = np.array([[[1.0]], [[np.log(3.0)]]])
    k, v = np.array([[[0.0]], [[1.0]]]), np.array([[[4.0]], [[8.0]]])
    out, lse = lm.attention(q, k, v, 1.0, True)
    assert np.allclose(out.ravel(), [4.0, 7.0], atol=1e-14) and np.allclose(lse.ravel(), [0.0, np.log(4.0)], atol=1e-14)
    out, lse = lm.attention(q, k, v, 1.0, False)
    e = np.e
    assert np.allclose(out.ravel(), [(4 + 8 * e) / (1 + e), 7.0], atol=1e-14)
    assert np.allclose(lse.ravel(), [np.log1p(e), np.log(4.0)], atol=1e-14)


def test_queries_stand_at_the_end_of_their_sequence():
    assert lm.seen(2, 4, True).tolist() == [[True] * 3 + [False], [True] * 4]
    assert lm.seen(3, 1, True).tolist() == [[False], [False], [True]]
    assert lm.seen(2, 2, False).all() and lm.seen(0, 3, True).shape == (0, 3)


def test_masked_keys_do_not_enter_and_empty_rows_are_zeros():
    rng = np.random.default_rng(0)
    q, k, v = rng.standard_normal((3, 2, 4)), rng.standard_normal((3, 1, 4)), rng.standard_normal((3, 1, 4))
    out, lse = lm.attention(q, k, v, 0.5, True)
    k[2], v[2] = np.nan, np.inf
    again, sums = lm.attention(q, k, v, 0.5, True)
    assert (again[:2] == out[:2]).all() and (sums[:2] == lse[:2]).all()
    out, lse = lm.attention(q, k[:0], v[:0], 0.5, True)
    assert (out == 0).all() and np.isneginf(lse).all()


def test_shared_heads_are_copies():
    rng = np.random.default_rng(1)
    q, k, v = rng.standard_normal((5, 6, 8)), rng.standard_normal((7, 2, 8)), rng.standard_normal((7, 2, 8))
    a, la = lm.attention(q, k, v, 0.3, True)
    b, lb = lm.attention(q, np.repeat(k, 3, 1), np.repeat(v, 3, 1), 0.3, True)
    assert np.allclose(a, b, atol=1e-14) and np.allclose(la, lb, atol=1e-14)


@pytest.mark.parametrize("causal", [True, False])
def test_gradients_by_differences(causal):
    rng = np.random.default_rng(2)
    x = [rng.standard_normal(s) for s in ((4, 4, 3), (5, 2, 3), (5, 2, 3))]
    g = rng.standard_normal((4, 4, 3))
    out, lse = lm.attention(*x, 0.7, causal)
    grads = lm.attention_bwd(g, *x, out, lse, 0.7, causal)
    h = 1e-5
    for i, got in enumerate(grads):
        for at in np.ndindex(x[i].shape):
            d = []
            for sign in (1, -1):
                moved = [t.copy() for t in x]
                moved[i][at] += sign * h
                d.append((g * lm.attention(*moved, 0.7, causal)[0]).sum())
            # a central difference is off by h^2 / 6 of a third derivative and 2^-52 / h of the value
            assert abs((d[0] - d[1]) / (2 * h) - got[at]) < 1e-8


def test_block_tables_by_hand():
    """Pages of 4, a stack 7 8 9: request 0 ends and gives back 1 and 2, request 1 needs one page more, request 2 two."""
    tables = np.array([[1, 2, 0], [3, 0, 0], [0, 0, 0]])
    stack = np.array([7, 8, 9, 0, 0, 0, 0, 0, 0, 0])
    t, s, n, cu, pos, slots, missing = lm.block_tables([6, 4, 0], [0, 5, 6], tables, stack, 3, 4, 10)
    assert t[1].tolist() == [3, 2, 0] and t[2].tolist() == [1, 9, 0] and n == 2 and s[:3].tolist() == [7, 8, 9]
    assert cu.tolist() == [0, 0, 1, 7] and missing == (0, 0)
    assert pos[:7].tolist() == [4, 0, 1, 2, 3, 4, 5] and slots.tolist() == [8, 4, 5, 6, 7, 36, 37, -1, -1, -1]


def test_block_tables_keep_every_page_once():
    rng = np.random.default_rng(3)
    page, width, n_pages, batch = 8, 6, 40, 9
    tables, stack, n = np.full((batch, width), -1), rng.permutation(n_pages), n_pages
    before = np.zeros(batch, int)
    for _ in range(40):
        after = rng.integers(0, width * page + 1, batch)
        tables, stack, n, cu, pos, slots, missing = lm.block_tables(before, after, tables, stack, n, page, 1000)
        held = [tables[b, p] for b in range(batch) for p in range(-(-after[b] // page))]
        real = [p for p in held if p >= 0]
        assert sorted(real + stack[:n].tolist()) == list(range(n_pages)) and len(held) - len(real) >= missing[0]
        assert len(set(s for s in slots[:cu[-1]] if s >= 0)) == sum(s >= 0 for s in slots[:cu[-1]])
        # a request without all its pages ends, so that the next step starts from held ones
        before = np.array([0 if (tables[b, :-(-after[b] // page)] < 0).any() else after[b] for b in range(batch)])
        for b in range(batch):
            if before[b] == 0:
                tables, stack, n, *_ = lm.block_tables(np.eye(batch, dtype=int)[b] * after[b], np.zeros(batch, int), tables, stack, n, page, 0)
