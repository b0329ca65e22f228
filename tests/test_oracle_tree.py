"""The 64-bit oracle of the tree operators against independent forms: a chain is causal
attention, filters against brute force over prefixes, the draw against frequencies, and
page bookkeeping against its own invariants.  CPU only."""
import itertools

import numpy as np
import pytest

from oracle import serving as osv
from oracle import tree as otr


def test_a_chain_is_causal_attention_and_a_star_sees_its_root():
    rng = np.random.default_rng(1)
    kc, vc = rng.normal(size=(2, 5, 4, 2, 8))
    table, kv, off = [[3, 1, 4, 0]], [13], [0, 6]
    q = rng.normal(size=(6, 4, 8))
    a = otr.attn_tree(q, kc, vc, table, kv, off, [-1, 0, 1, 2, 3, 4])
    b = osv.attn_paged(q, kc, vc, table, kv, off, True)
    for x, y in zip(a, b):
        np.testing.assert_allclose(x, y, rtol=1e-13)
    assert [otr.ancestors([-1, 0, 0, 1, 9, -7], i) for i in range(6)] == [[0], [1, 0], [2, 0], [3, 1, 0], [4], [5]]


@pytest.mark.parametrize("top_k,top_p,min_p", [(0, 1.0, 0.0), (3, 1.0, 0.0), (0, 0.6, 0.0), (4, 0.7, 0.2), (0, 0.0, 0.0),
                                               (0, 1.0, 1.0), (1, 1.0, 0.0)])
def test_distribution_is_the_only_set_that_meets_the_definition(top_k, top_p, min_p):
    rng = np.random.default_rng(2)
    for _ in range(20):
        x = np.round(rng.normal(size=7) * 2) / 2  # ties
        w = otr.distribution(x, 0.7, top_k, top_p, min_p)
        e = np.exp((x - x.max()) / 0.7)
        order = np.lexsort((np.arange(7), -x))
        k = order[:top_k] if top_k else order
        fits = [n for n in range(1, len(k) + 1) if top_p >= 1 and n == len(k)
                or top_p < 1 and e[k[:n]].sum() >= top_p * e[k].sum() - 1e-12]
        kept = [i for i in k[:min(fits)] if e[i] >= min_p]
        np.testing.assert_allclose(w, np.where(np.isin(np.arange(7), kept), e, 0))


def test_a_share_that_is_met_exactly():
    """Half of two equal weights is one of them, but less than half where anything follows, however little."""
    kept = lambda x, **s: np.flatnonzero(otr.distribution(x, 1.0, top_p=0.5, **s)).tolist()  # noqa: E731
    assert kept([0.0, 3.0, 3.0]) == [1, 2] and kept([3.0, -np.inf, 3.0]) == [0]
    for less in (40.0, 700.0, 2000.0):  # e^-40 is lost in a sum of 64 bits, e^-2000 by itself
        assert kept([3.0, 3.0, 3.0 - less]) == [0, 1] and kept([3.0, 3.0, 3.0 - less], top_k=2) == [0]


def test_sample_has_the_distribution():
    w = otr.distribution([1.0, -np.inf, 2.0, 0.5, np.nan], 1.0)
    assert w[1] == w[4] == 0
    u = (np.arange(4000) + 0.5) / 4000
    got = np.bincount([otr.sample(w, x) for x in u], minlength=5) / 4000
    np.testing.assert_allclose(got, w / w.sum(), atol=1e-3)
    assert otr.sample(np.zeros(3), 0.5) == 0 and not otr.distribution([-np.inf] * 3).any()


def test_accept_and_compact_on_a_tree_by_hand():
    parents, tokens = [-1, 0, 0, 1, 2, 2, 5], [9, 5, 7, 1, 3, 4, 8]
    sampled = [7, 0, 4, 0, 0, 8, 2]
    path, out, count = otr.accept(sampled, tokens, parents, [0, 7, 7], 5)
    assert path.tolist() == [[0, 2, 5, 6, -1], [-1] * 5] and out[0].tolist() == [7, 4, 8, 2, -1]
    assert count.tolist() == [4, 0]
    cache = np.arange(4 * 4).reshape(4, 4, 1, 1).astype(float)
    got, new = otr.compact(cache, [[2, 0, 3], [1, 1, 1]], [10, 2], [0, 7, 7], path, count)
    assert new == [7, 2]
    flat = np.concatenate([got[p].ravel() for p in (2, 0, 3)])
    was = np.concatenate([cache[p].ravel() for p in (2, 0, 3)])
    np.testing.assert_array_equal(flat, [*was[:3], was[3], was[5], was[8], was[9], *was[7:]])


def test_pages_keep_count():
    rng = np.random.default_rng(3)
    P, R = 4, 6
    table, refs, lens = np.full((R, 5), -1), np.zeros(12, int), [0] * R
    for step in range(60):
        new = [int(rng.integers(0, 12)) if rng.random() < 0.5 else n for n in lens]
        table, refs, missing = otr.resize(table, lens, new, refs, P)
        lens = new
        if missing:
            table, refs, _ = otr.resize(table, lens, [0] * R, refs, P)
            lens = [0] * R
        held = [g for row, n in zip(table, lens) for g in row[:-(-n // P)]]
        assert np.array_equal(np.bincount(held, minlength=12), refs) if held else not refs.any()
        assert all((row[-(-n // P):] == -1).all() for row, n in zip(table, lens))
    empty = [r for r in range(R) if lens[r] == 0][:1]
    full = [r for r in range(R) if lens[r]][:1]
    for a, b in itertools.product(full, empty):
        t, l, c, s, d, n, missing = otr.fork(table, lens, [a], [b], refs, P)
        assert l[b] == lens[a] and n[0] == lens[a] % P
        held = [g for row, m in zip(t, l) for g in row[:-(-m // P)] if g >= 0]
        assert np.array_equal(np.bincount(held, minlength=12), c)
