"""Pins of the serving oracle: closed forms, library routines and planted mistakes (CPU only)."""
import numpy as np
import pytest
from scipy import special

from oracle import serving_oracle as SO

rng = np.random.default_rng(5)


def paged(tokens, size, pages, table):
    """A pool [pages][1][size][dim] holding tokens [n][dim] by the table row."""
    pool = np.full((pages, 1, size, tokens.shape[1]), np.nan)
    for t, x in enumerate(tokens):
        pool[table[t // size], 0, t % size] = x
    return pool


def attend_case():
    k, v, q = rng.normal(size=(7, 4)), rng.normal(size=(7, 4)), rng.normal(size=(1, 2, 4))
    table = np.array([[2, 0, 3]])
    return k, v, q, paged(k, 3, 4, table[0]), paged(v, 3, 4, table[0]), table


def check_attend(attend):
    k, v, q, pk, pv, table = attend_case()
    got = attend(q, pk, pv, table, [7], 0.5)[0]
    s = 0.5 * q[0] @ k.T
    assert np.allclose(got["out"], special.softmax(s, axis=1) @ v)
    assert np.allclose(got["lse"], special.logsumexp(s, axis=1))
    assert np.allclose(got["drawn"].sum(), 2)


def test_attend_against_library_softmax():
    check_attend(SO.attend)


@pytest.mark.parametrize("wrong", [
    lambda q, k, v, t, n, s: SO.attend(q, k, v, t, n, s * s),                  # scale twice
    lambda q, k, v, t, n, s: SO.attend(q, k, v, t, [n[0] - 1], s),            # the new token left out
    lambda q, k, v, t, n, s: SO.attend(q, k, v, t[:, ::-1], n, s),            # pages in the wrong order
    lambda q, k, v, t, n, s: SO.attend(q[:, ::-1], k, v, t, n, s),            # heads swapped
])
def test_planted_attend_mistakes_are_seen(wrong):
    with pytest.raises((AssertionError, IndexError)):
        check_attend(wrong)


def test_attend_special_rows():
    z = np.zeros((1, 1, 4, 2))
    table = np.array([[0]])
    one = SO.attend(np.ones((1, 1, 2)), z, z + 3.0, table, [1], 1.0)[0]
    assert np.allclose(one["out"], 3.0) and one["lse"][0] == 0.0          # one token: its value
    none = SO.attend(np.ones((1, 1, 2)), z, z, table, [0], 1.0)[0]
    assert np.all(none["out"] == 0) and np.isneginf(none["lse"][0])
    masked = SO.attend(np.ones((1, 1, 2)), z - np.inf, z + 1, table, [4], 1.0)[0]
    assert np.all(masked["out"] == 0) and np.isneginf(masked["lse"][0])


def test_append_places_tokens():
    pool = np.zeros((3, 1, 2, 1))
    table = np.array([[2, 0], [1, -1]])
    k, _ = SO.append(pool, pool, table, np.array([[[7.0]], [[8.0]], [[9.0]]]), np.zeros((3, 1, 1)), [0, 0, 1], [1, 2, 0])
    assert k[2, 0, 1, 0] == 7 and k[0, 0, 0, 0] == 8 and k[1, 0, 0, 0] == 9 and k.sum() == 24


@pytest.mark.parametrize("weight,pos,seen,budget,sink,recent,want", [
    ([5, 1, 4, 2, 3], [0, 1, 2, 3, 4], 5, 3, 0, 0, [0, 2, 4]),               # by weight
    ([1, 1, 1, 1], [0, 1, 2, 3], 4, 2, 0, 0, [0, 1]),                        # ties: the lower index
    ([0, 9, 9, 0, 0], [0, 1, 2, 3, 4], 5, 3, 1, 1, [0, 1, 4]),               # first and last stay
    ([9, 0, 0, 9], [9, 3, 8, 2], 10, 2, 0, 2, [0, 2]),                       # recent by position, not by place
    ([np.nan, -np.inf, -1], [0, 1, 2], 3, 2, 0, 0, [1, 2]),                  # NaN last
    ([0.0, -0.0, 0.0], [0, 1, 2], 3, 2, 0, 0, [0, 1]),                       # -0 equals 0
])
def test_kept_tokens(weight, pos, seen, budget, sink, recent, want):
    assert SO.kept_tokens(np.array(weight, float), np.array(pos), seen, budget, sink, recent) == want


def test_evict_fills_holes_in_order():
    w = np.array([[[1.0, 9, 2, 8, 7, 6]]])
    pos = np.arange(6).reshape(1, 1, 6)
    toks = np.arange(6.0).reshape(6, 1)
    pool = paged(toks, 2, 3, [0, 1, 2])
    k, v, w2, p2, lens = SO.evict(pool, pool + 10, np.array([[0, 1, 2]]), [6], w, pos, [6], 4, 0, 0)
    assert lens == [4] and p2[0, 0, :4].tolist() == [4, 1, 5, 3] and w2[0, 0, :4].tolist() == [7, 9, 6, 8]
    assert SO.cached(k, [0, 1, 2], 0, 4)[:, 0].tolist() == [4, 1, 5, 3]
    assert SO.cached(v, [0, 1, 2], 0, 4)[:, 0].tolist() == [14, 11, 15, 13]


def test_logprobs_against_library():
    x = rng.normal(size=(3, 50)) * 4
    lp, h, idx, val, _ = SO.token_logprobs(x, [4, -1, 7], 5)
    want = special.log_softmax(x, axis=1)
    assert np.allclose(lp, [want[0, 4], 0, want[2, 7]])
    assert np.allclose(h, special.entr(np.exp(want)).sum(axis=1))
    assert np.array_equal(idx, np.argsort(-x, axis=1)[:, :5]) and np.allclose(val, np.take_along_axis(want, idx, 1))


def test_logprobs_special_rows():
    x = np.array([[-np.inf, 0.0, 0.0, -np.inf], [np.nan, 1, 2, 3], [-np.inf] * 4, [np.inf, 1, 2, 3], [0.0, -0.0, 1, 1]])
    lp, h, idx, val, _ = SO.token_logprobs(x, [1, 1, 1, 1, 2], 4)
    assert np.isclose(lp[0], -np.log(2)) and np.isclose(h[0], np.log(2)) and np.isneginf(val[0, 2])
    assert np.isnan(lp[1:4]).all() and np.isnan(h[1:4]).all()
    assert idx.tolist() == [[1, 2, 0, 3], [3, 2, 1, 0], [0, 1, 2, 3], [0, 3, 2, 1], [2, 3, 0, 1]]
