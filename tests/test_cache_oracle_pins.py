"""The oracles of the cache and beam operators against closed forms worked by hand, and the kernels' page arithmetic."""

import math

import numpy as np
import pytest

from oracle import cache_oracle as co


def test_places_of_packed_tokens():
    table = [[4, 7], [1, -1]]
    got = co.places(table, [18, 20], 16, 8, cu_seqlens=[0, 3, 5])
    assert got == [(0, 0, 15, 4, 15), (1, 0, 16, 7, 0), (2, 0, 17, 7, 1), (3, 1, 18, -1, 2), (4, 1, 19, -1, 3)]


def test_places_before_and_behind_the_table():
    assert [g[2:4] for g in co.places([[0]], [1], 16, 1, tokens=3)] == [(-2, -1), (-1, -1), (0, 0)]
    assert [g[3] for g in co.places([[0]], [18], 16, 1, tokens=3)] == [0, -1, -1]


@pytest.mark.parametrize("interleaved", [False, True])
def test_quarter_turn(interleaved):
    x = np.arange(1.0, 7.0)
    y, size = co.rotate(x, np.array([math.pi / 2, math.pi]), 4, interleaved)
    want = [-2, 1, -3, -4, 5, 6] if interleaved else [-3, -2, 1, -4, 5, 6]
    assert np.allclose(y, want, atol=1e-15)
    assert size.tolist() == ([3, 3, 7, 7, 5, 6] if interleaved else [4, 6, 4, 6, 5, 6])


def test_rotated_products_depend_on_the_distance():
    rng = np.random.default_rng(0)
    q, k, f = rng.standard_normal(8), rng.standard_normal(8), rng.random(4)
    dot = [co.rotate(q, (5 + n) * f, 8, False)[0] @ co.rotate(k, n * f, 8, False)[0] for n in (0, 3, 1000)]
    assert np.allclose(dot, dot[0], atol=1e-11)


def cache(keys, values, page=16):
    pages = -(-len(keys) // page)
    kc, vc = np.zeros((pages, 1, page, len(keys[0]))), np.zeros((pages, 1, page, len(keys[0])))
    for j, (k, v) in enumerate(zip(keys, values)):
        kc[j // page, 0, j % page], vc[j // page, 0, j % page] = k, v
    return kc, vc, np.arange(pages)[None]


def test_attention_of_equal_keys_is_the_mean():
    values = [[float(j), -float(j)] for j in range(20)]
    kc, vc, table = cache([[1.0, 2.0]] * 20, values)
    q = np.ones((3, 2, 2))
    o = co.attention(q, kc, vc, table, [20], 0.7)["o"]
    assert np.allclose(o[:, 0, 0], [8.5, 9.0, 9.5])
    o = co.attention(q, kc, vc, table, [20], 0.7, window=2)["o"]
    assert np.allclose(o[:, 1, 1], [-16.5, -17.5, -18.5])


def test_attention_of_two_keys():
    kc, vc, table = cache([[0.0, 0.0], [math.log(3.0), 0.0]], [[1.0, 0.0], [0.0, 1.0]])
    o = co.attention(np.array([[[1.0, 5.0]]]), kc, vc, table, [2], 1.0)["o"]
    assert np.allclose(o[0, 0], [0.25, 0.75])


def test_attention_without_keys_is_zero():
    kc, vc, table = cache([[1.0]], [[1.0]])
    assert not co.attention(np.ones((2, 1, 1)), kc, vc, table, [0], 1.0)["o"].any()
    assert not co.attention(np.ones((1, 1, 1)), kc, vc, [[-1]], [1], 1.0)["o"].any()
    assert not co.attention(np.ones((1, 1, 1)), kc, vc, [[9]], [1], 1.0)["o"].any()


def test_beams_by_hand():
    x = np.log([[[0.5, 0.25, 0.25], [0.1, 0.8, 0.1]]])
    tokens, parents, best, over = co.beam_select(x, [[math.log(0.4), math.log(0.6)]], 4, eos=1)
    # 0.48 (1, 1), 0.2 (0, 0), 0.1 (0, 1), 0.1 (0, 2)
    assert tokens.tolist() == [[1, 0, 1, 2]] and parents.tolist() == [[1, 0, 0, 0]]
    assert np.allclose(np.exp(best), [[0.48, 0.2, 0.1, 0.1]]) and over.tolist() == [[True, False, True, False]]


def test_finished_beams_go_on_with_the_pad_token():
    x = np.log([[[0.5, 0.5], [0.9, 0.1]]])
    tokens, parents, best, over = co.beam_select(x, [[-1.0, -1.2]], 3, finished=[[True, False]], pad=1)
    assert tokens.tolist() == [[1, 0, 1]] and parents.tolist() == [[0, 1, 1]]
    assert np.allclose(best, [[-1.0, -1.2 + math.log(0.9), -1.2 + math.log(0.1)]]) and over.tolist() == [[True, False, False]]


def test_absent_beams():
    inf = math.inf
    x = np.array([[[0.0, 0.0], [math.nan, 0.0], [inf, 0.0], [-inf, -inf], [0.0, -inf]]])
    tokens, parents, best, over = co.beam_select(x, [[-inf, 0.0, 0.0, 0.0, -2.0]], 2)
    assert tokens.tolist() == [[0, -1]] and parents.tolist() == [[4, -1]]
    assert best.tolist() == [[-2.0, -inf]] and over.tolist() == [[False, True]]


def test_reorder_by_hand():
    got = co.reorder(np.arange(6), [[2, -1, 0], [1, 1, 3]])
    assert got == [2, None, 0, 4, 4, None]


@pytest.mark.parametrize("granules", range(1, 65))
def test_page_of_a_granule_by_multiplication(granules):
    """page = g * ceil(2^32 / n) >> 32 is g // n for every granule of the longest table (2^26 keys) and the 64 behind."""
    magic = ((1 << 32) + granules - 1) // granules
    g = np.arange((1 << 22) + 64, dtype=np.uint64)
    assert np.array_equal((g * np.uint64(magic)) >> np.uint64(32), g // np.uint64(granules))
