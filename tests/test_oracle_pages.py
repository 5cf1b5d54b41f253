"""CPU pins of the page-selection oracle."""
import math

import numpy as np
import pytest
import torch

from oracle import mla_oracle as O
from oracle import page_select as PS


def test_page_keys_are_means_of_the_rows_a_page_has():
    rows = np.random.default_rng(0).standard_normal((130, 5))
    keys = PS.page_keys(rows)
    assert keys.shape == (3, 5)
    np.testing.assert_allclose(keys[1], rows[64:128].sum(0) / 64, atol=1e-14)
    np.testing.assert_allclose(keys[2], (rows[128] + rows[129]) / 2, atol=1e-15)


def test_page_scores_are_softmax_masses():
    g = np.random.default_rng(1)
    q, keys = g.standard_normal((6, 9)), g.standard_normal((17, 9))
    s = PS.page_scores(q, keys, 0.7)
    ref = torch.softmax(torch.from_numpy(0.7 * q @ keys.T), -1).sum(0).numpy()
    np.testing.assert_allclose(s, ref, rtol=1e-13)
    assert abs(s.sum() - 6) < 1e-12


def test_select_orders_forced_pages_ties_and_nans():
    nan, inf = math.nan, math.inf
    assert PS.select([1., 3., 3., 2.], 2, 0, 0) == [1, 2]
    assert PS.select([3., 3., 3., 3.], 2, 0, 0) == [0, 1]
    assert PS.select([0., 3., 3., 0.], 2, 1, 1) == [0, 3]
    assert PS.select([nan, -inf, -5., nan], 3, 0, 0) == [0, 1, 2]
    assert PS.select([5.], 4, 2, 3) == [0]
    assert PS.select([1., inf, 2., 0.], 2, 0, 1) == [1, 3]


def test_sparse_decode_of_every_page_is_the_dense_decode():
    g = np.random.default_rng(2)
    L, d_c, d_r = 150, 8, 4
    c, kr, q = g.standard_normal((L, d_c)), g.standard_normal((L, d_r)), g.standard_normal((3, d_c + d_r))
    o, l = PS.sparse_decode(q, c, kr, [0, 1, 2], L, 0.4)
    ro, rl = O.absorbed_decode(q[None], c, kr, L, 0.4)
    np.testing.assert_allclose(o, ro[0], atol=1e-13)
    np.testing.assert_allclose(l, rl[0], atol=1e-13)
    # two pages: softmax over just those rows, the last page cut at the visible positions
    o, l = PS.sparse_decode(q, c, kr, [0, 2], 140, 0.4)
    idx = np.r_[0:64, 128:140]
    u = 0.4 * q @ np.concatenate([c, kr], 1)[idx].T
    w = np.exp(u) / np.exp(u).sum(1, keepdims=True)
    np.testing.assert_allclose(o, w @ c[idx], atol=1e-12)
    o, l = PS.sparse_decode(q, c, kr, [], 140, 0.4)
    assert not o.any() and np.all(l == -np.inf)


@pytest.mark.parametrize("L,s_q,want", [(1, 1, [1]), (64, 1, [1]), (65, 1, [2]), (65, 2, [1, 2]), (1, 2, [0, 1])])
def test_visible_pages(L, s_q, want):
    assert [PS.visible_pages(L, s_q, t) for t in range(s_q)] == want
