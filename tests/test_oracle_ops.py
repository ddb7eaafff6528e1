"""The references of oracle/ops.py on cases small enough to work out by hand."""

import math

import numpy as np

from oracle import ops


def test_route_softmax_ties_and_weights():
    ids, w, bad = ops.route([[1.0, 3.0, 3.0, 2.0]], 3)
    assert ids.tolist() == [[1, 2, 3]] and not bad
    e = [math.exp(v) for v in (1, 3, 3, 2)]
    np.testing.assert_allclose(w[0], [e[1] / sum(e), e[2] / sum(e), e[3] / sum(e)], rtol=1e-15)
    _, w, _ = ops.route([[1.0, 3.0, 3.0, 2.0]], 3, renorm=True, scale=2.0)
    np.testing.assert_allclose(w.sum(), 2.0, rtol=1e-15)


def test_route_bias_moves_the_choice_not_the_weight():
    ids, w, _ = ops.route([[0.0, 1.0]], 1, score="sigmoid", bias=[1.0, 0.0])
    assert ids.tolist() == [[0]] and w[0, 0] == 0.5


def test_route_groups():
    # group 0 has the largest expert, group 1 the largest pair
    l = [[5.0, -9.0, 4.0, 4.0]]
    assert ops.route(l, 2, score="sigmoid", groups=2, topk_groups=1, group_score="max")[0].tolist() == [[0, 1]]
    assert ops.route(l, 2, score="sigmoid", groups=2, topk_groups=1, group_score="top2")[0].tolist() == [[2, 3]]


def test_route_masks():
    inf = math.inf
    ids, w, bad = ops.route([[-inf, 2.0, -inf, -inf], [-inf] * 4, [math.nan, inf, 0.0, 1.0]], 3, renorm=True)
    assert ids.tolist() == [[1, 0, 2], [0, 1, 2], [1, 3, 2]] and bad
    assert w.tolist() == [[1.0, 0.0, 0.0], [0.0, 0.0, 0.0], [1.0, 0.0, 0.0]]


def test_quantize_act_zp():
    codes, s, z = ops.quantize_act_zp([[0.0, 255.0, 51.0], [-1.0, 0.0, 0.0], [0.0, 0.0, 0.0], [math.inf, math.nan, 2.0]])
    assert codes[0].tolist() == [-128, 127, -77] and s[0] == 1.0 and z[0] == -128
    assert z[1] == 127 and codes[1].tolist() == [-128, 127, 127]
    assert codes[2].tolist() == [0, 0, 0] and s[2] == 1.0 and z[2] == 0
    assert codes[3].tolist() == [127, -128, 127] and z[3] == -128


def test_int_product_is_the_centred_product():
    rng = np.random.default_rng(0)
    a, b = rng.integers(-128, 128, (5, 33)), rng.integers(-128, 128, (7, 33))
    z = rng.integers(-128, 128, 5)
    want = [[sum((int(a[i, x]) - int(z[i])) * int(b[j, x]) for x in range(33)) for j in range(7)] for i in range(5)]
    assert ops.int_product(a, b, z).tolist() == want
