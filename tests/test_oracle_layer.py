"""The references of oracle/layer.py on cases small enough to work out by hand."""

import math

import numpy as np

from oracle import codecs, layer


def _bits(x):
    return layer.bf16_bits(np.array([x]))[0]


def test_bf16_rounding():
    assert _bits(1.0) == 0x3F80 and _bits(-2.0) == 0xC000
    assert _bits(1.0 + 2.0 ** -8) == 0x3F80 and _bits(1.0 + 3 * 2.0 ** -8) == 0x3F82  # ties to even
    assert _bits(1.0 + 2.0 ** -8 + 2.0 ** -20) == 0x3F81
    assert _bits(1e39) == 0x7F80 and _bits(float("nan")) == 0x7FC0


def test_norms_by_hand():
    y = layer.norm_rows([[3.0, 4.0]], False, 0.0)
    np.testing.assert_allclose(y, [[3 / math.sqrt(12.5), 4 / math.sqrt(12.5)]], rtol=1e-15)
    y = layer.norm_rows([[1.0, 3.0]], True, 0.0, [2.0, 1.0], [0.5, 0.0], 1.0)
    np.testing.assert_allclose(y, [[-3.0 + 0.5, 2.0]], rtol=1e-15)


def test_residual_is_rounded_before_its_norm():
    s, bits = layer.norm([[2.0 ** -9, 1.0]], [[1.0, 1.0]], eps=0.0)
    assert s.tolist() == [[1.0, 2.0]]
    np.testing.assert_array_equal(bits, layer.bf16_bits([[1 / math.sqrt(2.5), 2 / math.sqrt(2.5)]]))
    s, _ = layer.norm([[2.0 ** -9, 1.0]], [[1.0, 1.0]], gate=[[2.0, -1.0]], residual_scale=0.5, r_f32=True)
    assert s.tolist() == [[0.5 + 2.0 ** -8, -0.5]]


def test_gated_by_hand():
    y = codecs.bf16_bits_to_f64(layer.gated_act([[0.0, 1.0, -800.0, 5.0, 2.0, 3.0]]))
    assert y[0, 0] == 0.0 and y[0, 2] == 0.0
    assert abs(y[0, 1] - 2.0 / (1 + math.exp(-1.0))) <= 2.0 ** -8
    y = codecs.bf16_bits_to_f64(layer.gated_act([[1.0, 4.0]], "gelu"))
    assert abs(y[0, 0] - 2.0 * (1 + math.tanh(math.sqrt(2 / math.pi) * 1.044715))) <= 2.0 ** -6


def test_lora_by_hand():
    a = np.zeros((2, 2, 2, 3))
    a[1, 0, 0] = [1, 2, 3]
    a[1, 1, 0] = [0, 0, 1]
    a[1, :, 1] = 100.0  # behind the rank
    b = np.ones((2, 4, 2))
    y, err = layer.lora(np.ones((3, 4)), [[1, 1, 1], [2, 0, 1], [5, 5, 5]], [1, 1, -1], a, b, [3, 4], ranks=[2, 1],
                        scales=[1.0, 0.5])
    assert y.tolist() == [[4, 4, 4, 1.5], [3.5, 3.5, 3.5, 1.5], [1, 1, 1, 1]]
    assert (err[2] == 0).all() and (err[:2] > 0).all() and err.max() < 1e-3
