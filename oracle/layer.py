"""References of the operators around the products -- norms with gate and
residual, gated activations, low-rank adapters -- in float64.

Test infrastructure (see the package docstring): plain definitions. Values are
rounded once to binary32 and from there to bf16, as the operators are defined;
codes follow from the bf16 bits by the quantizers of ``quant`` and ``ops``.
"""

import numpy as np

from . import codecs, ops, quant


def bf16_bits(x):
    """float64 -> binary32 -> bf16 bits, each rounding to nearest even."""
    with np.errstate(over="ignore", invalid="ignore"):
        f = np.asarray(x, np.float64).astype(np.float32)
    u = f.view(np.uint32).astype(np.uint64)
    r = ((u + 0x7FFF + ((u >> 16) & 1)) >> 16).astype(np.uint16)
    return np.where(np.isnan(f), np.uint16(0x7FC0), r).astype(np.uint16)


def rounded(x, f32):
    """The values of x in the type, as float64."""
    if f32:
        with np.errstate(over="ignore"):
            return np.asarray(x, np.float64).astype(np.float32).astype(np.float64)
    return codecs.bf16_bits_to_f64(bf16_bits(x))


def norm_rows(v, layer, eps, weight=None, bias=None, offset=0.0):
    v = np.asarray(v, np.float64)
    if layer:
        v = v - v.mean(axis=1, keepdims=True)
    y = v / np.sqrt((v * v).mean(axis=1, keepdims=True) + float(np.float32(eps)))
    if weight is not None:
        y = y * (np.asarray(weight, np.float64) + float(np.float32(offset)))
    if bias is not None:
        y = y + np.asarray(bias, np.float64)
    return y


def norm(x, residual=None, gate=None, post=None, weight=None, bias=None, layer=False, eps=1e-5, residual_scale=1.0,
         offset=0.0, r_f32=False):
    """(residual_out as float64, rows as bf16 bits); post: None or (weight, bias)."""
    t = np.asarray(x, np.float64)
    if post is not None:
        t = norm_rows(t, layer, eps, post[0], post[1], offset)
    if gate is not None:
        t = t * np.asarray(gate, np.float64)
    if residual is not None:
        t = t + float(np.float32(residual_scale)) * np.asarray(residual, np.float64)
    s = rounded(t, r_f32)
    return s, bf16_bits(norm_rows(s, layer, eps, weight, bias, offset))


def gated_act(y, act="silu"):
    """Rows as bf16 bits of act(gate) * up."""
    y = np.asarray(y, np.float64)
    n = y.shape[1] // 2
    g, u = y[:, :n], y[:, n:]
    z = g if act == "silu" else 2.0 * np.sqrt(2.0 / np.pi) * (g + 0.044715 * g ** 3)
    with np.errstate(over="ignore"):
        return bf16_bits(g / (1.0 + np.exp(-z)) * u)


def codes(bits, kind):
    """(codes as stored u8 or int8, scales, zeros or None) of bf16 rows."""
    if kind == "int8":
        qa, s = quant.quantize_act_int8(bits)
        return qa.astype(np.int8), s, None
    if kind == "int8_zp":
        return ops.quantize_act_zp(codecs.bf16_bits_to_f64(bits))
    if kind == "fp8":
        qa, s = quant.quantize_act_fp8(bits)
        return qa, s, None
    qa, s = quant.quantize_act_mxfp4(bits)
    return codecs.pack_nibbles(qa), s, None


def lora(y, x, ids, a, b, slice_ends, ranks=None, scales=None):
    """(Y64, the largest error of a binary32 evaluation before its rounding to Y's type).

    y, x real [M][n], [M][k]; a [E][S][R][k]; b [E][n][R]. With e = 2^-23 (one
    step, so that sums that cut instead of rounding are held too):
      T    products of bf16 numbers are exact; k of them added in blocks of 32
           and those in a chain: (k / 32 + 64) e of sum |x a|
      T'   scaled (2^-24) and held with all 24 bits: 2^-23 of it
      sum  2 R products in blocks of 32 and a chain: (R / 16 + 64) e of sum |T' b|
      Y    one addition, half a step: 2^-24 of |y| + |sum|."""
    y, x = np.asarray(y, np.float64).copy(), np.asarray(x, np.float64)
    err = np.zeros_like(y)
    e, k = 2.0 ** -23, x.shape[1]
    for ad in range(a.shape[0]):
        rows = np.nonzero(np.asarray(ids) == ad)[0]
        r = a.shape[2] if ranks is None else int(np.clip(ranks[ad], 0, a.shape[2]))
        s = 1.0 if scales is None else float(scales[ad])
        j0 = 0
        for i, j1 in enumerate(slice_ends):
            if rows.size and r:
                t = x[rows] @ a[ad, i, :r].T
                dt = (k / 32 + 64) * e * (np.abs(x[rows]) @ np.abs(a[ad, i, :r]).T)
                bb = b[ad, j0:j1, :r].T
                add = s * (t @ bb)
                size = abs(s) * (np.abs(t) @ np.abs(bb))
                err[np.ix_(rows, range(j0, j1))] = (abs(s) * (dt @ np.abs(bb)) + 2.0 ** -23 * size
                                                    + (r / 16 + 64) * e * size
                                                    + 2.0 ** -24 * (np.abs(y[rows, j0:j1]) + np.abs(add)))
                y[rows, j0:j1] += add
            j0 = j1
    return y, err
