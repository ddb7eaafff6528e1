"""References of the expert router, the asymmetric activation quantizer and the
int8 products over stored operands, in float64 and int64.

Test infrastructure (see the package docstring): plain definitions, one token
or one row at a time where that is the plainest form.
"""

import math

import numpy as np


# ---------------------------------------------------------------- routing

def _sigmoid(x):
    if x >= 0:
        return 1.0 / (1.0 + math.exp(-x))
    e = math.exp(x)
    return e / (1.0 + e)


def route(logits, top_k, score="softmax", bias=None, groups=1, topk_groups=1, group_score="max", renorm=False,
          scale=1.0):
    """Expert ids int32 [T][top_k], weights float64 [T][top_k] and whether a
    logit or a bias was NaN or a logit +infinity.

    A masked expert (logit or bias -inf or NaN) scores 0, ranks behind all
    others and adds nothing to its group."""
    x = np.asarray(logits, np.float64)
    t, e = x.shape
    b = np.zeros(e) if bias is None else np.asarray(bias, np.float64)
    per = e // groups
    bad = bool(np.isnan(x).any() or (x == np.inf).any() or np.isnan(b).any())
    ids = np.zeros((t, top_k), np.int32)
    weights = np.zeros((t, top_k))
    fmax = float(np.finfo(np.float32).max)
    for row in range(t):
        l = [-math.inf if math.isnan(v) else min(float(v), fmax) for v in x[row]]
        masked = [l[i] == -math.inf or math.isnan(b[i]) or b[i] == -math.inf for i in range(e)]
        if score == "sigmoid":
            s = [0.0 if v == -math.inf else _sigmoid(v) for v in l]
        else:
            top = max(l)
            ex = [0.0 if v == -math.inf else math.exp(v - top) for v in l]
            total = math.fsum(ex)
            s = [v / total if total > 0 else 0.0 for v in ex]
        c = [-math.inf if masked[i] else s[i] + float(b[i]) for i in range(e)]
        s = [0.0 if masked[i] else s[i] for i in range(e)]
        values = []
        for g in range(groups):
            best = sorted((v for v in c[g * per:(g + 1) * per] if v != -math.inf), reverse=True)
            best = best[:1] if group_score == "max" else best[:2]
            values.append(sum(best) if best else -math.inf)
        stay = set(sorted(range(groups), key=lambda g: (-values[g], g))[:topk_groups])
        key = c if bias is not None else [-math.inf if masked[i] else l[i] for i in range(e)]
        open_ = [i for i in range(e) if i // per in stay]
        chosen = sorted(open_, key=lambda i: (-key[i], i))[:top_k]
        w = [s[i] for i in chosen]
        if renorm:
            total = math.fsum(w)
            w = [v / total if total > 0 else 0.0 for v in w]
        ids[row] = chosen
        weights[row] = [v * scale for v in w]
    return ids, weights, bad


# ---------------------------------------------------------------- asymmetric int8 activations

def quantize_act_zp(x):
    """Rows of real values -> (codes int8, scales float32, zeros int32)."""
    x = np.asarray(x, np.float64)
    m, k = x.shape
    codes = np.zeros((m, k), np.int8)
    scales = np.ones(m, np.float32)
    zeros = np.zeros(m, np.int32)
    for row in range(m):
        fin = x[row][np.isfinite(x[row])]
        lo, hi = min(0.0, fin.min(initial=0.0)), max(0.0, fin.max(initial=0.0))
        if hi > lo:
            scales[row] = max(np.float32((hi - lo) / 255.0), np.float32(2.0 ** -126))
        inv = 1.0 / float(scales[row])
        if hi > lo:
            zeros[row] = int(min(max(np.rint(-128.0 - lo * inv), -128.0), 127.0))
        v = np.where(np.isnan(x[row]), 0.0, x[row])
        codes[row] = np.clip(np.rint(v * inv) + zeros[row], -128, 127).astype(np.int8)
    return codes, scales, zeros


# ---------------------------------------------------------------- int8 products

def int_product(a, b, a_zeros=None):
    """sum_k (a - za) * b as int64 [M][n], exactly."""
    a = np.asarray(a, np.int64)
    if a_zeros is not None:
        a = a - np.asarray(a_zeros, np.int64)[:, None]
    # integers below 2^53 in float64: exact in any summation order
    return (a.astype(np.float64) @ np.asarray(b, np.float64).T).astype(np.int64)


def gemm_i8(a, a_scales, b, b_scales, a_zeros=None, bias=None, silu_mul=False):
    """(Y64, tolerance): the product in float64 and the largest error that a
    binary32 evaluation of scales, bias and epilogue can have.

    p = float(acc) * sa * sb takes three roundings of at most half a step
    (2^-24), the bias one of the result: |err| <= 4 * 2^-24 (|p| + |bias|)
    with 2nd-order terms to spare. silu(g) * u, with silu' below 1.1: the two
    inputs' errors, plus exp (2 units in the last place, 2^-22 of its value),
    the sum, the quotient (2.5 units) and two products: below 2^-20 of the
    result."""
    p = int_product(a, b, a_zeros).astype(np.float64)
    p = p * np.asarray(a_scales, np.float64)[:, None] * np.asarray(b_scales, np.float64)[None, :]
    bb = np.zeros(p.shape[1]) if bias is None else np.asarray(bias, np.float64)
    y = p + bb
    err = 4 * 2.0 ** -24 * (np.abs(p) + np.abs(bb))
    if not silu_mul:
        return y, err
    i = y.shape[1] // 2
    g, u, eg, eu = y[:, :i], y[:, i:], err[:, :i], err[:, i:]
    e = np.exp(-np.abs(g))
    s = g * np.where(g >= 0, 1.0 / (1.0 + e), e / (1.0 + e))
    return s * u, 2.0 ** -20 * np.abs(s * u) + 1.1 * eg * (np.abs(u) + eu) + np.abs(s) * eu
