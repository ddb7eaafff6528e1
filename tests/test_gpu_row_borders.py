"""qdg_norm where an operation of binary32 would leave its range or its bits, against the float64 references."""

import numpy as np
import pytest
import torch

import quantized_dequant_gemm_amd as q
from oracle import layer
from tests import gpu_helpers as H
from tests.test_gpu_norm import QUANTS, Out, _ptr, _typed

pytestmark = pytest.mark.gpu


def _call(x, xf32, quant="int8", residual=None, rf32=False, gate=None, weight=None, bias=None, wf32=False, kind="rms",
          post=None, scale=1.0, offset=0.0, eps=1e-5):
    """Runs the norm; returns (Out, the new stream in float64, the reference's stream and rows)."""
    M, n = x.shape
    dx, x64 = _typed(x, xf32)
    up = lambda v, f32: (None, None) if v is None else _typed(v, f32)  # noqa: E731
    (dr, r64), (dg, g64), (dw, w64), (db, b64) = up(residual, rf32), up(gate, wf32), up(weight, wf32), up(bias, wf32)
    (dpw, pw64), (dpb, pb64) = (up(v, wf32) for v in (post or (None, None)))
    with np.errstate(over="ignore", invalid="ignore", divide="ignore"):
        s, bits = layer.norm(x64, r64, g64, None if post is None else (pw64, pb64), w64, b64, kind == "layer", eps, scale,
                             offset, rf32)
    out = Out(M, n, quant, True)
    new = torch.empty((M, n), dtype=torch.float32 if rf32 else torch.bfloat16, device="cuda")
    code = lambda f32: q.QDG_O_F32 if f32 else q.QDG_O_BF16  # noqa: E731
    cfg = q.norm(n, kind=q.QDG_NORM_LAYER if kind == "layer" else q.QDG_NORM_RMS, xtype=code(xf32), rtype=code(rf32),
                 wtype=code(wf32), post_norm=int(post is not None), quant=QUANTS[quant], eps=eps, residual_scale=scale,
                 weight_offset=offset, ldg=n if gate is not None and len(gate) > 1 else 0, ldq=out.ldq)
    rows, qa, sc, ze = out.args()
    q.qdg_norm(cfg, dx.data_ptr(), _ptr(dr), _ptr(dg), _ptr(dpw), _ptr(dpb), _ptr(dw), _ptr(db), M, new.data_ptr(), rows,
               qa, sc, ze, q.current_stream())
    torch.cuda.synchronize()
    return out, H.to_f64(new), s, bits


def _same_codes(out):
    """The int8 codes with zero points are those of the library's quantizer over the rows of the call."""
    y = out.rows()
    lda, ldq = (out.n + 7) // 8 * 8, (out.n + 15) // 16 * 16
    a = torch.zeros((out.M, lda), dtype=torch.bfloat16, device="cuda")
    a[:, :out.n] = y
    qa = torch.zeros((out.M, ldq), dtype=torch.int8, device="cuda")
    s, z = torch.zeros(out.M, device="cuda"), torch.zeros(out.M, dtype=torch.int32, device="cuda")
    q.qdg_quantize_act_zp(a.data_ptr(), lda, out.M, out.n, qa.data_ptr(), ldq, s.data_ptr(), z.data_ptr(), q.current_stream())
    torch.cuda.synchronize()
    np.testing.assert_array_equal(out.codes(), qa[:, :out.n].cpu().numpy().view(np.uint8))
    np.testing.assert_array_equal(out.scales.cpu().numpy(), s.cpu().numpy())
    np.testing.assert_array_equal(out.zeros.cpu().numpy(), z.cpu().numpy())


@pytest.mark.parametrize("rf32", [False, True])
@pytest.mark.parametrize("n", [1024, 1001, 5])
def test_gate_products_outside_binary32s_range(qdg, n, rf32):
    """gate * x above the largest binary32 number that the residual takes back, and below the normal ones beside
    residuals of that size."""
    rng = np.random.default_rng(n)
    M = 6
    x, g, r = (rng.standard_normal((M, n)) for _ in range(3))
    x[:2], g[:2] = 2e19 * np.sign(x[:2]), 2e19 * (1 + rng.random((2, n)) / 8)
    r[:2] = -2e38 * np.sign(x[:2])
    x[2:4], g[2:4] = x[2:4] * 2.0 ** -70, g[2:4] * 2.0 ** -69
    r[2:4] = r[2:4] * 2.0 ** -140
    x[4, ::3] = 0.0  # exact zeros, an infinity and a NaN go the same way as in 64 bits
    x[5, 1], x[5, 2] = np.inf, np.nan
    for kind, bias in (("rms", None), ("layer", rng.standard_normal(n))):
        for scale in (1.0, 0.75):
            out, new, s, bits = _call(x, False, "int8_zp", r, rf32, g, rng.standard_normal(n), bias, kind=kind, scale=scale)
            assert np.isfinite(s[:5]).all()
            np.testing.assert_array_equal(new, s)
            np.testing.assert_array_equal(out.row_bits()[:5], bits[:5])
            _same_codes(out)


@pytest.mark.parametrize("n", [1024, 1001])
@pytest.mark.parametrize("wf32", [False, True])
def test_weights_with_an_offset_past_binary32s_range(qdg, n, wf32):
    """weight + offset above the largest binary32 number beside values that bring the product back."""
    rng = np.random.default_rng(n)
    x = rng.standard_normal((4, n)) * 2.0 ** -6
    x[:, ::16] *= 2.0 ** 9
    w = rng.standard_normal(n)
    w[::2] = 3e38
    w[1::8] = -3e38
    for kind, bias in (("rms", None), ("rms", rng.standard_normal(n)), ("layer", None)):
        out, new, s, bits = _call(x, False, "int8_zp", weight=w, bias=bias, wf32=wf32, kind=kind, offset=3e38)
        np.testing.assert_array_equal(new, s)
        assert (bits[:, 2::16] & 0x7FFF < 0x7F80).any()
        np.testing.assert_array_equal(out.row_bits(), bits)
        _same_codes(out)


@pytest.mark.parametrize("n", [49, 196, 1001, 3136, 7488, 8191, 24500])
def test_layer_norm_of_constant_rows(qdg, n):
    """A row of one value has that value as its mean (n of them add up without a rounding), so it is 0 beside eps > 0 and
    0 / 0 beside eps = 0."""
    values = np.array([1.0, -3.140625, 0.1, 1e15, 1.1754944e-38, 7.0 / 3.0, -2e30])
    x = np.tile(values[:, None], (1, n))
    rng = np.random.default_rng(n)
    w, b = rng.standard_normal(n), rng.standard_normal(n)
    quants = ["none", "int8", "int8_zp"] + ["fp8"] * (n % 128 == 0) + ["mxfp4"] * (n % 32 == 0)
    for i, quant in enumerate(quants):
        for f32 in (False, True):
            for bias in (None, b):
                out, new, s, bits = _call(x, f32, quant, rf32=f32, weight=w, bias=bias, wf32=i == 2, kind="layer")
                np.testing.assert_array_equal(new, s)
                out.check(bits)
            out, new, s, _ = _call(x, f32, quant, rf32=f32, weight=w, kind="layer", eps=0.0)
            assert torch.isnan(out.rows()).all()
    # the norm of x, as it joins the stream
    for eps in (1e-5, 0.0):
        out, new, s, bits = _call(x, True, "int8", rng.standard_normal(x.shape), True, weight=w, kind="layer", post=(w, b), eps=eps)
        if eps:
            np.testing.assert_array_equal(new, s)
            out.check(bits)
        else:
            assert np.isnan(new).all()


@pytest.mark.parametrize("M,k", [(2049, 1040), (2048, 4090), (8195, 500), (8192, 1024)])
def test_zero_point_codes_do_not_depend_on_the_batch(qdg, M, k):
    """Many short rows take another instance of the quantizer than few: the same codes, with infinities and NaN too."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(k)
    lda, ldq = (k + 7) // 8 * 8, (k + 15) // 16 * 16
    a = torch.randn((M, lda), generator=gen, device="cuda").to(torch.bfloat16)
    a[3, 7], a[4, 1], a[5, k - 1] = float("inf"), float("nan"), -float("inf")
    a[6], a[7] = 0.0, 2.5

    def quantize(rows):
        m = rows.shape[0]
        qa = torch.zeros((m, ldq), dtype=torch.int8, device="cuda")
        s, z = torch.zeros(m, device="cuda"), torch.zeros(m, dtype=torch.int32, device="cuda")
        q.qdg_quantize_act_zp(rows.data_ptr(), lda, m, k, qa.data_ptr(), ldq, s.data_ptr(), z.data_ptr(), q.current_stream())
        return qa, s, z

    whole = quantize(a)
    for at in range(0, M, 500):
        part = quantize(a[at:at + 500])
        for w, p in zip(whole, part):
            assert torch.equal(w[at:at + 500], p)
    bits = a[:40, :k].contiguous().view(torch.int16).cpu().numpy().view(np.uint16)
    codes, scales, zeros = layer.codes(bits, "int8_zp")
    np.testing.assert_array_equal(whole[0][:40, :k].cpu().numpy(), codes)
    np.testing.assert_array_equal(whole[1][:40].cpu().numpy(), scales)
    np.testing.assert_array_equal(whole[2][:40].cpu().numpy(), zeros)
