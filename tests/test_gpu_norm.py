"""qdg_norm and qdg_gated_act against the float64 references. Residuals, rows
and codes are decided in binary64 on both sides, so they are equal bit for bit;
with unusual values the codes are those of the library's quantizers over the
rows of the same call."""

import numpy as np
import pytest
import torch

import quantized_dequant_gemm_amd as q
from oracle import codecs, layer
from tests import gpu_helpers as H

pytestmark = pytest.mark.gpu

QUANTS = {"none": q.QDG_Q_NONE, "int8": q.QDG_Q_INT8, "int8_zp": q.QDG_Q_INT8_ZP, "fp8": q.QDG_Q_FP8E4M3,
          "mxfp4": q.QDG_Q_MXFP4}
FILL = 0x5A


def _ptr(t):
    return None if t is None else t.data_ptr()


def _typed(x, f32):
    """Real values as a device tensor of the type, and what it holds in float64."""
    t = torch.from_numpy(np.ascontiguousarray(x, np.float32)).cuda()
    t = t if f32 else t.to(torch.bfloat16)
    return t, H.to_f64(t)


def _strided(t, pad, shift):
    """A copy with rows `pad` elements apart that starts `shift` elements into its buffer."""
    M, n = t.shape
    flat = torch.full((shift + M * (n + pad) + 8,), 3.0, dtype=t.dtype, device="cuda")
    view = flat[shift:shift + M * (n + pad)].view(M, n + pad)
    view[:, :n] = t
    return flat, view[:, :n], n + pad


class Out:
    """Rows and codes with guards around them."""

    def __init__(self, M, n, quant, rows, pad=0, shift=0):
        self.M, self.n, self.quant, self.ldo = M, n, quant, n + pad
        self.flat = torch.full((shift + M * self.ldo + 8,), 77.0, dtype=torch.bfloat16, device="cuda") if rows else None
        self.shift = shift
        self.bytes = n // 2 if quant == "mxfp4" else n
        self.ldq = (self.bytes + 15) // 16 * 16 + 16 * (pad > 0)
        per = {"fp8": (n // 128,), "mxfp4": (n // 32,)}.get(quant, ())
        self.qa = torch.full((M + 1, self.ldq), FILL, dtype=torch.uint8, device="cuda")
        self.scales = torch.full((M,) + per, -7.0, device="cuda") if quant != "mxfp4" else torch.full(
            (M,) + per, FILL, dtype=torch.uint8, device="cuda")
        self.zeros = torch.full((M,), 999, dtype=torch.int32, device="cuda")

    def args(self):
        rows = None if self.flat is None else self.flat.data_ptr() + 2 * self.shift
        if self.quant == "none":
            return rows, None, None, None
        return rows, self.qa.data_ptr(), self.scales.data_ptr(), self.zeros.data_ptr() if self.quant == "int8_zp" else None

    def rows(self):
        M, n = self.M, self.n
        body = self.flat[self.shift:self.shift + M * self.ldo].view(M, self.ldo)
        assert (self.flat[:self.shift] == 77).all() and (self.flat[self.shift + M * self.ldo:] == 77).all()
        assert (body[:, n:] == 77).all()
        return body[:, :n].contiguous()

    def row_bits(self):
        return self.rows().view(torch.int16).cpu().numpy().view(np.uint16)

    def codes(self):
        assert (self.qa[self.M] == FILL).all() and (self.qa[:, self.bytes:] == FILL).all()
        return self.qa[:self.M, :self.bytes].contiguous().cpu().numpy()

    def check(self, bits):
        """Against the reference's rows and the codes that follow from them."""
        if self.flat is not None:
            np.testing.assert_array_equal(self.row_bits(), bits)
        if self.quant != "none":
            codes, scales, zeros = layer.codes(bits, self.quant)
            np.testing.assert_array_equal(self.codes(), codes.view(np.uint8))
            np.testing.assert_array_equal(self.scales.cpu().numpy(), scales)
            if zeros is not None:
                np.testing.assert_array_equal(self.zeros.cpu().numpy(), zeros)
        else:
            assert (self.qa == FILL).all()


class Case:
    def __init__(self, seed, M, n, kind="rms", post=False, xf32=False, rf32=False, wf32=False, gate="none",
                 residual=True, weights=True, bias=False, scale=1.0, offset=0.0, eps=1e-5, pad=0, shift=0, spread=1.0):
        rng = np.random.default_rng(seed)
        draw = lambda *s: rng.standard_normal(s).astype(np.float32)  # noqa: E731
        self.M, self.n, self.kind, self.post = M, n, kind, post
        self.pad, self.shift = pad, shift
        x = spread * draw(M, n)
        self.dx, x = _typed(x, xf32)
        self.flat_x, self.vx, self.ldx = _strided(self.dx, pad, shift)
        self.dr = r = None
        self.ldr = n
        if residual:
            self.dr, r = _typed(spread * draw(M, n), rf32)
            self.flat_r, self.dr, self.ldr = _strided(self.dr, pad, shift)
        vec = lambda v: (None, None) if v is None else _typed(v, wf32)  # noqa: E731
        self.dg, g = vec({"none": None, "channels": draw(1, n), "rows": draw(M, n)}[gate])
        self.dw, w = vec((1 - offset + 0.3 * draw(n)) if weights else None)
        self.db, b = vec(0.2 * draw(n) if bias else None)
        self.dpw, pw = vec((1 - offset + 0.3 * draw(n)) if post and weights else None)
        self.dpb, pb = vec(0.2 * draw(n) if post and bias else None)
        code = lambda f: q.QDG_O_F32 if f else q.QDG_O_BF16  # noqa: E731
        self.rf32 = rf32
        self.kw = dict(kind=q.QDG_NORM_LAYER if kind == "layer" else q.QDG_NORM_RMS, post_norm=int(post),
                       xtype=code(xf32), rtype=code(rf32), wtype=code(wf32), eps=eps, residual_scale=scale,
                       weight_offset=offset, ldg=n if gate == "rows" else 0, ldx=self.ldx, ldr=self.ldr)
        self.s, self.bits = layer.norm(x, r, g, (pw, pb) if post else None, w, b, kind == "layer", eps, scale, offset, rf32)

    def run(self, quant="none", rows=True, keep=True, in_place=False, stream=None):
        M, n = self.M, self.n
        out = Out(M, n, quant, rows, self.pad, self.shift)
        lds = n + self.pad
        flat = torch.full((self.shift + M * lds + 8,), 55.0, dtype=torch.float32 if self.rf32 else torch.bfloat16, device="cuda")
        body = flat[self.shift:self.shift + M * lds].view(M, lds)
        if in_place:
            body = self.dr
        cfg = q.norm(n, quant=QUANTS[quant], lds=self.ldr if in_place else lds, ldo=out.ldo, ldq=out.ldq, **self.kw)
        rows_p, qa, sc, ze = out.args()
        q.qdg_norm(cfg, self.vx.data_ptr(), _ptr(self.dr), _ptr(self.dg), _ptr(self.dpw), _ptr(self.dpb), _ptr(self.dw),
                   _ptr(self.db), M, body.data_ptr() if keep else None, rows_p, qa, sc, ze,
                   q.current_stream() if stream is None else stream)
        torch.cuda.synchronize()
        if keep:
            np.testing.assert_array_equal(H.to_f64(body[:, :n]), self.s)
        if keep and not in_place:
            assert (flat[:self.shift] == 55).all() and (flat[self.shift + M * lds:] == 55).all() and (body[:, n:] == 55).all()
        return out


# one row to several blocks of rows; every shape of the kernel and its borders; odd lengths
SIZES = [(1, 1), (3, 2), (5, 7), (4, 64), (9, 100), (7, 511), (6, 512), (5, 513), (3, 1001), (2, 2048), (3, 2049), (2, 4096),
         (2, 4100), (3, 7168), (1, 8192), (2, 8193), (1, 14336), (2, 16385), (1, 32768), (1, 32767)]


@pytest.mark.parametrize("M,n", SIZES)
def test_norm_sizes(qdg, M, n):
    for i, quant in enumerate(("none", "int8", "int8_zp")):
        c = Case(n + i, M, n, kind=("rms", "layer")[(n + i) & 1], post=bool(i & 1), xf32=bool(n & 1), rf32=i == 2,
                 wf32=i == 1, gate=("none", "rows", "channels")[i], bias=i != 0, scale=(1.0, 0.75, 0.3)[i],
                 offset=(0.0, 1.0, 0.0)[i], pad=(0, 3, 8)[i], shift=(0, 1, 0)[i])
        c.run(quant).check(c.bits)


@pytest.mark.parametrize("quant", list(QUANTS))
@pytest.mark.parametrize("xf32", [False, True])
@pytest.mark.parametrize("rf32", [False, True])
def test_norm_types_and_codes(qdg, quant, xf32, rf32):
    for i, (M, n) in enumerate(((5, 128), (3, 384), (4, 640), (6, 2176), (2, 5120), (3, 8320), (1, 17408))):
        c = Case(i, M, n, kind=("rms", "layer")[i & 1], post=i % 3 == 1, xf32=xf32, rf32=rf32, wf32=bool(i & 2),
                 gate=("channels", "none", "rows")[i % 3], bias=bool(i & 1), pad=(0, 5)[i & 1], shift=(0, 3)[i & 1])
        c.run(quant, rows=bool(i & 1) or quant == "none").check(c.bits)


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("post", [False, True])
def test_what_may_be_absent(qdg, kind, post):
    for residual in (False, True):
        for weights in (False, True):
            for bias in (False, True):
                c = Case(5, 3, 640, kind, post, residual=residual, weights=weights, bias=bias, gate="rows", offset=1.0)
                c.run("int8").check(c.bits)
                c.run("fp8", keep=False, rows=False).check(c.bits)
    c = Case(6, 4, 640, kind, post)
    c.run("none", rows=False)  # the stream alone


def test_residual_in_place_and_rows_over_x(qdg):
    for rf32 in (False, True):
        for n, pad in ((100, 0), (4096, 3), (9001, 1)):
            c = Case(n, 5, n, rf32=rf32, pad=pad, shift=1)
            c.run("none", in_place=True).check(c.bits)
    c = Case(8, 6, 4100, post=True)
    cfg = q.norm(4100, **c.kw)
    q.qdg_norm(cfg, c.vx.data_ptr(), c.dr.data_ptr(), None, _ptr(c.dpw), None, _ptr(c.dw), None, 6, None,
               c.vx.data_ptr(), None, None, None, q.current_stream())
    torch.cuda.synchronize()
    np.testing.assert_array_equal(c.vx.contiguous().view(torch.int16).cpu().numpy().view(np.uint16), c.bits)


@pytest.mark.parametrize("spread", [1e-30, 1e-4, 1e4, 1e18, 3e37])
@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_ranges(qdg, spread, kind):
    """Squares beyond binary32's range, and rows in which eps decides."""
    for quant in ("int8", "int8_zp", "mxfp4"):
        c = Case(11, 4, 1024, kind, xf32=True, rf32=True, spread=spread, bias=True)
        c.run(quant).check(c.bits)


def test_rows_that_nearly_cancel(qdg):
    """A layer norm of rows that lie far from 0, and gates that take the stream back."""
    rng = np.random.default_rng(3)
    M, n = 4, 2050
    x = (1000.0 + rng.standard_normal((M, n)) * 1e-3).astype(np.float32)
    r = (-x * (1 + 1e-6 * rng.standard_normal((M, n)))).astype(np.float32)
    for residual in (None, r):
        dx = torch.from_numpy(x).cuda()
        dr = None if residual is None else torch.from_numpy(residual).cuda()
        s, bits = layer.norm(x.astype(np.float64), residual, None, None, None, None, True, 1e-12, 1.0, 0.0, True)
        out = Out(M, n, "int8", True)
        new = torch.empty((M, n), device="cuda")
        cfg = q.norm(n, kind=q.QDG_NORM_LAYER, xtype=q.QDG_O_F32, rtype=q.QDG_O_F32, quant=q.QDG_Q_INT8, eps=1e-12, ldq=out.ldq)
        rows, qa, sc, _ = out.args()
        q.qdg_norm(cfg, dx.data_ptr(), _ptr(dr), None, None, None, None, None, M, new.data_ptr(), rows, qa, sc, None,
                   q.current_stream())
        torch.cuda.synchronize()
        np.testing.assert_array_equal(H.to_f64(new), s)
        out.check(bits)


def _library_codes(rows, quant):
    """What the library's quantizers give for bf16 rows."""
    M, n = rows.shape
    if quant == "int8_zp":
        ld = (n + 15) // 16 * 16
        qa = torch.zeros((M, ld), dtype=torch.int8, device="cuda")
        s, z = torch.zeros(M, device="cuda"), torch.zeros(M, dtype=torch.int32, device="cuda")
        q.qdg_quantize_act_zp(rows.data_ptr(), n, M, n, qa.data_ptr(), ld, s.data_ptr(), z.data_ptr(), q.current_stream())
        return qa[:, :n].contiguous().view(torch.uint8), s, z
    make = {"int8": q.layer_w8a8, "fp8": q.layer_mxfp4, "mxfp4": q.layer_w4a4}[quant]
    qa = torch.zeros((M, n // 2 if quant == "mxfp4" else n), dtype=torch.uint8, device="cuda")
    s = {"int8": torch.zeros(M, device="cuda"), "fp8": torch.zeros((M, n // 128), device="cuda"),
         "mxfp4": torch.zeros((M, n // 32), dtype=torch.uint8, device="cuda")}[quant]
    q.qdg_quantize_act(make(128, n), rows.data_ptr(), M, qa.data_ptr(), s.data_ptr(), q.current_stream())
    return qa, s, None


@pytest.mark.parametrize("quant", ["int8", "int8_zp", "fp8", "mxfp4"])
def test_codes_of_unusual_rows_are_the_quantizers(qdg, quant):
    """Zeros, infinities, NaN and values at the ends of the types, through the norm and through the activation."""
    M, n = 10, 1024
    rng = np.random.default_rng(2)
    x = rng.standard_normal((M, n)).astype(np.float32)
    x[0] = 0.0
    x[1, 5] = np.inf
    x[2, 700] = -np.inf
    x[3, 3] = np.nan
    x[4, :] = -0.0
    x[5, 1:] = 0.0
    x[6] = 3.3e38
    x[7] = 1e-41
    x[8, 17] = 3e38
    x[9, :128] = 0.0
    dx = torch.from_numpy(x).cuda()
    for eps in (0.0, 1e-5):
        out, new = Out(M, n, quant, True), torch.empty((M, n), device="cuda")
        rows, qa, sc, ze = out.args()
        cfg = q.norm(n, xtype=q.QDG_O_F32, rtype=q.QDG_O_F32, quant=QUANTS[quant], eps=eps, ldq=out.ldq)
        q.qdg_norm(cfg, dx.data_ptr(), None, None, None, None, None, None, M, new.data_ptr(), rows, qa, sc, ze, q.current_stream())
        torch.cuda.synchronize()
        np.testing.assert_array_equal(new.cpu().numpy(), x)
        y = out.rows()
        nan = torch.isnan(y)
        assert nan[3].all() and nan[1, 5] and nan[2, 700] and (y[1, :5] == 0).all()
        assert nan[0].all() == (eps == 0.0) and not nan[5:].any()
        _same_codes(out, y, quant)
    yy = torch.cat([dx, 2.0 * torch.ones_like(dx)], dim=1).contiguous()
    yy[:, n + 1] = float("nan")
    out = Out(M, n, quant, True)
    rows, qa, sc, ze = out.args()
    cfg = q.gated_act(n, ytype=q.QDG_O_F32, quant=QUANTS[quant], ldq=out.ldq)
    q.qdg_gated_act(cfg, yy.data_ptr(), M, rows, qa, sc, ze, q.current_stream())
    torch.cuda.synchronize()
    y = out.rows()
    assert torch.isnan(y[:, 1]).all() and torch.isnan(y[3, 3]) and torch.isinf(y[1, 5]) and torch.isnan(y[2, 700])
    _same_codes(out, y, quant)


def _same_codes(out, y, quant):
    qa, s, z = _library_codes(y, quant)
    torch.cuda.synchronize()
    np.testing.assert_array_equal(out.codes(), qa.cpu().numpy())
    np.testing.assert_array_equal(out.scales.cpu().numpy(), s.cpu().numpy())
    if z is not None:
        np.testing.assert_array_equal(out.zeros.cpu().numpy(), z.cpu().numpy())


def _gated(seed, M, n, act, yf32, quant, rows, pad=0, shift=0, spread=2.0):
    rng = np.random.default_rng(seed)
    t, y = _typed(spread * rng.standard_normal((M, 2 * n)), yf32)
    flat, view, ldy = _strided(t, pad, shift)
    out = Out(M, n, quant, rows, pad, shift)
    r, qa, sc, ze = out.args()
    cfg = q.gated_act(n, act=q.QDG_ACT_SILU if act == "silu" else q.QDG_ACT_GELU_TANH,
                      ytype=q.QDG_O_F32 if yf32 else q.QDG_O_BF16, quant=QUANTS[quant], ldy=ldy, ldo=out.ldo, ldq=out.ldq)
    q.qdg_gated_act(cfg, view.data_ptr(), M, r, qa, sc, ze, q.current_stream())
    torch.cuda.synchronize()
    out.check(layer.gated_act(y, act))


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("yf32", [False, True])
def test_gated_sizes(qdg, act, yf32):
    for i, (M, n) in enumerate(SIZES + [(1, 53248), (2, 65536), (1, 65535)]):
        _gated(n, M, n, act, yf32, ("none", "int8", "int8_zp")[i % 3], rows=i % 3 == 0 or bool(i & 1), pad=(0, 3)[i & 1],
               shift=(0, 1, 2)[i % 3])


@pytest.mark.parametrize("quant", list(QUANTS))
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_gated_codes(qdg, quant, act):
    for i, (M, n) in enumerate(((1, 128), (5, 256), (3, 1152), (4, 2304), (2, 14336), (1, 33024))):
        _gated(i, M, n, act, bool(i & 1), quant, rows=quant == "none" or bool(i & 1))


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("spread", [1e-30, 1e-3, 30.0, 200.0, 1e30])
def test_gated_ranges(qdg, act, spread):
    """Gates at which the exponential leaves binary32's and binary64's range. No code of a value that is an infinity."""
    _gated(7, 6, 1024, act, True, "none", True, spread=spread)


def test_every_bf16_gate(qdg):
    """act over every finite bf16 number, beside several factors."""
    bits = np.arange(65536, dtype=np.uint32).astype(np.uint16)
    bits = bits[(bits & 0x7F80) != 0x7F80]
    g = codecs.bf16_bits_to_f64(bits)
    n = g.size
    y = np.empty((3, 2 * n))
    y[:, :n] = g
    y[:, n:] = np.array([1.0, -0.7109375, 1.9921875])[:, None]
    t = torch.from_numpy(y.astype(np.float32)).cuda().to(torch.bfloat16)
    for act, code in (("silu", q.QDG_ACT_SILU), ("gelu", q.QDG_ACT_GELU_TANH)):
        out = Out(3, n, "none", True)
        q.qdg_gated_act(q.gated_act(n, act=code), t.data_ptr(), 3, out.args()[0], stream=q.current_stream())
        torch.cuda.synchronize()
        np.testing.assert_array_equal(out.row_bits(), layer.gated_act(H.to_f64(t), act))


def test_many_rows(qdg):
    """More rows than workgroups of one launch walk at once, every row its own result."""
    M, n = (1 << 22) + 5, 8
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    x = torch.randn((M, n), generator=gen, device="cuda").to(torch.bfloat16)
    out, new = torch.zeros_like(x), torch.zeros_like(x)
    q.qdg_norm(q.norm(n), x.data_ptr(), None, None, None, None, None, None, M, new.data_ptr(), out.data_ptr(),
               stream=q.current_stream())
    torch.cuda.synchronize()
    assert torch.equal(new, x)
    for at in (0, (1 << 21) - 3, M - 1000):
        _, bits = layer.norm(H.to_f64(x[at:at + 1000]))
        np.testing.assert_array_equal(out[at:at + 1000].view(torch.int16).cpu().numpy().view(np.uint16), bits)


def test_offsets_past_32_bits(qdg):
    """The last of rows whose stride takes them past 4 GiB."""
    M, n, ld = 3, 640, (1 << 30) + 3
    x = torch.zeros((M - 1) * ld + n, dtype=torch.bfloat16, device="cuda")
    rng = np.random.default_rng(9)
    want = []
    for m in range(M):
        t, v = _typed(rng.standard_normal((1, n)), False)
        x[m * ld:m * ld + n] = t[0]
        want.append(v)
    _, bits = layer.norm(np.concatenate(want))
    out = Out(M, n, "int8", True)
    rows, qa, sc, _ = out.args()
    q.qdg_norm(q.norm(n, quant=q.QDG_Q_INT8, ldx=ld, ldq=out.ldq), x.data_ptr(), None, None, None, None, None, None, M, None,
               rows, qa, sc, None, q.current_stream())
    torch.cuda.synchronize()
    out.check(bits)
    bits = layer.gated_act(np.concatenate(want))
    out = Out(M, n // 2, "int8_zp", True)
    rows, qa, sc, ze = out.args()
    q.qdg_gated_act(q.gated_act(n // 2, quant=q.QDG_Q_INT8_ZP, ldy=ld, ldq=out.ldq), x.data_ptr(), M, rows, qa, sc, ze,
                    q.current_stream())
    torch.cuda.synchronize()
    out.check(bits)


def test_replayed_graph_and_other_stream(qdg):
    M, n = 7, 1152
    side = torch.cuda.Stream()
    c = Case(1, M, n, post=True, gate="rows")
    torch.cuda.synchronize()
    c.run("int8", stream=side.cuda_stream).check(c.bits)
    x = torch.zeros((M, n), dtype=torch.bfloat16, device="cuda")
    stream_rows, w = torch.zeros_like(x), torch.ones(n, dtype=torch.bfloat16, device="cuda")
    out, gated = Out(M, n, "fp8", True), Out(M, n // 2, "int8_zp", False)
    cfg = q.norm(n, quant=q.QDG_Q_FP8E4M3, ldq=out.ldq)
    gcfg = q.gated_act(n // 2, quant=q.QDG_Q_INT8_ZP, ldq=gated.ldq)
    rows, qa, sc, _ = out.args()
    _, gqa, gsc, gze = gated.args()

    def calls():
        q.qdg_norm(cfg, x.data_ptr(), stream_rows.data_ptr(), None, None, None, w.data_ptr(), None, M, stream_rows.data_ptr(),
                   rows, qa, sc, None, q.current_stream())
        q.qdg_gated_act(gcfg, rows, M, None, gqa, gsc, gze, q.current_stream())

    calls()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        calls()
    rng = np.random.default_rng(4)
    for _ in range(4):
        t, v = _typed(rng.standard_normal((M, n)), False)
        r, rv = _typed(rng.standard_normal((M, n)), False)
        x.copy_(t)
        stream_rows.copy_(r)
        g.replay()
        torch.cuda.synchronize()
        s, bits = layer.norm(v, rv)
        np.testing.assert_array_equal(H.to_f64(stream_rows), s)
        out.check(bits)
        gated.check(layer.gated_act(codecs.bf16_bits_to_f64(bits)))


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_gates_and_factors_far_apart(qdg, act):
    """Gates near 0 and far below it beside large factors: the quotient alone would leave binary32's normal range."""
    rng = np.random.default_rng(21)
    M, n = 8, 1024
    g = np.concatenate([-rng.uniform(80.0, 100.0, n // 4), -rng.uniform(8.0, 11.0, n // 4),
                        10.0 ** rng.uniform(-44, -30, n // 4), -(10.0 ** rng.uniform(-44, -30, n // 4))])
    y = np.empty((M, 2 * n), np.float32)
    y[:, :n] = rng.permutation(g).astype(np.float32)
    y[:, n:] = (10.0 ** rng.uniform(0, 38, (M, n)) * rng.choice([-1, 1], (M, n))).astype(np.float32)
    t = torch.from_numpy(y).cuda()
    out = Out(M, n, "none", True)
    q.qdg_gated_act(q.gated_act(n, act=q.QDG_ACT_SILU if act == "silu" else q.QDG_ACT_GELU_TANH, ytype=q.QDG_O_F32),
                    t.data_ptr(), M, out.args()[0], stream=q.current_stream())
    torch.cuda.synchronize()
    out.check(layer.gated_act(y.astype(np.float64), act))


def test_stream_and_weights_far_apart(qdg):
    """Products of factors at the ends of binary32's range."""
    rng = np.random.default_rng(22)
    M, n = 6, 1024
    r = (10.0 ** rng.uniform(-40, 0, (M, n))).astype(np.float32)
    r[3:] = (10.0 ** rng.uniform(0, 38, (3, n))).astype(np.float32)
    w = (10.0 ** rng.uniform(-38, 38, n) * rng.choice([-1, 1], n)).astype(np.float32)
    b = (10.0 ** rng.uniform(-38, 38, n)).astype(np.float32)
    dr, dw, db = (torch.from_numpy(v).cuda() for v in (r, w, b))
    for wf32, bias in ((True, False), (True, True), (False, False)):
        cw = dw if wf32 else dw.to(torch.bfloat16)
        out = Out(M, n, "none", True)
        cfg = q.norm(n, xtype=q.QDG_O_F32, rtype=q.QDG_O_F32, wtype=q.QDG_O_F32 if wf32 else q.QDG_O_BF16)
        q.qdg_norm(cfg, dr.data_ptr(), None, None, None, None, cw.data_ptr(), db.data_ptr() if bias else None, M, None,
                   out.args()[0], stream=q.current_stream())
        torch.cuda.synchronize()
        _, bits = layer.norm(r, weight=H.to_f64(cw), bias=b if bias else None, r_f32=True)
        out.check(bits)


@pytest.mark.parametrize("n", [3, 13, 1001, 2047, 4099, 8191, 16387])
@pytest.mark.parametrize("wf32", [False, True])
def test_cut_rows_with_tiny_ends(qdg, n, wf32):
    """The last chunk of a row of an odd length holds zeros, subnormal and tiny values, or nothing but those."""
    rng = np.random.default_rng(n)
    ends = np.array([0.0, -0.0, 1e-40, -3e-39, 2.0 ** -100, 2.0 ** -101, 1.5 * 2.0 ** -126], np.float32)
    x = rng.standard_normal((4, n)).astype(np.float32)
    for row in range(3):
        k = min(n, (n % 8, 1, 7)[row])
        x[row, n - k:] = rng.permutation(ends)[:k]
    x[3] = rng.choice(ends, n)
    wt = torch.float32 if wf32 else torch.bfloat16
    w, b = (torch.from_numpy(rng.standard_normal(n).astype(np.float32)).to(wt) for _ in range(2))
    dx, dw, db = torch.from_numpy(x).cuda(), w.cuda(), b.cuda()
    for kind, bias in (("rms", False), ("rms", True), ("layer", False)):
        _, bits = layer.norm(x.astype(np.float64), None, None, None, w.double().numpy(), b.double().numpy() if bias else None,
                             kind == "layer", 1e-30, 1.0, 0.0, True)
        out = Out(4, n, "int8", True)
        cfg = q.norm(n, kind=q.QDG_NORM_LAYER if kind == "layer" else q.QDG_NORM_RMS, xtype=q.QDG_O_F32, rtype=q.QDG_O_F32,
                     wtype=q.QDG_O_F32 if wf32 else q.QDG_O_BF16, quant=q.QDG_Q_INT8, eps=1e-30, ldq=out.ldq)
        rows, qa, sc, _ = out.args()
        q.qdg_norm(cfg, dx.data_ptr(), None, None, None, None, dw.data_ptr(), _ptr(db if bias else None), 4, None, rows, qa,
                   sc, None, q.current_stream())
        torch.cuda.synchronize()
        out.check(bits)
