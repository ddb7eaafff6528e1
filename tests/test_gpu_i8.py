"""qdg_quantize_act_zp, qdg_gemm_i8 and qdg_moe_gemm_i8 against the int64 /
float64 references: codes, zero points and int32 outputs equal; f32 outputs
within the bound of oracle.ops.gemm_i8 (counted binary32 roundings), bf16
outputs within half a step (2^-8) more."""

import numpy as np
import pytest
import torch

import quantized_dequant_gemm_amd as q
from oracle import codecs, ops, ref
from tests import gpu_helpers as H

pytestmark = pytest.mark.gpu


def _dev_codes(codes, ld, fill):
    """Codes [rows][k] in rows of ld bytes, `fill` behind each row's end."""
    buf = np.full((codes.shape[0], ld), fill, np.int8)
    buf[:, :codes.shape[1]] = codes
    return H.dev(buf)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _close(y, y64, err, bf16):
    y = H.to_f64(y)
    bound = err + (2.0 ** -8 * (np.abs(y64) + err) if bf16 else 2.0 ** -24 * np.abs(y64)) + 2.0 ** -126
    bad = np.argwhere(~(np.abs(y - y64) <= bound))
    assert bad.size == 0, [(tuple(b), y[tuple(b)], y64[tuple(b)], bound[tuple(b)]) for b in bad[:5]]


class Layer:
    """One set of operands of a product and its reference."""

    def __init__(self, rng, M, n, k, zeros, bias, experts=1, pad_a=0, pad_b=0, extremes=False):
        self.M, self.n, self.k, self.experts = M, n, k, experts
        lo, hi = (-128, 128)
        self.a = rng.integers(lo, hi, (M, k)).astype(np.int8)
        self.b = rng.integers(lo, hi, (experts, n, k)).astype(np.int8)
        self.za = rng.integers(-128, 128, M).astype(np.int32) if zeros else None
        if extremes:
            self.a[:], self.b[:] = -128, -128
            if zeros:
                self.za[:] = 127
        self.sa = rng.uniform(0.001, 0.05, M).astype(np.float32)
        self.sb = rng.uniform(1e-4, 1e-3, (experts, n)).astype(np.float32)
        self.bias = (10.0 * rng.standard_normal((experts, n))).astype(np.float32) if bias else None
        k16 = (k + 15) // 16 * 16
        self.lda, self.ldb = k16 + 16 * pad_a, k16 + 16 * pad_b
        self.dA = _dev_codes(self.a, self.lda, 113)
        self.dB = _dev_codes(self.b.reshape(experts * n, k), self.ldb, -77)
        self.dza = None if self.za is None else H.dev(self.za)
        self.dsa, self.dsb = H.dev(self.sa), H.dev(self.sb)
        self.dbias = None if self.bias is None else H.dev(self.bias)

    def cfg(self, otype, epi, ldy=None):
        return q.gemm_i8(self.n, self.k, lda=self.lda, ldb=self.ldb, ldy=ldy, num_experts=self.experts, otype=otype,
                         epilogue=epi)

    def ref(self, epi, rows=slice(None), e=0):
        return ops.gemm_i8(self.a[rows], self.sa[rows], self.b[e], self.sb[e],
                           None if self.za is None else self.za[rows], None if self.bias is None else self.bias[e],
                           epi == q.QDG_EPI_SILU_MUL)


def _dense(L, otype, epi=q.QDG_EPI_NONE, pad_y=0, shift_y=0):
    cols = L.n // 2 if epi else L.n
    dt = {q.QDG_O_BF16: torch.bfloat16, q.QDG_O_F32: torch.float32, q.QDG_O_I32: torch.int32}[otype]
    ldy = cols + pad_y
    cfg = L.cfg(otype, epi, ldy)
    flat = torch.full(((L.M + 1) * ldy + 8,), 77, dtype=dt, device="cuda")
    nbytes = q.qdg_gemm_i8_workspace(cfg, L.M)
    ws = torch.full((max(nbytes, 16),), 0x5A, dtype=torch.uint8, device="cuda")
    q.qdg_gemm_i8(cfg, L.dA.data_ptr(), L.dsa.data_ptr(), _ptr(L.dza), L.dB.data_ptr(), L.dsb.data_ptr(),
                  _ptr(L.dbias), flat.data_ptr() + shift_y * flat.element_size(), L.M, ws.data_ptr(), nbytes,
                  q.current_stream())
    torch.cuda.synchronize()
    body = flat[shift_y:shift_y + L.M * ldy].view(L.M, ldy)
    assert (flat[:shift_y] == 77).all() and (flat[shift_y + L.M * ldy:] == 77).all()
    assert (body[:, cols:] == 77).all()  # elements between the rows
    return body[:, :cols]


MS = [1, 2, 15, 16, 17, 31, 33, 63, 64, 65, 100, 127, 129, 257, 300]
NS = [1, 3, 15, 16, 17, 33, 64, 100, 130, 255, 256, 257, 513]
KS = [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 192, 320, 640, 1000, 1025, 4100]


@pytest.mark.parametrize("case", range(60))
def test_integer_sums_are_exact(qdg, case):
    rng = np.random.default_rng(case)
    M, n, k = MS[case % len(MS)], NS[(case * 5 + 2) % len(NS)], KS[(case * 7 + 3) % len(KS)]
    L = Layer(rng, M, n, k, zeros=bool(case & 1), bias=False, pad_a=case % 3, pad_b=(case // 2) % 2)
    y = _dense(L, q.QDG_O_I32, pad_y=(0, 1, 4)[case % 3], shift_y=(0, 0, 1)[case % 3])
    np.testing.assert_array_equal(y.cpu().numpy(), ops.int_product(L.a, L.b[0], L.za))


@pytest.mark.parametrize("otype", ["bf16", "f32"])
@pytest.mark.parametrize("epi", [q.QDG_EPI_NONE, q.QDG_EPI_SILU_MUL])
@pytest.mark.parametrize("M,n,k", [(1, 2, 1), (1, 128, 512), (3, 62, 100), (16, 256, 1024), (17, 514, 640), (48, 96, 2048),
                                   (65, 130, 333), (128, 512, 256), (200, 770, 1100), (513, 1026, 129)])
def test_scales_bias_epilogue(qdg, otype, epi, M, n, k):
    code = q.QDG_O_BF16 if otype == "bf16" else q.QDG_O_F32
    for v in range(4):
        rng = np.random.default_rng(M * 7 + n + v)
        L = Layer(rng, M, n, k, zeros=bool(v & 1), bias=bool(v & 2))
        if epi:  # gates in the range where silu bends
            L.sb /= np.float32(np.sqrt(k) * 5)
            L.dsb = H.dev(L.sb)
        y = _dense(L, code, epi, pad_y=(0, 2, 3, 4)[v], shift_y=(0, 1, 0, 4)[v])
        y64, err = L.ref(epi)
        _close(y, y64, err, otype == "bf16")


@pytest.mark.parametrize("M,n", [(1, 5), (64, 70), (150, 300)])
def test_largest_sums(qdg, M, n):
    """k = 65536 with every code -128 and zero points 127: 255 * 128 * 65536, next to the end of int32."""
    L = Layer(np.random.default_rng(0), M, n, 65536, zeros=True, bias=False, extremes=True)
    y = _dense(L, q.QDG_O_I32)
    assert (y == 255 * 128 * 65536).all()


@pytest.mark.parametrize("M,n,k", [(1, 64, 65536), (16, 512, 16384), (40, 128, 8192), (70, 48, 30000), (130, 96, 16400)])
def test_long_k_with_few_columns(qdg, M, n, k):
    rng = np.random.default_rng(k)
    L = Layer(rng, M, n, k, zeros=True, bias=True)
    np.testing.assert_array_equal(_dense(L, q.QDG_O_I32).cpu().numpy(), ops.int_product(L.a, L.b[0], L.za))
    y64, err = L.ref(q.QDG_EPI_NONE)
    _close(_dense(L, q.QDG_O_F32), y64, err, False)
    y64, err = L.ref(q.QDG_EPI_SILU_MUL)
    _close(_dense(L, q.QDG_O_F32, q.QDG_EPI_SILU_MUL), y64, err, False)


@pytest.mark.parametrize("M,n,k", [(5, 40, 200), (70, 200, 300), (60, 128, 16400)])
def test_raw_output_reads_no_scales(qdg, M, n, k):
    L = Layer(np.random.default_rng(3), M, n, k, zeros=True, bias=False)
    cfg = L.cfg(q.QDG_O_I32, q.QDG_EPI_NONE)
    y = torch.zeros((M, n), dtype=torch.int32, device="cuda")
    nbytes = q.qdg_gemm_i8_workspace(cfg, M)
    ws = torch.zeros(max(nbytes, 16), dtype=torch.uint8, device="cuda")
    q.qdg_gemm_i8(cfg, L.dA.data_ptr(), None, L.dza.data_ptr(), L.dB.data_ptr(), None, None, y.data_ptr(), M,
                  ws.data_ptr(), nbytes, q.current_stream())
    torch.cuda.synchronize()
    np.testing.assert_array_equal(y.cpu().numpy(), ops.int_product(L.a, L.b[0], L.za))


def test_every_tile_and_a_split_at_odd_sizes(qdg):
    """Sizes for which the time model takes each kernel: rows, 64 x 64 (whole and split), 128 x 64, 128 x 128,
    128 x 256 and 256 x 256 tiles; every row and column is compared."""
    assert q.qdg_gemm_i8_workspace(q.gemm_i8(500, 16385), 33) > 0  # the split
    for M, n, k in ((16, 4099, 130), (33, 500, 16385), (200, 1030, 515), (130, 4100, 2050), (257, 7300, 1030),
                    (513, 14337, 700), (2049, 4099, 1027), (4097, 5000, 515), (4096, 4610, 900)):
        rng = np.random.default_rng(M)
        L = Layer(rng, M, n, k, zeros=True, bias=False)
        a = L.dA[:, :k].float() - L.dza.float()[:, None]
        want = (a.double() @ L.dB[:, :k].double().t()).to(torch.int32)
        got = _dense(L, q.QDG_O_I32, pad_y=3)
        assert torch.equal(got, want), (M, n, k)


@pytest.mark.parametrize("epi", [q.QDG_EPI_NONE, q.QDG_EPI_SILU_MUL])
def test_columns_behind_whole_rounds_of_tiles(qdg, epi):
    """4096 x 4620 columns are one round of 256 x 256 tiles and a rest in another tile."""
    M, n, k = 4096, 4620, 600
    L = Layer(np.random.default_rng(9), M, n, k, zeros=True, bias=True)
    L.sb /= np.float32(np.sqrt(k) * 5)
    L.dsb = H.dev(L.sb)
    y = _dense(L, q.QDG_O_F32, epi)
    for rows in (slice(0, 40), slice(2040, 2080), slice(4060, 4096)):  # every column of these
        y64, err = L.ref(epi, rows)
        _close(y[rows], y64, err, False)


@pytest.mark.parametrize("epi", [q.QDG_EPI_NONE, q.QDG_EPI_SILU_MUL])
def test_rows_do_not_depend_on_the_batch(qdg, epi):
    rng = np.random.default_rng(21)
    L = Layer(rng, 300, 384, 1000, zeros=True, bias=True)
    full = _dense(L, q.QDG_O_F32, epi)
    for m in (1, 16, 40, 64, 65, 128, 200):
        S = Layer.__new__(Layer)
        S.__dict__.update(L.__dict__)
        S.M = m
        assert torch.equal(_dense(S, q.QDG_O_F32, epi), full[:m])


def test_split_product_in_two_graphs(qdg):
    """Two captured products with a workspace each, replayed in turn with eager work between."""
    rng = np.random.default_rng(23)
    sides = []
    for M in (33, 40):
        L = Layer(rng, M, 256, 16400, zeros=True, bias=True)
        cfg = L.cfg(q.QDG_O_F32, q.QDG_EPI_NONE)
        nbytes = q.qdg_gemm_i8_workspace(cfg, M)
        assert nbytes > 0
        ws = torch.zeros(nbytes, dtype=torch.uint8, device="cuda")
        y = torch.zeros((M, 256), device="cuda")
        want = _dense(L, q.QDG_O_F32).clone()
        call = lambda st, L=L, cfg=cfg, ws=ws, y=y, nbytes=nbytes: q.qdg_gemm_i8(
            cfg, L.dA.data_ptr(), L.dsa.data_ptr(), L.dza.data_ptr(), L.dB.data_ptr(), L.dsb.data_ptr(),
            L.dbias.data_ptr(), y.data_ptr(), L.M, ws.data_ptr(), nbytes, st)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call(q.current_stream())
        sides.append((L, call, g, y, want))
    for _ in range(4):
        for L, call, g, y, want in sides:
            y.zero_()
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(y, want)
            y.fill_(7.0)
            call(q.current_stream())
            torch.cuda.synchronize()
            assert torch.equal(y, want)


def test_unusual_scales(qdg):
    """Scales whose product leaves binary32's range while the result does not."""
    L = Layer(np.random.default_rng(2), 20, 40, 64, zeros=False, bias=False)
    L.sa[:], L.sb[:] = 1e-30, 1e30
    L.a[3] = 0
    L.sa[3] = 1e38
    L.dA, L.dsa, L.dsb = _dev_codes(L.a, L.lda, 1), H.dev(L.sa), H.dev(L.sb)
    y64, err = L.ref(q.QDG_EPI_NONE)
    _close(_dense(L, q.QDG_O_F32), y64, err, False)


def test_offsets_past_32_bits(qdg):
    """A, B and Y each longer than 4 GiB: their last rows."""
    k, ld = 128, 65536
    rows = (1 << 32) // ld + 300
    rng = np.random.default_rng(4)
    tail = rng.integers(-128, 128, (40, k)).astype(np.int8)
    few = rng.integers(-128, 128, (24, k)).astype(np.int8)
    big = torch.zeros((rows, ld), dtype=torch.int8, device="cuda")
    big[-40:, :k] = H.dev(tail)
    small = H.dev(few)
    ones = torch.ones(rows, device="cuda")
    want = ops.int_product(tail, few)
    # long A, long Y
    ldy = (1 << 31) // rows + 40
    Y = torch.zeros((rows, ldy), dtype=torch.int32, device="cuda")
    cfg = q.gemm_i8(24, k, lda=ld, ldb=k, ldy=ldy, otype=q.QDG_O_I32)
    q.qdg_gemm_i8(cfg, big.data_ptr(), ones.data_ptr(), None, small.data_ptr(), ones.data_ptr(), None, Y.data_ptr(),
                  rows, None, 0, q.current_stream())
    torch.cuda.synchronize()
    np.testing.assert_array_equal(Y[-40:, :24].cpu().numpy(), want)
    assert int(Y[:-40].abs().max()) == 0 and int(Y[:, 24:].abs().max()) == 0
    del Y
    # long B
    Z = torch.zeros((24, rows), dtype=torch.int32, device="cuda")
    cfg = q.gemm_i8(rows, k, lda=k, ldb=ld, otype=q.QDG_O_I32)
    q.qdg_gemm_i8(cfg, small.data_ptr(), ones.data_ptr(), None, big.data_ptr(), ones.data_ptr(), None, Z.data_ptr(),
                  24, None, 0, q.current_stream())
    torch.cuda.synchronize()
    np.testing.assert_array_equal(Z[:, -40:].cpu().numpy(), want.T)
    assert int(Z[:, :-40].abs().max()) == 0


# ---------------------------------------------------------------- grouped by expert

def _align(ids, E, bm):
    t, top_k = ids.shape
    cap = q.qdg_moe_align_capacity(t, top_k, E, bm)
    sid = torch.empty(cap, dtype=torch.int32, device="cuda")
    blk = torch.empty(cap // bm, dtype=torch.int32, device="cuda")
    npad = torch.zeros(1, dtype=torch.int32, device="cuda")
    q.qdg_moe_align(H.dev(ids.astype(np.int32)).data_ptr(), t, top_k, E, bm, sid.data_ptr(), blk.data_ptr(),
                    npad.data_ptr(), q.current_stream())
    torch.cuda.synchronize()
    return sid, blk, npad


def _grouped(L, ids, bm, per_pair, otype, epi=q.QDG_EPI_NONE):
    t, top_k = ids.shape
    sid, blk, npad = _align(ids, L.experts, bm)
    cols = L.n // 2 if epi else L.n
    dt = {q.QDG_O_BF16: torch.bfloat16, q.QDG_O_F32: torch.float32, q.QDG_O_I32: torch.int32}[otype]
    y = torch.full((t * top_k + 1, cols), 77, dtype=dt, device="cuda")
    q.qdg_moe_gemm_i8(L.cfg(otype, epi), L.dA.data_ptr(), L.dsa.data_ptr(), _ptr(L.dza), L.dB.data_ptr(),
                      L.dsb.data_ptr(), _ptr(L.dbias), sid.data_ptr(), blk.data_ptr(), npad.data_ptr(), t, top_k, bm,
                      int(per_pair), y.data_ptr(), q.current_stream())
    torch.cuda.synchronize()
    assert (y[t * top_k:] == 77).all()
    return y[:t * top_k]


@pytest.mark.parametrize("bm", [16, 32, 64, 128])
@pytest.mark.parametrize("per_pair", [False, True])
@pytest.mark.parametrize("T,E,top_k,n,k", [(1, 8, 2, 64, 128), (5, 3, 3, 34, 100), (64, 16, 4, 130, 640),
                                           (200, 4, 2, 514, 257), (37, 60, 6, 96, 2000), (300, 2, 1, 258, 64)])
def test_grouped(qdg, bm, per_pair, T, E, top_k, n, k):
    rng = np.random.default_rng(T * 100 + bm + n)
    ids = np.stack([rng.permutation(E)[:top_k] for _ in range(T)])
    rows = T * top_k if per_pair else T
    flat = ids.reshape(-1)
    arow = np.arange(T * top_k) if per_pair else np.arange(T * top_k) // top_k
    for zeros, bias in ((False, True), (True, False)):
        L = Layer(rng, rows, n, k, zeros, bias, experts=E)
        y = _grouped(L, ids, bm, per_pair, q.QDG_O_I32).cpu().numpy()
        for e in range(E):
            pairs = np.nonzero(flat == e)[0]
            r = arow[pairs]
            np.testing.assert_array_equal(y[pairs], ops.int_product(L.a[r], L.b[e], None if L.za is None else L.za[r]))
        L.sb /= np.float32(np.sqrt(k) * 5)
        L.dsb = H.dev(L.sb)
        for otype, epi in ((q.QDG_O_BF16, q.QDG_EPI_NONE), (q.QDG_O_F32, q.QDG_EPI_SILU_MUL), (q.QDG_O_BF16, q.QDG_EPI_SILU_MUL)):
            y = _grouped(L, ids, bm, per_pair, otype, epi)
            for e in range(E):
                pairs = np.nonzero(flat == e)[0]
                y64, err = L.ref(epi, arow[pairs], e)
                _close(y[torch.from_numpy(pairs).cuda()], y64, err, otype == q.QDG_O_BF16)


def test_grouped_leaves_out_bad_ids(qdg):
    """An id outside [0, E) has no block: its row stays as it was."""
    rng = np.random.default_rng(8)
    ids = rng.integers(0, 4, (9, 2))
    ids[3, 1], ids[5, 0] = -1, 4
    L = Layer(rng, 9, 48, 96, zeros=True, bias=False, experts=4)
    y = _grouped(L, ids, 16, False, q.QDG_O_I32).cpu().numpy()
    for p, e in enumerate(ids.reshape(-1)):
        if 0 <= e < 4:
            np.testing.assert_array_equal(y[p], ops.int_product(L.a[p // 2:p // 2 + 1], L.b[e], L.za[p // 2:p // 2 + 1])[0])
        else:
            assert (y[p] == 77).all()


# ---------------------------------------------------------------- asymmetric quantizer

def _quantize(x, lda, ldq):
    """x: bf16 bits [M][k]."""
    M, k = x.shape
    buf = np.full((M, lda), 0x7F80, np.uint16)  # +infinity behind each row's end
    buf[:, :k] = x
    a = H.bf16_dev(buf)
    qa = torch.full((M + 1, ldq), 99, dtype=torch.int8, device="cuda")
    s = torch.full((M + 1,), -5.0, device="cuda")
    z = torch.full((M + 1,), 999, dtype=torch.int32, device="cuda")
    q.qdg_quantize_act_zp(a.data_ptr(), lda, M, k, qa.data_ptr(), ldq, s.data_ptr(), z.data_ptr(), q.current_stream())
    torch.cuda.synchronize()
    assert (qa[M] == 99).all() and (qa[:, k:] == 99).all() and float(s[M]) == -5.0 and int(z[M]) == 999
    return qa[:M, :k].cpu().numpy(), s[:M].cpu().numpy(), z[:M].cpu().numpy()


def _check_quant(x, pad=0):
    k = x.shape[1]
    got = _quantize(x, (k + 7) // 8 * 8 + 8 * pad, (k + 15) // 16 * 16 + 16 * pad)
    want = ops.quantize_act_zp(codecs.bf16_bits_to_f64(x))
    np.testing.assert_array_equal(got[2], want[2])
    np.testing.assert_array_equal(got[1], want[1])
    np.testing.assert_array_equal(got[0], want[0])


@pytest.mark.parametrize("k", [1, 2, 7, 8, 9, 15, 17, 64, 100, 511, 512, 513, 2048, 2049, 4100, 14336, 20000, 40003])
def test_quantizer_matches_bit_for_bit(qdg, k):
    rng = np.random.default_rng(k)
    for M, pad in ((1, 0), (7, 2), (33, 1)):
        x = rng.standard_normal((M, k)) * np.exp(rng.uniform(-20, 20, (M, 1)))
        x[::3] = np.maximum(x[::3], 0)          # one side only
        x[1::5] = -np.abs(x[1::5])
        x[2::4] += 100.0 * np.abs(x).max()  # far from zero
        _check_quant(codecs.f32_to_bf16_bits(x.astype(np.float32)), pad)


def test_quantizer_borders(qdg):
    """Values on and next to the border between two codes, in whole and in odd scales."""
    rows = []
    for top in (255.0, 127.5, 85.0, 51.0, 1.0, 3.0):
        step = top / 255.0
        v = (np.arange(0, 256) + 0.5) * step
        rows.append(np.concatenate([[0.0, top], v, v * (1 + 2.0 ** -8), v * (1 - 2.0 ** -8)]))
        rows.append(np.concatenate([[-top / 3, top * 2 / 3], v - top / 3, v * (1 + 2.0 ** -8) - top / 3, v - top / 3]))
    _check_quant(codecs.f32_to_bf16_bits(np.clip(np.array(rows), -255, 255).astype(np.float32)))


def test_quantizer_special_rows(qdg):
    rng = np.random.default_rng(6)
    x = codecs.f32_to_bf16_bits(rng.standard_normal((14, 300)).astype(np.float32))
    x[0] = 0
    x[1] = 0x8000                     # -0
    x[2, 5], x[2, 70] = 0x7FC0, 0xFFC1  # NaN
    x[3, 9], x[3, 100] = 0x7F80, 0xFF80  # infinities
    x[4] = 0x7FC0
    x[5] = 0x7F80
    x[6] = 0xFF80
    x[7] = rng.integers(1, 128, 300)  # subnormal
    x[8, 0], x[8, 1] = 0x7F7F, 0xFF7F  # the type's ends: hi - lo leaves binary32
    x[9] = 0x0001
    x[10] = 0x7F7F
    x[11] = 0x3F80
    x[12] = 0xBF80
    x[13, 1:] = 0
    _check_quant(x)


# ---------------------------------------------------------------- together

def test_moe_block(qdg):
    """hidden -> quantize -> route -> align -> gate+up with SiLU*mul -> quantize -> down -> combine, every step on
    the device's output of the one before, captured and replayed on new inputs with eager work between."""
    T, E, top_k, hid, inter, bm = 45, 12, 3, 264, 200, 32
    rng = np.random.default_rng(31)
    W1 = Layer(rng, 1, 2 * inter, hid, False, True, experts=E)
    W2 = Layer(rng, 1, hid, inter, False, False, experts=E)
    for W in (W1, W2):
        W.sb /= np.float32(8.0)
        W.dsb = H.dev(W.sb)
    pairs = T * top_k
    ldh, ldi = 272, 208
    hidden = torch.zeros((T, hid), dtype=torch.bfloat16, device="cuda")
    logits = torch.zeros((T, E), dtype=torch.bfloat16, device="cuda")
    bias = H.dev((0.1 * rng.standard_normal(E)).astype(np.float32))
    cap = q.qdg_moe_align_capacity(T, top_k, E, bm)
    new = lambda *s, dt=torch.int32: torch.zeros(s, dtype=dt, device="cuda")
    qa, sa, za = new(T, ldh, dt=torch.int8), new(T, dt=torch.float32), new(T)
    ids, w = new(T, top_k), new(T, top_k, dt=torch.float32)
    sid, blk, npad = new(cap), new(cap // bm), new(1)
    h = new(pairs, inter, dt=torch.bfloat16)
    qh, sh, zh = new(pairs, ldi, dt=torch.int8), new(pairs, dt=torch.float32), new(pairs)
    yp, out = new(pairs, hid, dt=torch.bfloat16), new(T, hid, dt=torch.float32)
    rcfg = q.route(E, top_k, score=q.QDG_SCORE_SIGMOID, num_groups=4, topk_groups=2, group_score=q.QDG_GROUP_TOP2,
                   renormalize=1, scale=2.5)
    c1 = q.gemm_i8(2 * inter, hid, lda=ldh, ldb=W1.ldb, num_experts=E, epilogue=q.QDG_EPI_SILU_MUL)
    c2 = q.gemm_i8(hid, inter, lda=ldi, ldb=W2.ldb, num_experts=E)

    def block(st):
        q.qdg_quantize_act_zp(hidden.data_ptr(), hid, T, hid, qa.data_ptr(), ldh, sa.data_ptr(), za.data_ptr(), st)
        q.qdg_moe_route(rcfg, logits.data_ptr(), E, bias.data_ptr(), T, ids.data_ptr(), w.data_ptr(), st)
        q.qdg_moe_align(ids.data_ptr(), T, top_k, E, bm, sid.data_ptr(), blk.data_ptr(), npad.data_ptr(), st)
        q.qdg_moe_gemm_i8(c1, qa.data_ptr(), sa.data_ptr(), za.data_ptr(), W1.dB.data_ptr(), W1.dsb.data_ptr(),
                          W1.dbias.data_ptr(), sid.data_ptr(), blk.data_ptr(), npad.data_ptr(), T, top_k, bm, 0,
                          h.data_ptr(), st)
        q.qdg_quantize_act_zp(h.data_ptr(), inter, pairs, inter, qh.data_ptr(), ldi, sh.data_ptr(), zh.data_ptr(), st)
        q.qdg_moe_gemm_i8(c2, qh.data_ptr(), sh.data_ptr(), zh.data_ptr(), W2.dB.data_ptr(), W2.dsb.data_ptr(), None,
                          sid.data_ptr(), blk.data_ptr(), npad.data_ptr(), T, top_k, bm, 1, yp.data_ptr(), st)
        q.qdg_moe_combine_bf16(yp.data_ptr(), w.data_ptr(), T, top_k, hid, out.data_ptr(), q.QDG_O_F32, st)

    def fresh():
        hidden.copy_(torch.from_numpy(rng.standard_normal((T, hid)).astype(np.float32)))
        logits.copy_(torch.from_numpy(rng.standard_normal((T, E)).astype(np.float32)))

    def verify():
        torch.cuda.synchronize()
        cq, cs, cz = ops.quantize_act_zp(hidden.float().cpu().numpy())
        np.testing.assert_array_equal(qa[:, :hid].cpu().numpy(), cq)
        np.testing.assert_array_equal(za.cpu().numpy(), cz)
        rid, rw, _ = ops.route(logits.float().cpu().numpy(), top_k, "sigmoid", bias.cpu().numpy(), 4, 2, "top2", True, 2.5)
        np.testing.assert_array_equal(ids.cpu().numpy(), rid)
        flat = rid.reshape(-1)
        hq, hs, hz = ops.quantize_act_zp(h.float().cpu().numpy())
        np.testing.assert_array_equal(qh[:, :inter].cpu().numpy(), hq)
        for e in range(E):
            p = np.nonzero(flat == e)[0]
            sel = torch.from_numpy(p).cuda()
            y64, err = ops.gemm_i8(cq[p // top_k], cs[p // top_k], W1.b[e], W1.sb[e], cz[p // top_k], W1.bias[e], True)
            _close(h[sel], y64, err, True)
            y64, err = ops.gemm_i8(hq[p], hs[p], W2.b[e], W2.sb[e], hz[p])
            _close(yp[sel], y64, err, True)
        # top_k products and sums of binary32 on the rows of yp: at most 2 * top_k half steps of sum |w y|
        rows = H.to_f64(yp).reshape(T, top_k, hid)
        want = ref.moe_combine(H.to_f64(yp), w.cpu().numpy(), top_k)
        slack = 2 * top_k * 2.0 ** -24 * np.einsum("tj,tjc->tc", np.abs(w.cpu().numpy().astype(np.float64)), np.abs(rows))
        assert np.all(np.abs(H.to_f64(out) - want) <= slack + 1e-30)

    fresh()
    block(q.current_stream())
    verify()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        block(q.current_stream())
    for _ in range(3):
        fresh()
        for t in (qa, h, qh, yp, out, ids, sid):
            t.zero_()
        g.replay()
        verify()


def test_two_streams_with_their_own_workspaces(qdg):
    rng = np.random.default_rng(41)
    L = Layer(rng, 8, 256, 16384, zeros=True, bias=True)
    cfg = L.cfg(q.QDG_O_F32, q.QDG_EPI_NONE)
    nbytes = q.qdg_gemm_i8_workspace(cfg, L.M)
    want = _dense(L, q.QDG_O_F32)
    streams = [torch.cuda.Stream() for _ in range(2)]
    ys = [torch.zeros((L.M, L.n), device="cuda") for _ in streams]
    wss = [torch.zeros(max(nbytes, 16), dtype=torch.uint8, device="cuda") for _ in streams]
    torch.cuda.synchronize()
    for _ in range(5):
        for st, y, ws in zip(streams, ys, wss):
            q.qdg_gemm_i8(cfg, L.dA.data_ptr(), L.dsa.data_ptr(), _ptr(L.dza), L.dB.data_ptr(), L.dsb.data_ptr(),
                          _ptr(L.dbias), y.data_ptr(), L.M, ws.data_ptr(), nbytes, st.cuda_stream)
    torch.cuda.synchronize()
    for y in ys:
        assert torch.equal(y, want)


def test_one_workspace_for_every_batch(qdg):
    """The bytes asked for the largest batch, which is not split itself, serve the smaller ones that are."""
    n, k, rows = 2050, 16400, 600
    L = Layer(np.random.default_rng(51), rows, n, k, zeros=True, bias=False)
    cfg = L.cfg(q.QDG_O_I32, q.QDG_EPI_NONE)
    nbytes = q.qdg_gemm_i8_workspace(cfg, rows)
    assert nbytes > 0
    ws = torch.full((nbytes + 256,), 0x5A, dtype=torch.uint8, device="cuda")
    want = ops.int_product(L.a, L.b[0], L.za)
    for M in (1, 17, 33, 64, 65, 128, 129, 300, 600):
        y = torch.full((M + 1, n), 77, dtype=torch.int32, device="cuda")
        q.qdg_gemm_i8(cfg, L.dA.data_ptr(), L.dsa.data_ptr(), L.dza.data_ptr(), L.dB.data_ptr(), L.dsb.data_ptr(),
                      None, y.data_ptr(), M, ws.data_ptr(), nbytes, q.current_stream())
        torch.cuda.synchronize()
        np.testing.assert_array_equal(y[:M].cpu().numpy(), want[:M])
        assert (y[M] == 77).all() and (ws[nbytes:] == 0x5A).all()
