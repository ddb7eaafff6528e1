"""Every kernel that qdg_gemm_i8 may choose, named by qdg_gemm_i8_describe, with
and without zero points and bias, in every output type, with and without
SiLU*mul, at odd sizes with several groups of K and a cut one: int32 outputs
equal, f32 and bf16 within the bound of oracle.ops.gemm_i8; rows that do not
depend on the batch across the tiles; workspaces."""

import numpy as np
import pytest
import torch

import quantized_dequant_gemm_amd as q
from oracle import ops

pytestmark = pytest.mark.gpu

NONE, SILU = q.QDG_EPI_NONE, q.QDG_EPI_SILU_MUL
DT = {q.QDG_O_BF16: torch.bfloat16, q.QDG_O_F32: torch.float32, q.QDG_O_I32: torch.int32}


class Operands:
    def __init__(self, seed, M, n, k):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        ld = (k + 15) // 16 * 16
        codes = lambda rows: torch.randint(-128, 128, (rows, ld), generator=g, device="cuda", dtype=torch.int8)
        self.M, self.n, self.k, self.ld = M, n, k, ld
        self.A, self.B = codes(M), codes(n)  # bytes behind k are codes too
        self.za = torch.randint(-128, 128, (M,), generator=g, device="cuda", dtype=torch.int32)
        self.sa = torch.rand(M, generator=g, device="cuda") * 0.05 + 0.001
        # gates in the range where silu bends
        self.sb = (torch.rand(n, generator=g, device="cuda") * 9e-4 + 1e-4) / (5 * k ** 0.5)
        self.bias = torch.randn(n, generator=g, device="cuda")

    def cfg(self, otype, epi):
        return q.gemm_i8(self.n, self.k, lda=self.ld, ldb=self.ld, otype=otype, epilogue=epi)

    def call(self, M, otype, epi, zeros, bias, ws_bytes=None, first=0):
        """Rows first .. first + M - 1 of the batch as a product of their own."""
        cfg = self.cfg(otype, epi)
        cols = self.n // 2 if epi else self.n
        y = torch.full((M + 1, cols), 77, dtype=DT[otype], device="cuda")
        need = q.qdg_gemm_i8_workspace(cfg, M) if ws_bytes is None else ws_bytes
        ws = torch.full((max(16, need),), 0x5A, dtype=torch.uint8, device="cuda")
        q.qdg_gemm_i8(cfg, self.A[first:].data_ptr(), self.sa[first:].data_ptr(), self.za[first:].data_ptr() if zeros else None,
                      self.B.data_ptr(), self.sb.data_ptr(), self.bias.data_ptr() if bias else None, y.data_ptr(), M,
                      ws.data_ptr(), need, q.current_stream())
        torch.cuda.synchronize()
        assert (y[M] == 77).all()
        return y[:M]

    def sums(self, zeros):
        """The integer sums, exact in float64."""
        a = self.A[:, :self.k].double()
        if zeros:
            a -= self.za.double()[:, None]
        return a @ self.B[:, :self.k].double().t()

    def ref(self, sums, epi, bias):
        """The value and bound of oracle.ops.gemm_i8, on the device."""
        p = sums * self.sa.double()[:, None] * self.sb.double()
        b = self.bias.double() if bias else torch.zeros_like(self.sb).double()
        y, err = p + b, 4 * 2.0 ** -24 * (p.abs() + b.abs())
        if not epi:
            return y, err
        i = self.n // 2
        g, u, eg, eu = y[:, :i], y[:, i:], err[:, :i], err[:, i:]
        s = g / (1.0 + torch.exp(-g))
        return s * u, 2.0 ** -20 * (s * u).abs() + 1.1 * eg * (u.abs() + eu) + s.abs() * eu


def _record(M, n, k, epi=NONE):
    return q.qdg_gemm_i8_describe(q.gemm_i8(n, k, epilogue=epi), M)


def _kernel(record):
    f = dict(w.split("=") for w in record.split() if "=" in w)
    name = "rows" if f["family"] == "rows" else f["block_m"] + "x" + f["block_n"]
    return name + ("/" + f["split_k"] if f["split_k"] != "1" else "") + ("+" + f["rest"] if f["rest"] != "none" else "")


CASES = [("rows", 13, 4098, 1030), ("64x64", 129, 1026, 1030), ("64x64/8", 33, 514, 16386), ("128x64", 250, 4100, 4090),
         ("128x64", 193, 4098, 1030), ("128x64/8", 65, 1026, 40001), ("128x128", 257, 7302, 1030),
         ("128x128/8", 65, 2050, 40001), ("128x256", 513, 9002, 1030), ("256x256", 1025, 9002, 1030),
         ("256x256/8", 193, 4098, 40001), ("128x128+64x64", 1025, 4098, 1030), ("128x256+64x64", 2049, 4098, 1030),
         ("256x256+128x128", 4096, 4610, 900), ("256x256+128x256", 4097, 5000, 515)]


@pytest.mark.parametrize("kernel,M,n,k", CASES)
def test_every_dense_kernel(qdg, kernel, M, n, k):
    assert _kernel(_record(M, n, k)) == kernel
    assert _kernel(_record(M, n, k, SILU)) == kernel
    o = Operands(M + n, M, n, k)
    for zeros in (False, True):
        sums = o.sums(zeros)
        some = [0, M // 2, M - 1]
        want = ops.int_product(o.A[some, :k].cpu().numpy(), o.B[:, :k].cpu().numpy(),
                               o.za[some].cpu().numpy() if zeros else None)
        np.testing.assert_array_equal(sums[some].cpu().numpy(), want)
        assert torch.equal(o.call(M, q.QDG_O_I32, NONE, zeros, False), sums.to(torch.int32))
        for epi in (NONE, SILU):
            for bias in (False, True):
                y64, err = o.ref(sums, epi, bias)
                for otype in (q.QDG_O_F32, q.QDG_O_BF16):
                    # bf16: half a step (2^-8) of the value; f32: the one rounding of y64 itself
                    slack = err + (2.0 ** -8 * (y64.abs() + err) if otype == q.QDG_O_BF16 else 2.0 ** -24 * y64.abs())
                    y = o.call(M, otype, epi, zeros, bias).double()
                    assert bool(((y - y64).abs() <= slack + 2.0 ** -126).all()), (kernel, zeros, epi, bias, otype)


@pytest.mark.parametrize("otype", [q.QDG_O_F32, q.QDG_O_BF16])
@pytest.mark.parametrize("epi", [NONE, SILU])
@pytest.mark.parametrize("zeros", [False, True])
def test_rows_do_not_depend_on_the_tile(qdg, otype, epi, zeros):
    n, k = 4610, 900
    o = Operands(5, 4097, n, k)
    full = o.call(4097, otype, epi, zeros, True)
    seen = set()
    for m in (1, 16, 33, 193, 449, 900, 1025, 2049, 4096):
        seen.add(_kernel(_record(m, n, k, epi)))
        for first in (0, 4097 - m):
            assert torch.equal(o.call(m, otype, epi, zeros, True, first=first), full[first:first + m]), (m, first)
    assert {"rows", "64x64", "128x64", "128x128", "128x256", "256x256"} <= seen


def test_two_streams_with_a_split_each(qdg):
    """Two split products with inputs and a workspace of their own, on two streams at once."""
    n, k = 514, 16386
    runs = []
    for i, M in enumerate((33, 40)):
        o = Operands(60 + i, M, n, k)
        cfg = o.cfg(q.QDG_O_F32, NONE)
        need = q.qdg_gemm_i8_workspace(cfg, M)
        assert need > 0 and _kernel(_record(M, n, k)) == "64x64/8"
        want = o.call(M, q.QDG_O_F32, NONE, True, True)
        runs.append((o, cfg, need, want, torch.empty(need, dtype=torch.uint8, device="cuda"),
                     torch.zeros((8, M, n), device="cuda"), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for i in range(8):
        for o, cfg, need, want, ws, ys, st in runs:
            q.qdg_gemm_i8(cfg, o.A.data_ptr(), o.sa.data_ptr(), o.za.data_ptr(), o.B.data_ptr(), o.sb.data_ptr(),
                          o.bias.data_ptr(), ys[i].data_ptr(), o.M, ws.data_ptr(), need, st.cuda_stream)
    torch.cuda.synchronize()
    for o, cfg, need, want, ws, ys, st in runs:
        for i in range(8):
            assert torch.equal(ys[i], want)
