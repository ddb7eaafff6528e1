"""qdg_lora: values at which the inner sums' way into the second product shows. Every case runs through the kernel that
does both products, the one for few rows and the one for many, each with and without cut loads."""

import numpy as np
import pytest
import torch

import quantized_dequant_gemm_amd as q
from tests import gpu_helpers as H
from tests.test_gpu_lora import Group, Pool, _ptr, _run

pytestmark = pytest.mark.gpu

# (rows, block_m, k): one launch; two launches with few rows; with 64 rows at once
PATHS = {"fused": (5, 16, 128), "fused cut": (5, 16, 72), "up": (20, 16, 4224), "up cut": (20, 16, 4168),
         "wide": (70, 64, 4224), "wide cut": (70, 64, 4168)}


def _bf16(x):
    with np.errstate(over="ignore"):
        return torch.from_numpy(np.ascontiguousarray(x, np.float32)).cuda().to(torch.bfloat16)


def _lora(path, x, a, b, y, f32, scales=None):
    """x [k'], a [R][k'], b [n][R], y [n]: every row of the call is this one, k' filled up with zeros. Returns the rows."""
    M, bm, k = PATHS[path]
    rank, n = a.shape[0], b.shape[0]
    full = np.zeros((M, k))
    full[:, :x.size] = x
    fa = np.zeros((1, 1, rank, k))
    fa[0, 0, :, :x.size] = a
    dx, da, db = _bf16(full), _bf16(fa), _bf16(b[None])
    dy = torch.from_numpy(np.tile(np.asarray(y, np.float32), (M, 1))).cuda().to(torch.float32 if f32 else torch.bfloat16)
    ds = None if scales is None else H.dev(np.asarray(scales, np.float32))
    g = Group(np.zeros(M, np.int32), 1, bm)
    cfg = q.lora(n, k, rank, otype=q.QDG_O_F32 if f32 else q.QDG_O_BF16)
    nbytes = q.qdg_lora_workspace(cfg, M, bm)
    assert (nbytes == 0) == path.startswith("fused")
    ws = torch.full((max(16, nbytes),), 0xFF, dtype=torch.uint8, device="cuda")
    q.qdg_lora(cfg, dx.data_ptr(), da.data_ptr(), db.data_ptr(), None, _ptr(ds), *g.args(), dy.data_ptr(), ws.data_ptr(),
               nbytes, q.current_stream())
    torch.cuda.synchronize()
    got = H.to_f64(dy)
    np.testing.assert_array_equal(got, np.tile(got[:1], (M, 1)))
    return got[0]


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("path", list(PATHS))
def test_inner_sums_keep_all_bits_of_binary32(qdg, path, f32):
    """T of 24 significant bits: Y is T times a power of two, and of two inner sums that differ in their last eight bits
    only the difference, so that a lost, doubled or misplaced term of T shows."""
    rng = np.random.default_rng(7)
    n = 200
    x = np.array([1.0, 2.0 ** -8, 2.0 ** -16])
    for rank in (2, 8, 18, 34, 64):
        if path.startswith("fused") and rank > 32:
            continue
        a = np.zeros((rank, 3))
        r0, r1 = rng.choice(rank, 2, replace=False)
        a[r0] = 2 * rng.integers(64, 128, 3) + 1  # 128 to 255, odd: every bit of the 24 counts
        a[r1] = -a[r0, 0], -a[r0, 1], 0.0
        t = a @ x
        b = np.zeros((n, rank))
        power = 2.0 ** rng.integers(-20, 20, n)
        b[:, r0] = power
        # one inner sum: exact in binary32; two additions inside the product, each off by a step at most
        got = _lora(path, x, a, b, np.zeros(n), f32)
        assert np.all(np.abs(got - t[r0] * power) <= (2.0 ** -22 + (0 if f32 else 2.0 ** -8)) * t[r0] * power)
        # two that cancel: what is left has eight bits, and the sums on the way at most 24
        b[:, r1] = power
        got = _lora(path, x, a, b, np.zeros(n), f32)
        np.testing.assert_array_equal(got, (t[r0] + t[r1]) * power)


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("path", list(PATHS))
def test_inner_sums_next_to_binary32s_largest(qdg, path, f32):
    """Finite inner sums whose bf16 rounding would be infinite, and products that only the rounding would take past the
    largest number."""
    n = 130
    # T = 2^128 - 2^104, the largest binary32 number, from three bf16 numbers
    x, a = np.ones(3), np.array([[255 * 2.0 ** 120, 255 * 2.0 ** 112, 255 * 2.0 ** 104]])
    b = 2.0 ** -np.arange(1.0, n + 1)[:, None]
    want = (2.0 ** 128 - 2.0 ** 104) * b[:, 0]
    got = _lora(path, x, a, b, np.zeros(n), f32)
    # two additions inside the product, each off by a step at most; bf16 Y: half a step
    assert np.all(np.abs(got - want) <= (2.0 ** -22 + (0 if f32 else 2.0 ** -8)) * want)
    got = _lora(path, x, -a, b, np.zeros(n), f32, scales=[1.0])
    assert np.all(np.abs(got + want) <= (2.0 ** -22 + (0 if f32 else 2.0 ** -8)) * want)
    # T = 1 + 2^-8 + 2^-20 beside 255 2^120: 0.99998 of 2^128; T's nearest bf16 number 1 + 2^-7 would overflow
    x, a = np.ones(3), np.array([[1.0, 2.0 ** -8, 2.0 ** -20]])
    b = np.full((n, 1), 255 * 2.0 ** 120)
    want = (1 + 2.0 ** -8 + 2.0 ** -20) * b[:, 0]
    # bf16 Y: brought into its range by the Y that is there
    y0 = 0.0 if f32 else -(2.0 ** 127)
    got = _lora(path, x, a, b, np.full(n, y0), f32)
    assert np.all(np.abs(got - (want + y0)) <= (2.0 ** -22 + (0 if f32 else 2.0 ** -8)) * want)


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("path", list(PATHS))
@pytest.mark.parametrize("rank", [1, 8, 20])
def test_infinities_and_nan_in_b(qdg, path, f32, rank):
    """An infinite entry of B makes its column infinite, with the sign of T times it; NaN, infinities of both signs and an
    infinity beside T = 0 make it NaN. Other columns keep their values."""
    rng = np.random.default_rng(rank)
    n, k = 300, 72
    for exact in (True, False):
        # T that bf16 holds (nothing is left for its other terms), and any T
        x, a = (np.ones(k), np.ones((rank, k))) if exact else (rng.standard_normal(k), rng.standard_normal((rank, k)))
        a[-1] *= -1.0
        b = rng.standard_normal((n, rank))
        clean = b.copy()
        b[3, 0], b[64, 0], b[130, rank - 1], b[299, rank - 1], b[17, 0] = np.inf, -np.inf, np.inf, -np.inf, np.nan
        b[200, 0] = np.inf
        b[200, rank - 1] = np.inf if (a @ x)[0] * (a @ x)[-1] < 0 else -np.inf
        x64, a64, b64 = (H.to_f64(_bf16(v)) for v in (x, a, b))
        y0 = rng.standard_normal(n).astype(np.float32) if f32 else H.to_f64(_bf16(rng.standard_normal(n)))
        with np.errstate(invalid="ignore"):
            want = y0 + ((a64 @ x64) * b64).sum(axis=1)
        got = _lora(path, x, a, b, y0, f32)
        bad = ~np.isfinite(want)
        assert bad.sum() == 6
        np.testing.assert_array_equal(got[bad], want[bad])
        np.testing.assert_array_equal(got[~bad], _lora(path, x, a, clean, y0, f32)[~bad])
    # T = 0: NaN; T infinite: an infinity
    for first, result in ((0.0, np.nan), (np.inf, np.inf)):
        b = np.ones((n, rank))
        b[5] = np.inf
        got = _lora(path, np.array([first]), np.ones((rank, 1)), b, np.zeros(n), f32)
        np.testing.assert_array_equal(got[5], result)


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("rank", [16, 28, 64])
def test_several_units_of_columns_a_workgroup(qdg, f32, rank):
    """So many blocks and columns that a workgroup of the kernel for many rows walks several units of B, one of them with
    an infinity and one with a NaN: only their columns change."""
    rng = np.random.default_rng(rank)
    M, n, k, E, bm = 2048, 2100, 4200, 3, 64
    pool = Pool(rng, n, k, rank, E, scales=False)
    ids = rng.integers(0, E, M).astype(np.int32)
    _run(rng, pool, ids, bm, f32)
    g = Group(ids, E, bm)
    x = _bf16(rng.standard_normal((M, k)))
    cfg = q.lora(n, k, rank, num_adapters=E, otype=q.QDG_O_F32 if f32 else q.QDG_O_BF16)
    nbytes = q.qdg_lora_workspace(cfg, M, bm)
    ws = torch.zeros(nbytes, dtype=torch.uint8, device="cuda")
    got = []
    for bad in (False, True):
        if bad:
            pool.dB[1, 1900, rank - 1], pool.dB[2, 700, 0] = float("inf"), float("nan")
        y = torch.zeros((M, n), dtype=torch.float32 if f32 else torch.bfloat16, device="cuda")
        q.qdg_lora(cfg, x.data_ptr(), pool.dA.data_ptr(), pool.dB.data_ptr(), None, None, *g.args(), y.data_ptr(),
                   ws.data_ptr(), nbytes, q.current_stream())
        torch.cuda.synchronize()
        got.append(y)
    first, second = torch.from_numpy(ids == 1).cuda(), torch.from_numpy(ids == 2).cuda()
    assert torch.isinf(got[1][first, 1900]).all() and torch.isnan(got[1][second, 700]).all()
    got[1][first, 1900], got[1][second, 700] = got[0][first, 1900], got[0][second, 700]
    assert torch.equal(got[0], got[1])
