"""qdg_lora against the float64 reference, within the bound of oracle.layer.lora
(counted binary32 roundings) plus half a step of Y's type."""

import numpy as np
import pytest
import torch

import quantized_dequant_gemm_amd as q
from oracle import codecs, layer, ops
from tests import gpu_helpers as H

pytestmark = pytest.mark.gpu


def _ptr(t):
    return None if t is None else t.data_ptr()


def _bf16(x):
    t = torch.from_numpy(np.ascontiguousarray(x, np.float32)).cuda().to(torch.bfloat16)
    return t, H.to_f64(t)


def _close(y, y64, err, bf16):
    y = H.to_f64(y)
    bound = err + (2.0 ** -8 * (np.abs(y64) + err) if bf16 else 2.0 ** -24 * np.abs(y64)) + 2.0 ** -126
    bad = np.argwhere(~(np.abs(y - y64) <= bound))
    assert bad.size == 0, [(tuple(b), y[tuple(b)], y64[tuple(b)], bound[tuple(b)]) for b in bad[:5]]


class Group:
    """The rows of a step grouped by adapter."""

    def __init__(self, ids, adapters, bm):
        self.M, self.bm = len(ids), bm
        cap = q.qdg_moe_align_capacity(self.M, 1, adapters, bm)
        self.ids = H.dev(np.asarray(ids, np.int32))
        new = lambda k: torch.full((k,), -5, dtype=torch.int32, device="cuda")  # noqa: E731
        self.sid, self.blk, self.npad = new(cap), new(max(1, cap // bm)), new(1)
        q.qdg_moe_align(self.ids.data_ptr(), self.M, 1, adapters, bm, self.sid.data_ptr(), self.blk.data_ptr(),
                        self.npad.data_ptr(), q.current_stream())

    def args(self):
        return self.sid.data_ptr(), self.blk.data_ptr(), self.npad.data_ptr(), self.M, self.bm


class Pool:
    """A pool of adapters; what lies behind an adapter's rank is NaN."""

    def __init__(self, rng, n, k, rank, adapters, ends=None, mixed=False, scales=True, spread=0.3):
        self.n, self.k, self.rank, self.adapters = n, k, rank, adapters
        self.ends = ends or [n]
        a = rng.standard_normal((adapters, len(self.ends), rank, k)) / np.sqrt(k)
        b = spread * rng.standard_normal((adapters, n, rank))
        self.ranks = rng.integers(0, rank + 1, adapters).astype(np.int32) if mixed else None
        self.scales = rng.uniform(0.5, 2.0, adapters).astype(np.float32) if scales else None
        self.dA, self.a = _bf16(a)
        self.dB, self.b = _bf16(b)
        if mixed:
            for e in range(adapters):
                self.dA[e, :, self.ranks[e]:] = float("nan")
                self.dB[e, :, self.ranks[e]:] = float("nan")
        self.dranks = None if self.ranks is None else H.dev(self.ranks)
        self.dscales = None if self.scales is None else H.dev(self.scales)

    def ref(self, y, x, ids):
        return layer.lora(y, x, ids, self.a, self.b, self.ends, self.ranks, self.scales)


def _run(rng, pool, ids, bm, f32, pad=0, shift=0):
    M, n, k = len(ids), pool.n, pool.k
    g = Group(ids, pool.adapters, bm)
    dt = torch.float32 if f32 else torch.bfloat16
    x, x64 = _bf16(rng.standard_normal((M, k)))
    fx = torch.full((shift + M * (k + pad) + 8,), float("nan"), dtype=torch.bfloat16, device="cuda")
    vx = fx[shift:shift + M * (k + pad)].view(M, k + pad)
    vx[:, :k] = x
    base = torch.from_numpy(rng.standard_normal((M, n)).astype(np.float32)).cuda().to(dt)
    fy = torch.full((shift + M * (n + pad) + 8,), 77.0, dtype=dt, device="cuda")
    vy = fy[shift:shift + M * (n + pad)].view(M, n + pad)
    vy[:, :n] = base
    cfg = q.lora(n, k, pool.rank, num_adapters=pool.adapters, slice_ends=pool.ends,
                 otype=q.QDG_O_F32 if f32 else q.QDG_O_BF16, ldx=k + pad, ldy=n + pad)
    nbytes = q.qdg_lora_workspace(cfg, M, bm)
    ws = torch.full((nbytes + 64,), 0xFF, dtype=torch.uint8, device="cuda")  # NaN as binary32
    q.qdg_lora(cfg, vx.data_ptr(), pool.dA.data_ptr(), pool.dB.data_ptr(), _ptr(pool.dranks), _ptr(pool.dscales), *g.args(),
               vy.data_ptr(), ws.data_ptr(), nbytes, q.current_stream())
    torch.cuda.synchronize()
    assert (fy[:shift] == 77).all() and (fy[shift + M * (n + pad):] == 77).all() and (vy[:, n:] == 77).all()
    assert (ws[nbytes:] == 0xFF).all()
    y64, err = pool.ref(H.to_f64(base), x64, ids)
    out = np.nonzero((np.asarray(ids) < 0) | (np.asarray(ids) >= pool.adapters))[0]
    sel = torch.from_numpy(out).cuda()
    assert torch.equal(vy[sel, :n], base[sel])
    _close(vy[:, :n], y64, err, not f32)
    return vy[:, :n]


MS = [1, 2, 15, 16, 17, 31, 33, 64, 65, 100, 130, 257]
NS = [1, 3, 15, 16, 17, 63, 64, 65, 100, 130, 257, 520]
KS = [1, 7, 8, 31, 32, 33, 64, 100, 129, 1000, 2050, 4100]
RANKS = [1, 2, 7, 8, 15, 16, 17, 24, 32, 33, 64, 100, 256]


@pytest.mark.parametrize("case", range(48))
def test_sizes(qdg, case):
    rng = np.random.default_rng(case)
    M, n, k = MS[case % 12], NS[(case * 5 + 2) % 12], KS[(case * 7 + 3) % 12]
    rank, E = RANKS[case % 13], (1, 3, 8, 20)[case % 4]
    ids = rng.integers(-1, E + 1, M).astype(np.int32)  # -1 and E: no adapter
    pool = Pool(rng, n, k, rank, E, mixed=bool(case & 1), scales=case % 3 != 0)
    _run(rng, pool, ids, (16, 32, 64, 128)[(case // 4) % 4], bool(case & 2), pad=(0, 1, 8)[case % 3], shift=(0, 1)[case % 2])


@pytest.mark.parametrize("bm", [16, 32, 64, 128])
@pytest.mark.parametrize("k", [6208, 6150, 12289])
def test_long_k_in_two_launches(qdg, k, bm):
    """Ranks below, at and between the tiles of 16; columns that end inside a unit of 64 or 128."""
    for i, (rank, n) in enumerate(((1, 65), (4, 130), (8, 129), (12, 255), (16, 257), (24, 300), (32, 96), (40, 131))):
        rng = np.random.default_rng(k + rank)
        ids = rng.integers(-1, 3, 75).astype(np.int32)
        pool = Pool(rng, n, k, rank, 3, ends=[n] if i & 1 else [n // 3, n], mixed=bool(i & 2))
        assert q.qdg_lora_workspace(q.lora(n, k, rank, num_adapters=3, slice_ends=pool.ends), 75, bm) > 0
        _run(rng, pool, ids, bm, bool(i & 1), pad=i % 3, shift=i % 2)


def test_many_tiles_of_a_short_k(qdg):
    """More workgroups than run at once: two launches for sizes that take one where rows are few."""
    rng = np.random.default_rng(77)
    for bm, M, n, rank in ((16, 1500, 4200, 8), (64, 3000, 6600, 16), (128, 2600, 8200, 32)):
        ids = rng.integers(-1, 6, M).astype(np.int32)
        pool = Pool(rng, n, 200, rank, 6, ends=[n // 2 + 3, n])
        assert q.qdg_lora_workspace(q.lora(n, 200, rank, num_adapters=6, slice_ends=pool.ends), M, bm) > 0
        _run(rng, pool, ids, bm, rank == 16)


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("ends", [[1, 2, 3, 4], [64, 100], [30, 31, 200], [512, 576, 640], [1, 300, 301, 365]])
def test_slices(qdg, ends, f32):
    for i, (M, rank, bm) in enumerate(((1, 16, 16), (37, 8, 16), (150, 40, 64))):
        rng = np.random.default_rng(ends[-1] + i)
        ids = rng.integers(-1, 5, M).astype(np.int32)
        _run(rng, Pool(rng, ends[-1], 520, rank, 5, ends=ends, mixed=bool(i & 1)), ids, bm, f32)


@pytest.mark.parametrize("M,E,bm", [(1, 1, 16), (1, 64, 16), (64, 64, 16), (300, 2, 64), (700, 3, 128), (513, 200, 32)])
@pytest.mark.parametrize("n,k,rank", [(1024, 4096, 16), (640, 9000, 64)])
def test_serving_shapes(qdg, M, E, bm, n, k, rank):
    rng = np.random.default_rng(M + E)
    ids = np.sort(rng.integers(0, E, M)).astype(np.int32)
    _run(rng, Pool(rng, n, k, rank, E), ids, bm, False)
    _run(rng, Pool(rng, n, k, rank, E, mixed=True), rng.permutation(ids), bm, True)


def test_no_row_has_an_adapter(qdg):
    rng = np.random.default_rng(0)
    _run(rng, Pool(rng, 100, 64, 8, 3), np.full(40, -1, np.int32), 16, False)
    pool = Pool(rng, 100, 64, 8, 3, mixed=True)
    pool.ranks[:] = 0
    pool.dranks.zero_()
    _run(rng, pool, np.arange(40, dtype=np.int32) % 3, 16, True)


def test_ranks_outside_their_range_are_clamped(qdg):
    rng = np.random.default_rng(1)
    pool = Pool(rng, 130, 200, 12, 3)
    pool.ranks = np.array([-4, 5, 12], np.int32)
    pool.dranks = H.dev(np.array([-4, 5, 4000], np.int32))
    _run(rng, pool, rng.integers(0, 3, 50).astype(np.int32), 16, False)


def test_rows_with_infinities_and_nan_keep_to_themselves(qdg):
    rng = np.random.default_rng(2)
    M, n, k, bm = 40, 200, 300, 16
    pool = Pool(rng, n, k, 20, 2)
    ids = (np.arange(M) % 2).astype(np.int32)
    for f32 in (False, True):
        dt = torch.float32 if f32 else torch.bfloat16
        g = Group(ids, 2, bm)
        x, _ = _bf16(rng.standard_normal((M, k)))
        base = torch.zeros((M, n), dtype=dt, device="cuda")
        cfg = q.lora(n, k, 20, num_adapters=2, otype=q.QDG_O_F32 if f32 else q.QDG_O_BF16)
        nbytes = q.qdg_lora_workspace(cfg, M, bm)
        ws = torch.zeros(nbytes, dtype=torch.uint8, device="cuda")
        got = []
        for bad in (False, True):
            if bad:
                x[3, 7], x[8, 299] = float("inf"), float("nan")
            y = base.clone()
            q.qdg_lora(cfg, x.data_ptr(), pool.dA.data_ptr(), pool.dB.data_ptr(), None, _ptr(pool.dscales), *g.args(),
                       y.data_ptr(), ws.data_ptr(), nbytes, q.current_stream())
            torch.cuda.synchronize()
            got.append(y)
        assert torch.isnan(got[1][8]).all() and not torch.isfinite(got[1][3]).any()
        others = [m for m in range(M) if m not in (3, 8)]
        assert torch.equal(got[0][others], got[1][others])


def test_one_infinite_inner_sum_gives_infinities(qdg):
    """Rank 1, A and B of ones: T = inf, Y = inf, not NaN."""
    x = torch.ones((1, 40), dtype=torch.bfloat16, device="cuda")
    x[0, 5] = float("inf")
    a, b = torch.ones((1, 1, 1, 40), dtype=torch.bfloat16, device="cuda"), torch.ones((1, 30, 1), dtype=torch.bfloat16, device="cuda")
    y = torch.zeros((1, 30), device="cuda")
    g = Group([0], 1, 16)
    cfg = q.lora(30, 40, 1, otype=q.QDG_O_F32)
    nbytes = q.qdg_lora_workspace(cfg, 1, 16)
    ws = torch.zeros(nbytes, dtype=torch.uint8, device="cuda")
    q.qdg_lora(cfg, x.data_ptr(), a.data_ptr(), b.data_ptr(), None, None, *g.args(), y.data_ptr(), ws.data_ptr(), nbytes,
               q.current_stream())
    torch.cuda.synchronize()
    assert (y == float("inf")).all()


def test_offsets_past_32_bits(qdg):
    """Rows of X and Y whose strides take the last past 4 GiB, and the last adapter of a pool above 4 GiB."""
    rng = np.random.default_rng(5)
    M, n, k, rank = 3, 70, 100, 16
    pool = Pool(rng, n, k, rank, 2)
    ids = np.array([0, 1, 1], np.int32)
    g = Group(ids, 2, 16)
    ldx, ldy = (1 << 30) + 1, (1 << 30) + 5
    x, x64 = _bf16(rng.standard_normal((M, k)))
    base, b64 = _bf16(rng.standard_normal((M, n)))
    fx = torch.zeros(2 * ldx + k, dtype=torch.bfloat16, device="cuda")
    fy = torch.zeros(2 * ldy + n, dtype=torch.bfloat16, device="cuda")
    for m in range(M):
        fx[m * ldx:m * ldx + k] = x[m]
        fy[m * ldy:m * ldy + n] = base[m]
    cfg = q.lora(n, k, rank, num_adapters=2, ldx=ldx, ldy=ldy)
    nbytes = q.qdg_lora_workspace(cfg, M, 16)
    ws = torch.zeros(nbytes, dtype=torch.uint8, device="cuda")
    q.qdg_lora(cfg, fx.data_ptr(), pool.dA.data_ptr(), pool.dB.data_ptr(), None, _ptr(pool.dscales), *g.args(), fy.data_ptr(),
               ws.data_ptr(), nbytes, q.current_stream())
    torch.cuda.synchronize()
    y = torch.stack([fy[m * ldy:m * ldy + n] for m in range(M)])
    y64, err = pool.ref(b64, x64, ids)
    _close(y, y64, err, True)
    del fx, fy
    E, n, k, rank = 600, 16, 32768, 128  # A: 600 * 128 * 32768 * 2 bytes = 4.7 GiB
    a = torch.zeros((E, 1, rank, k), dtype=torch.bfloat16, device="cuda")
    b = torch.zeros((E, n, rank), dtype=torch.bfloat16, device="cuda")
    da, a64 = _bf16(rng.standard_normal((rank, k)) / np.sqrt(k))
    db, bb64 = _bf16(rng.standard_normal((n, rank)))
    a[E - 1, 0], b[E - 1] = da, db
    x, x64 = _bf16(rng.standard_normal((2, k)))
    y = torch.zeros((2, n), device="cuda")
    g = Group([E - 1, E - 1], E, 16)
    cfg = q.lora(n, k, rank, num_adapters=E, otype=q.QDG_O_F32)
    nbytes = q.qdg_lora_workspace(cfg, 2, 16)
    ws = torch.zeros(nbytes, dtype=torch.uint8, device="cuda")
    q.qdg_lora(cfg, x.data_ptr(), a.data_ptr(), b.data_ptr(), None, None, *g.args(), y.data_ptr(), ws.data_ptr(), nbytes,
               q.current_stream())
    torch.cuda.synchronize()
    y64, err = layer.lora(np.zeros((2, n)), x64, [0, 0], a64[None, None], bb64[None], [n])
    _close(y, y64, err, False)


def test_same_result_on_every_call_and_other_stream(qdg):
    rng = np.random.default_rng(6)
    M, n, k, E, bm = 90, 1000, 3000, 7, 16
    pool = Pool(rng, n, k, 24, E)
    ids = rng.integers(-1, E, M).astype(np.int32)
    g = Group(ids, E, bm)
    x, x64 = _bf16(rng.standard_normal((M, k)))
    base = torch.from_numpy(rng.standard_normal((M, n)).astype(np.float32)).cuda()
    cfg = q.lora(n, k, 24, num_adapters=E, otype=q.QDG_O_F32)
    nbytes = q.qdg_lora_workspace(cfg, M, bm)
    streams = [torch.cuda.Stream() for _ in range(3)]
    ys, wss = [base.clone() for _ in streams], [torch.zeros(nbytes, dtype=torch.uint8, device="cuda") for _ in streams]
    torch.cuda.synchronize()
    for st, y, ws in zip(streams, ys, wss):
        q.qdg_lora(cfg, x.data_ptr(), pool.dA.data_ptr(), pool.dB.data_ptr(), None, _ptr(pool.dscales), *g.args(), y.data_ptr(),
                   ws.data_ptr(), nbytes, st.cuda_stream)
    torch.cuda.synchronize()
    y64, err = pool.ref(H.to_f64(base), x64, ids)
    _close(ys[0], y64, err, False)
    assert torch.equal(ys[0], ys[1]) and torch.equal(ys[0], ys[2])


def test_one_workspace_for_every_batch(qdg):
    rng = np.random.default_rng(8)
    n, k, E, bm = 300, 5000, 6, 16
    pool = Pool(rng, n, k, 33, E)
    cfg = q.lora(n, k, 33, num_adapters=E, otype=q.QDG_O_F32)
    nbytes = q.qdg_lora_workspace(cfg, 600, bm)
    ws = torch.full((nbytes + 256,), 0x5A, dtype=torch.uint8, device="cuda")
    for M in (1, 16, 17, 100, 257, 600):
        ids = rng.integers(0, E, M).astype(np.int32)
        g = Group(ids, E, bm)
        x, x64 = _bf16(rng.standard_normal((M, k)))
        y = torch.zeros((M, n), device="cuda")
        q.qdg_lora(cfg, x.data_ptr(), pool.dA.data_ptr(), pool.dB.data_ptr(), None, _ptr(pool.dscales), *g.args(), y.data_ptr(),
                   ws.data_ptr(), nbytes, q.current_stream())
        torch.cuda.synchronize()
        y64, err = pool.ref(np.zeros((M, n)), x64, ids)
        _close(y, y64, err, False)
        assert (ws[nbytes:] == 0x5A).all()


# ---------------------------------------------------------------- together

def test_layer_with_adapters(qdg):
    """norm -> int8 codes and rows -> gate+up product with its adapters -> gated activation to codes -> down product
    with its adapters -> norm on both sides into the next block, every step on the device's output of the one before,
    captured and replayed on new inputs with eager work between."""
    M, hid, inter, E, bm, rank = 45, 264, 200, 5, 16, 12
    rng = np.random.default_rng(31)
    ld_h, ld_i = 272, 208
    wts = lambda n, k: (rng.integers(-127, 128, (n, k)).astype(np.int8), rng.uniform(1e-4, 5e-4, n).astype(np.float32))  # noqa: E731
    (w1, s1), (w2, s2) = wts(2 * inter, hid), wts(hid, inter)

    def stored(w, ld):
        buf = np.zeros((w.shape[0], ld), np.int8)
        buf[:, :w.shape[1]] = w
        return H.dev(buf)

    dw1, ds1, dw2, ds2 = stored(w1, ld_h), H.dev(s1), stored(w2, ld_i), H.dev(s2)
    up, down = Pool(rng, 2 * inter, hid, rank, E, ends=[inter, 2 * inter], mixed=True), Pool(rng, hid, inter, rank, E, mixed=True)
    new = lambda *s, dt=torch.bfloat16: torch.zeros(s, dtype=dt, device="cuda")  # noqa: E731
    x, res, rows, res2, rows2, inner, y1, y2 = (new(M, hid), new(M, hid), new(M, hid), new(M, hid), new(M, hid), new(M, inter),
                                               new(M, 2 * inter), new(M, hid))
    nw, nw64 = _bf16(1.0 + 0.2 * rng.standard_normal(hid))
    pw, pw64 = _bf16(1.0 + 0.2 * rng.standard_normal(hid))
    qh, sh, zh = new(M, ld_h, dt=torch.int8), new(M, dt=torch.float32), new(M, dt=torch.int32)
    qi, si, zi = new(M, ld_i, dt=torch.int8), new(M, dt=torch.float32), new(M, dt=torch.int32)
    ids = rng.integers(-1, E, M).astype(np.int32)
    g = Group(ids, E, bm)
    n1 = q.norm(hid, quant=q.QDG_Q_INT8_ZP, ldq=ld_h)
    n2 = q.norm(hid, post_norm=1, residual_scale=0.5)
    act = q.gated_act(inter, quant=q.QDG_Q_INT8_ZP, ldq=ld_i)
    c1, c2 = q.gemm_i8(2 * inter, hid, lda=ld_h, ldb=ld_h), q.gemm_i8(hid, inter, lda=ld_i, ldb=ld_i)
    l1 = q.lora(2 * inter, hid, rank, num_adapters=E, slice_ends=up.ends)
    l2 = q.lora(hid, inter, rank, num_adapters=E)
    nbytes = max(q.qdg_lora_workspace(l1, M, bm), q.qdg_lora_workspace(l2, M, bm))
    ws = new(nbytes, dt=torch.uint8)

    def block(st):
        q.qdg_moe_align(g.ids.data_ptr(), M, 1, E, bm, g.sid.data_ptr(), g.blk.data_ptr(), g.npad.data_ptr(), st)
        q.qdg_norm(n1, x.data_ptr(), res.data_ptr(), None, None, None, nw.data_ptr(), None, M, res.data_ptr(),
                   rows.data_ptr(), qh.data_ptr(), sh.data_ptr(), zh.data_ptr(), st)
        q.qdg_gemm_i8(c1, qh.data_ptr(), sh.data_ptr(), zh.data_ptr(), dw1.data_ptr(), ds1.data_ptr(), None, y1.data_ptr(), M,
                      None, 0, st)
        q.qdg_lora(l1, rows.data_ptr(), up.dA.data_ptr(), up.dB.data_ptr(), up.dranks.data_ptr(), up.dscales.data_ptr(),
                   *g.args(), y1.data_ptr(), ws.data_ptr(), nbytes, st)
        q.qdg_gated_act(act, y1.data_ptr(), M, inner.data_ptr(), qi.data_ptr(), si.data_ptr(), zi.data_ptr(), st)
        q.qdg_gemm_i8(c2, qi.data_ptr(), si.data_ptr(), zi.data_ptr(), dw2.data_ptr(), ds2.data_ptr(), None, y2.data_ptr(), M,
                      None, 0, st)
        q.qdg_lora(l2, inner.data_ptr(), down.dA.data_ptr(), down.dB.data_ptr(), down.dranks.data_ptr(), down.dscales.data_ptr(),
                   *g.args(), y2.data_ptr(), ws.data_ptr(), nbytes, st)
        q.qdg_norm(n2, y2.data_ptr(), res.data_ptr(), None, pw.data_ptr(), None, nw.data_ptr(), None, M, res2.data_ptr(),
                   rows2.data_ptr(), None, None, None, st)

    def fresh():
        nonlocal ids
        ids = rng.integers(-1, E, M).astype(np.int32)
        g.ids.copy_(torch.from_numpy(ids))
        x.copy_(torch.from_numpy(rng.standard_normal((M, hid)).astype(np.float32)))
        res.copy_(torch.from_numpy(rng.standard_normal((M, hid)).astype(np.float32)))
        return H.to_f64(x), H.to_f64(res)

    def verify(x64, r64):
        torch.cuda.synchronize()
        bits_of = lambda t: t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)  # noqa: E731
        s, bits = layer.norm(x64, r64, weight=nw64)
        np.testing.assert_array_equal(H.to_f64(res), s)
        np.testing.assert_array_equal(bits_of(rows), bits)
        cq, cs, cz = layer.codes(bits, "int8_zp")
        np.testing.assert_array_equal(qh[:, :hid].cpu().numpy(), cq)
        # the product leaves bf16 rows, the adapters' sum joins those: half a step each
        p64, perr = ops.gemm_i8(cq, cs, w1, s1, cz)
        perr = perr + 2.0 ** -8 * (np.abs(p64) + perr)
        y64, err = up.ref(p64, codecs.bf16_bits_to_f64(bits), ids)
        _close(y1, y64, err + perr, True)
        inner_bits = layer.gated_act(H.to_f64(y1))
        np.testing.assert_array_equal(bits_of(inner), inner_bits)
        cq, cs, cz = layer.codes(inner_bits, "int8_zp")
        np.testing.assert_array_equal(qi[:, :inter].cpu().numpy(), cq)
        p64, perr = ops.gemm_i8(cq, cs, w2, s2, cz)
        perr = perr + 2.0 ** -8 * (np.abs(p64) + perr)
        y64, err = down.ref(p64, codecs.bf16_bits_to_f64(inner_bits), ids)
        _close(y2, y64, err + perr, True)
        s2_, bits = layer.norm(H.to_f64(y2), s, post=(pw64, None), weight=nw64, residual_scale=0.5)
        np.testing.assert_array_equal(H.to_f64(res2), s2_)
        np.testing.assert_array_equal(bits_of(rows2), bits)

    before = fresh()
    block(q.current_stream())
    verify(*before)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        block(q.current_stream())
    for _ in range(3):
        before = fresh()
        for t in (rows, y1, inner, y2, rows2, qh, qi, g.sid, ws):
            t.zero_()
        graph.replay()
        verify(*before)


def test_adapters_share_a_workspace_in_two_graphs(qdg):
    """Two captured calls over one workspace, replayed in turn on one stream."""
    rng = np.random.default_rng(12)
    shapes = ((20, 300, 4100, 16, 16), (70, 900, 500, 40, 16))
    calls = []
    for M, n, k, rank, bm in shapes:
        pool = Pool(rng, n, k, rank, 4)
        ids = rng.integers(0, 4, M).astype(np.int32)
        cfg = q.lora(n, k, rank, num_adapters=4, otype=q.QDG_O_F32)
        calls.append((pool, ids, Group(ids, 4, bm), cfg, torch.zeros((M, k), dtype=torch.bfloat16, device="cuda"),
                      torch.zeros((M, n), device="cuda")))
    nbytes = max(q.qdg_lora_workspace(c[3], len(c[1]), 16) for c in calls)
    ws = torch.zeros(nbytes, dtype=torch.uint8, device="cuda")
    graphs = []
    for pool, ids, g, cfg, x, y in calls:
        def go():
            y.zero_()
            q.qdg_lora(cfg, x.data_ptr(), pool.dA.data_ptr(), pool.dB.data_ptr(), None, _ptr(pool.dscales), *g.args(),
                       y.data_ptr(), ws.data_ptr(), nbytes, q.current_stream())
        go()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            go()
        graphs.append(graph)
    for _ in range(3):
        want = []
        for pool, ids, g, cfg, x, y in calls:
            t, x64 = _bf16(rng.standard_normal(tuple(x.shape)))
            x.copy_(t)
            want.append(pool.ref(np.zeros(tuple(y.shape)), x64, ids))
        for graph in graphs:
            graph.replay()
        torch.cuda.synchronize()
        for (y64, err), c in zip(want, calls):
            _close(c[5], y64, err, False)
