"""Host-side validation of the norms, the gated activation and the low-rank
adapters on the CPU: every refusal happens before any device work."""

import pytest

import quantized_dequant_gemm_amd as q

P = 0x10000  # a 16-byte aligned address that no refused call reads
INV, UNS, MIS, WS = q.QDG_ERR_INVALID_ARG, q.QDG_ERR_UNSUPPORTED, q.QDG_ERR_MISALIGNED, q.QDG_ERR_WORKSPACE


def _status(fn, *a):
    try:
        fn(*a)
    except q.QdgError as e:
        return e.status
    return q.QDG_OK


def _norm(n=64, M=4, x=P, residual=P, gate=P, post_weight=None, post_bias=None, weight=P, bias=P, residual_out=2 * P,
          out=3 * P, qa=4 * P, scales=P, zeros=P, reserved=0, **kw):
    cfg = q.norm(n, **kw)
    cfg.reserved = reserved
    return _status(q.qdg_norm, cfg, x, residual, gate, post_weight, post_bias, weight, bias, M, residual_out, out, qa,
                   scales, zeros)


def test_norm_refusals():
    assert _norm(M=0) == q.QDG_OK and _norm(M=0, x=None, out=None, residual_out=None) == q.QDG_OK
    assert _norm(M=-1) == INV and _norm(M=1 << 31) == UNS
    assert _norm(n=0) == INV and _norm(n=32769) == UNS
    for bad in ({"kind": 2}, {"kind": -1}, {"post_norm": 2}, {"xtype": q.QDG_O_I32}, {"rtype": 3}, {"wtype": -1},
                {"quant": 5}, {"quant": -1}, {"reserved": 1}, {"eps": -1e-6}, {"eps": float("nan")},
                {"eps": float("inf")}, {"residual_scale": float("inf")}, {"weight_offset": float("nan")},
                {"ldx": 63}, {"ldr": 63}, {"lds": 63}, {"ldg": 63}, {"ldg": -1}, {"ldo": 63}, {"x": None},
                {"residual_out": None, "out": None}, {"post_weight": P}, {"post_bias": P}, {"ldx": (1 << 31) + 1}):
        assert _norm(**bad) == INV, bad
    for bad in ({"x": P + 1}, {"residual": P + 1}, {"gate": P + 1}, {"weight": P + 1}, {"bias": P + 1},
                {"residual_out": P + 1}, {"out": P + 1}, {"x": P + 2, "xtype": q.QDG_O_F32},
                {"residual": P + 2, "rtype": q.QDG_O_F32}, {"residual_out": P + 2, "rtype": q.QDG_O_F32},
                {"weight": P + 2, "wtype": q.QDG_O_F32}, {"post_weight": P + 1, "post_norm": 1},
                {"post_bias": P + 1, "post_norm": 1}):
        assert _norm(**bad) == MIS, bad


def test_norm_in_place_rules():
    assert _norm(residual=P, residual_out=P, ldr=64, lds=72) == INV
    assert _norm(x=P, out=P, xtype=q.QDG_O_F32) == INV
    assert _norm(x=P, out=P, ldx=72, ldo=64) == INV


@pytest.mark.parametrize("quant", [q.QDG_Q_INT8, q.QDG_Q_INT8_ZP, q.QDG_Q_FP8E4M3, q.QDG_Q_MXFP4])
def test_code_refusals(quant):
    row = 64 if quant == q.QDG_Q_MXFP4 else 128
    assert _norm(n=128, quant=quant, M=0, qa=None, scales=None) == q.QDG_OK
    for call in (_norm, _gated):
        assert call(n=128, quant=quant, qa=None) == INV and call(n=128, quant=quant, scales=None) == INV
        assert call(n=128, quant=quant, ldq=row - 16) == INV
        assert call(n=128, quant=quant, ldq=row + 8) == MIS
        assert call(n=128, quant=quant, qa=P + 8) == MIS
        if quant != q.QDG_Q_MXFP4:
            assert call(n=128, quant=quant, scales=P + 2) == MIS
        if quant == q.QDG_Q_INT8_ZP:
            assert call(n=128, quant=quant, zeros=None) == INV and call(n=128, quant=quant, zeros=P + 2) == MIS
        if quant == q.QDG_Q_FP8E4M3:
            assert call(n=192, quant=quant) == UNS
        if quant == q.QDG_Q_MXFP4:
            assert call(n=80, quant=quant) == UNS


def _gated(n=64, M=4, Y=P, out=2 * P, qa=4 * P, scales=P, zeros=P, reserved=0, **kw):
    cfg = q.gated_act(n, **kw)
    cfg.reserved = reserved
    return _status(q.qdg_gated_act, cfg, Y, M, out, qa, scales, zeros)


def test_gated_refusals():
    assert _gated(M=0) == q.QDG_OK and _gated(M=0, Y=None) == q.QDG_OK
    assert _gated(M=-1) == INV and _gated(M=1 << 31) == UNS and _gated(n=0) == INV and _gated(n=65537) == UNS
    for bad in ({"act": 2}, {"act": -1}, {"ytype": q.QDG_O_I32}, {"quant": 9}, {"reserved": 3}, {"ldy": 127},
                {"ldo": 63}, {"Y": None}, {"out": None}):
        assert _gated(**bad) == INV, bad
    assert _gated(Y=P + 1) == MIS and _gated(Y=P + 2, ytype=q.QDG_O_F32) == MIS and _gated(out=P + 1) == MIS


def _lora(n=64, k=32, rank=8, M=4, block_m=16, X=P, A=P, B=P, ranks=P, scales=P, sid=P, blk=P, npad=P, Y=P, ws=P,
          ws_bytes=1 << 40, **kw):
    cfg = q.lora(n, k, rank, **kw)
    return _status(q.qdg_lora, cfg, X, A, B, ranks, scales, sid, blk, npad, M, block_m, Y, ws, ws_bytes)


def test_lora_refusals():
    assert _lora(M=0) == q.QDG_OK and _lora(M=0, X=None, ws=None) == q.QDG_OK
    assert _lora(M=-1) == INV and _lora(M=(1 << 20) + 1) == UNS
    assert _lora(n=0) == INV and _lora(k=0) == INV and _lora(rank=0) == INV and _lora(num_adapters=0) == INV
    assert _lora(n=(1 << 20) + 1) == UNS and _lora(k=(1 << 20) + 1) == UNS and _lora(rank=257) == UNS
    assert _lora(num_adapters=1025) == UNS
    assert _lora(slice_ends=[]) == INV and _lora(slice_ends=[10, 20, 30, 40, 64]) == UNS
    for ends in ([32], [32, 32, 64], [40, 30, 64], [0, 64], [-1, 64], [32, 65]):
        assert _lora(slice_ends=ends) == INV, ends
    assert _lora(otype=q.QDG_O_I32) == INV and _lora(ldx=31) == INV and _lora(ldy=63) == INV
    assert _lora(block_m=8) == UNS and _lora(block_m=256) == UNS
    for name in ("X", "A", "B", "Y", "sid", "blk", "npad"):
        assert _lora(**{name: None}) == INV, name
        assert _lora(**{name: P + 1}) == MIS, name
    assert _lora(ranks=P + 2) == MIS and _lora(scales=P + 2) == MIS
    assert _lora(otype=q.QDG_O_F32, Y=P + 2) == MIS
    assert _lora(ws=P + 8) == MIS
    need = q.qdg_lora_workspace(q.lora(64, 16384, 8), 4, 16)
    assert need > 0 and _lora(k=16384, ws_bytes=need - 1) == WS and _lora(k=16384, ws=None) == WS
    assert q.qdg_lora_workspace(q.lora(64, 32, 8), 4, 16) == 0  # both products in one launch
    # 2^20 rows in tiles of 16 and 2^20 columns in units of 64: more workgroups than a launch holds
    assert _lora(M=1 << 20, n=1 << 20) == UNS


def test_lora_workspace():
    assert q.qdg_lora_workspace(q.lora(64, 32, 8), 0, 16) == 0
    assert _status(q.qdg_lora_workspace, q.lora(64, 32, 8), -1, 16) == INV
    assert _status(q.qdg_lora_workspace, q.lora(64, 32, 8), 4, 24) == UNS
    assert q.load().qdg_lora_workspace(None, 4, 16, None) == INV


@pytest.mark.parametrize("k", [64, 4090, 14336])
@pytest.mark.parametrize("rank,slices,adapters", [(4, 1, 1), (16, 3, 48), (64, 1, 12), (256, 4, 1024)])
def test_lora_workspace_of_the_largest_batch_serves_smaller_ones(k, rank, slices, adapters):
    ends = [100 * (i + 1) for i in range(slices)]
    cfg = q.lora(ends[-1], k, rank, num_adapters=adapters, slice_ends=ends)
    for bm in (16, 64):
        need = [q.qdg_lora_workspace(cfg, m, bm) for m in list(range(0, 300)) + [1000, 4096, 1 << 20]]
        assert need == sorted(need)
        for m in (1, 5, 33, 299):  # what a call for fewer rows asks for is covered
            assert _lora(n=ends[-1], k=k, rank=rank, num_adapters=adapters, slice_ends=ends, M=m, block_m=bm,
                         ws=P + 8, ws_bytes=need[m]) == MIS


def test_messages_name_the_cause():
    with pytest.raises(q.QdgError, match="slice_end must ascend"):
        q.qdg_lora(q.lora(64, 32, 8, slice_ends=[40, 30, 64]), P, P, P, P, P, P, P, P, 4, 16, P, P, 1 << 30)
    with pytest.raises(q.QdgError, match="multiple of 128"):
        q.qdg_norm(q.norm(100, quant=q.QDG_Q_FP8E4M3), P, P, None, None, None, P, None, 1, P, P, P, P)
    assert q.load().qdg_norm(None, *[P] * 7, 1, *[P] * 5, None) == INV
    assert q.load().qdg_gated_act(None, P, 1, P, P, P, P, None) == INV
