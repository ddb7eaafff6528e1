"""Host-side validation of the router, the asymmetric quantizer and the int8
products on the CPU: every refusal happens before any device work."""

import pytest

import quantized_dequant_gemm_amd as q

P = 0x10000  # a 16-byte aligned address that no refused call reads


def _status(fn, *a, **kw):
    try:
        fn(*a, **kw)
    except q.QdgError as e:
        return e.status
    return q.QDG_OK


def _route(T=4, ld=None, logits=P, ids=P, w=P, bias=None, status=None, **kw):
    cfg = q.route(kw.pop("E", 64), kw.pop("top_k", 4), **kw)
    return _status(q.qdg_moe_route, cfg, logits, cfg.num_experts if ld is None else ld, bias, T, ids, w, 0, status)


def test_route_refusals():
    inv, uns, mis = q.QDG_ERR_INVALID_ARG, q.QDG_ERR_UNSUPPORTED, q.QDG_ERR_MISALIGNED
    assert _route(T=0) == q.QDG_OK
    assert _route(T=0, logits=None, ids=None, w=None) == q.QDG_OK
    assert _route(T=-1) == inv
    assert _route(E=0) == inv and _route(top_k=0) == inv
    assert _route(E=1025) == uns and _route(E=256, top_k=33) == uns
    assert _route(E=4, top_k=5) == inv
    assert _route(num_groups=-1) == inv
    assert _route(num_groups=3) == inv  # 64 experts in 3 groups
    assert _route(E=260, num_groups=65, topk_groups=1) == uns
    assert _route(num_groups=8, topk_groups=0) == inv and _route(num_groups=8, topk_groups=9) == inv
    assert _route(num_groups=32, topk_groups=1, top_k=3) == inv  # two experts stay
    assert _route(ltype=3) == inv and _route(score=2) == inv and _route(group_score=-1) == inv
    assert _route(scale=float("inf")) == inv and _route(scale=float("nan")) == inv
    assert _route(ld=63) == inv
    assert _route(T=1 << 31) == uns
    assert _route(logits=None) == inv and _route(ids=None) == inv and _route(w=None) == inv
    assert _route(logits=P + 1) == mis and _route(ltype=q.QDG_L_F32, logits=P + 2) == mis
    assert _route(bias=P + 2) == mis and _route(ids=P + 2) == mis and _route(w=P + 1) == mis
    assert _route(status=P + 2) == mis
    assert q.load().qdg_moe_route(None, P, 64, None, 1, P, P, None, None) == inv


def _quant(a=P, lda=64, M=4, k=64, qa=P, ldq=64, s=P, z=P):
    return _status(q.qdg_quantize_act_zp, a, lda, M, k, qa, ldq, s, z)


def test_quantize_refusals():
    inv, uns, mis = q.QDG_ERR_INVALID_ARG, q.QDG_ERR_UNSUPPORTED, q.QDG_ERR_MISALIGNED
    assert _quant(M=0) == q.QDG_OK
    assert _quant(M=-1) == inv and _quant(k=0) == inv
    assert _quant(lda=56) == inv and _quant(ldq=48) == inv
    assert _quant(lda=68) == mis and _quant(ldq=72) == mis
    assert _quant(a=P + 2) == mis and _quant(qa=P + 8) == mis and _quant(s=P + 2) == mis and _quant(z=P + 1) == mis
    for name in ("a", "qa", "s", "z"):
        assert _quant(**{name: None}) == inv
    assert _quant(M=1 << 31) == uns
    assert _quant(k=(1 << 30) + 8, lda=1 << 31, ldq=1 << 31) == uns


def _gemm(n=64, k=64, M=4, A=P, s=P, z=P, B=P, bs=P, bias=P, Y=P, ws=P, ws_bytes=1 << 40, **kw):
    cfg = q.gemm_i8(n, k, **{x: kw[x] for x in kw if x not in ("reserved",)})
    cfg.reserved = kw.get("reserved", 0)
    return _status(q.qdg_gemm_i8, cfg, A, s, z, B, bs, bias, Y, M, ws, ws_bytes)


def test_gemm_refusals():
    inv, uns, mis = q.QDG_ERR_INVALID_ARG, q.QDG_ERR_UNSUPPORTED, q.QDG_ERR_MISALIGNED
    assert _gemm(M=0) == q.QDG_OK and _gemm(M=-1) == inv and _gemm(M=(1 << 26) + 1) == uns
    assert _gemm(n=0) == inv and _gemm(k=0) == inv
    assert _gemm(k=65537) == uns and _gemm(n=(1 << 26) + 1) == uns
    assert _gemm(num_experts=2) == inv and _gemm(num_experts=0) == inv
    assert _gemm(otype=3) == inv and _gemm(epilogue=2) == inv and _gemm(reserved=1) == inv
    assert _gemm(n=63, epilogue=q.QDG_EPI_SILU_MUL) == inv
    assert _gemm(otype=q.QDG_O_I32, epilogue=q.QDG_EPI_SILU_MUL) == uns
    assert _gemm(lda=48) == inv and _gemm(ldb=32) == inv and _gemm(ldy=63) == inv
    assert _gemm(lda=72) == mis and _gemm(ldb=100) == mis
    assert _gemm(A=P + 8) == mis and _gemm(B=P + 4) == mis and _gemm(Y=P + 1) == mis
    assert _gemm(otype=q.QDG_O_F32, Y=P + 2) == mis
    assert _gemm(s=P + 2) == mis and _gemm(z=P + 2) == mis and _gemm(bs=P + 2) == mis and _gemm(bias=P + 2) == mis
    for name in ("A", "B", "Y", "s", "bs"):
        assert _gemm(**{name: None}) == inv
    assert q.load().qdg_gemm_i8(None, P, P, P, P, P, P, P, 1, None, 0, None) == inv


def test_gemm_workspace():
    assert q.qdg_gemm_i8_workspace(q.gemm_i8(64, 64), 0) == 0
    assert _status(q.qdg_gemm_i8_workspace, q.gemm_i8(64, 64), -1) == q.QDG_ERR_INVALID_ARG
    assert _status(q.qdg_gemm_i8_workspace, q.gemm_i8(64, 64, num_experts=2), 1) == q.QDG_ERR_INVALID_ARG
    for M, n, k in ((1, 64, 65536), (16, 512, 16384), (64, 128, 8192), (300, 128, 65536)):
        need = q.qdg_gemm_i8_workspace(q.gemm_i8(n, k), M)
        assert need % (M * n * 4) == 0
        if need:
            assert _gemm(M=M, n=n, k=k, ws_bytes=need - 1) == q.QDG_ERR_WORKSPACE
            assert _gemm(M=M, n=n, k=k, ws=None) == q.QDG_ERR_WORKSPACE
            assert _gemm(M=M, n=n, k=k, ws=P + 8) == q.QDG_ERR_MISALIGNED


def _moe(E=8, T=4, top_k=2, bm=16, sid=P, blk=P, npad=P, A=P, B=P, Y=P, **kw):
    cfg = q.gemm_i8(64, 64, num_experts=E, **kw)
    return _status(q.qdg_moe_gemm_i8, cfg, A, P, P, B, P, P, sid, blk, npad, T, top_k, bm, 0, Y)


def test_moe_refusals():
    inv, uns, mis = q.QDG_ERR_INVALID_ARG, q.QDG_ERR_UNSUPPORTED, q.QDG_ERR_MISALIGNED
    assert _moe(T=0) == q.QDG_OK and _moe(T=-1) == inv
    assert _moe(E=0) == inv and _moe(E=1025) == uns
    assert _moe(top_k=0) == inv and _moe(top_k=33) == inv
    assert _moe(bm=8) == uns and _moe(bm=256) == uns
    assert _moe(T=(1 << 19) + 1) == uns
    assert _moe(sid=None) == inv and _moe(blk=None) == inv and _moe(npad=None) == inv
    assert _moe(sid=P + 2) == mis and _moe(npad=P + 1) == mis
    assert _moe(T=1 << 17, top_k=8, lda=1 << 15) == uns  # 4 GiB of token rows
    assert _moe(A=None) == inv and _moe(Y=None) == inv and _moe(B=P + 4) == mis


def test_more_tiles_than_a_launch_holds():
    """2^20 pairs in 16-row blocks and 2^16 columns: refused before anything is enqueued."""
    cfg = q.gemm_i8(1 << 16, 64, num_experts=8)
    assert _status(q.qdg_moe_gemm_i8, cfg, P, P, P, P, P, P, P, P, P, 1 << 19, 2, 16, 0, P) == q.QDG_ERR_UNSUPPORTED
    assert _gemm(M=1 << 26, n=1 << 20, k=16) == q.QDG_ERR_UNSUPPORTED


def test_messages_name_the_cause():
    with pytest.raises(q.QdgError, match="num_groups must divide"):
        q.qdg_moe_route(q.route(64, 4, num_groups=3), P, 64, None, 1, P, P)
    with pytest.raises(q.QdgError, match="multiples of 16"):
        q.qdg_gemm_i8(q.gemm_i8(64, 64, lda=72), P, P, None, P, P, None, P, 1)


def test_route_refuses_what_one_launch_cannot_hold():
    """Four tokens a block of 256 threads, below 2^32 threads: 2^26 - 4 tokens are the most."""
    for t in ((1 << 26) - 3, 1 << 26, (1 << 26) + 1):
        assert _route(T=t) == q.QDG_ERR_UNSUPPORTED


def test_workspace_of_the_largest_batch_serves_smaller_ones():
    """Fewer rows may be split where many are not: the bytes never fall with M."""
    for n, k, epi in ((4096, 14336, 0), (4096, 4096, 0), (576, 7168, 0), (130, 65536, 1), (9002, 40001, 0), (28672, 8192, 1)):
        cfg = q.gemm_i8(n, k, epilogue=epi)
        need = [q.qdg_gemm_i8_workspace(cfg, m) for m in list(range(0, 700)) + [4096, 32769, 1 << 26]]
        assert need == sorted(need), (n, k)
    cfg = q.gemm_i8(4096, 14336)
    assert q.qdg_gemm_i8_workspace(cfg, 4096) >= q.qdg_gemm_i8_workspace(cfg, 64) > 0
    assert q.qdg_gemm_i8_workspace(q.gemm_i8(4096, 1920), 1 << 26) == 0  # no K that is ever split
    assert q.qdg_gemm_i8_workspace(q.gemm_i8(33000, 65536), 1 << 26) == 0  # nor so many columns
    # a split product is refused a workspace that is too small or misaligned, others need none
    for M, n, k in ((33, 514, 16386), (64, 128, 8192), (300, 128, 65536)):
        need = q.qdg_gemm_i8_workspace(q.gemm_i8(n, k), M)
        assert need > 0
        assert _gemm(M=M, n=n, k=k, ws_bytes=need - 1) == q.QDG_ERR_WORKSPACE
        assert _gemm(M=M, n=n, k=k, ws=None) == q.QDG_ERR_WORKSPACE
        assert _gemm(M=M, n=n, k=k, ws=P + 8) == q.QDG_ERR_MISALIGNED


def test_gemm_describe():
    record = q.qdg_gemm_i8_describe(q.gemm_i8(4096, 4096), 16)
    assert record == ("gemm-i8 dense n=4096 k=4096 M=16: family=rows block_m=16 block_n=16 split_k=1 columns=4096 "
                      "rest=none epilogue=none arch=gfx950")
    record = q.qdg_gemm_i8_describe(q.gemm_i8(4610, 900, epilogue=q.QDG_EPI_SILU_MUL), 4096)
    assert "family=tile block_m=256 block_n=256 split_k=1 columns=4096 rest=128x128 epilogue=silu_mul" in record
    assert "split_k=8" in q.qdg_gemm_i8_describe(q.gemm_i8(514, 16386), 33)
    assert q.qdg_gemm_i8_describe(q.gemm_i8(64, 64), 0).startswith("gemm-i8 dense n=64 k=64 M=0: ")
    describe = q.load().qdg_gemm_i8_describe
    assert describe(None, 1, None, 0) == -1
    for cfg, M in ((q.gemm_i8(0, 64), 1), (q.gemm_i8(64, 64, num_experts=2), 1), (q.gemm_i8(64, 64), -1),
                   (q.gemm_i8(64, 64), (1 << 26) + 1)):
        with pytest.raises(q.QdgError):
            q.qdg_gemm_i8_describe(cfg, M)


@pytest.mark.parametrize("raw", [True, False])
def test_current_stream_handle(monkeypatch, raw):
    """The handle of the current device's current stream, from torch's raw handle where that exists."""
    import types

    import torch
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 3)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: types.SimpleNamespace(cuda_stream=1000 + torch.cuda.current_device()))
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: 1000 + d, raising=False)
    if not raw:
        monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream")
    assert q.current_stream() == 1003
