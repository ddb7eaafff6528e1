"""qdg_moe_route against the float64 reference: ids equal, weights within
2^-21 relative (the documented bound), over every score, bias, grouping and
logit type, expert counts around the wave's width, ties, masks and keys that
binary32 cannot tell apart."""

import numpy as np
import pytest
import torch

import quantized_dequant_gemm_amd as q
from oracle import ops

pytestmark = pytest.mark.gpu

DT = {"bf16": (q.QDG_L_BF16, torch.bfloat16), "f16": (q.QDG_L_F16, torch.float16), "f32": (q.QDG_L_F32, torch.float32)}
SCORE = {"softmax": q.QDG_SCORE_SOFTMAX, "sigmoid": q.QDG_SCORE_SIGMOID}
GROUP = {"max": q.QDG_GROUP_MAX, "top2": q.QDG_GROUP_TOP2}


def run(x, top_k, ltype="f32", score="softmax", bias=None, groups=1, topk_groups=1, group_score="max", renorm=False,
        scale=1.0, pad=0):
    """(ids, weights, flag) of the kernel on logits x (numpy), and the values it saw."""
    t, e = x.shape
    code, dt = DT[ltype]
    buf = torch.full((t, e + pad), 7.0, dtype=dt, device="cuda")
    buf[:, :e] = torch.from_numpy(np.ascontiguousarray(x)).cuda().to(dt)
    b = None if bias is None else torch.from_numpy(np.asarray(bias, np.float32)).cuda()
    ids = torch.full((t + 2, top_k), -7, dtype=torch.int32, device="cuda")
    w = torch.full((t + 2, top_k), -7.0, dtype=torch.float32, device="cuda")
    flag = torch.zeros(1, dtype=torch.int32, device="cuda")
    cfg = q.route(e, top_k, ltype=code, score=SCORE[score], num_groups=groups, topk_groups=topk_groups,
                  group_score=GROUP[group_score], renormalize=int(renorm), scale=scale)
    q.qdg_moe_route(cfg, buf.data_ptr(), e + pad, None if b is None else b.data_ptr(), t, ids.data_ptr(),
                    w.data_ptr(), q.current_stream(), flag.data_ptr())
    torch.cuda.synchronize()
    assert (ids[t:] == -7).all() and (w[t:] == -7.0).all()  # rows behind the last token
    seen = buf[:, :e].float().cpu().numpy()
    return ids[:t].cpu().numpy(), w[:t].cpu().numpy(), int(flag.item()), seen


def check(x, top_k, **kw):
    ids, w, flag, seen = run(x, top_k, **kw)
    ref_kw = {k: v for k, v in kw.items() if k not in ("ltype", "pad")}
    if ref_kw.get("bias") is not None:
        ref_kw["bias"] = np.asarray(ref_kw["bias"], np.float32)
    rid, rw, bad = ops.route(seen, top_k, **ref_kw)
    np.testing.assert_array_equal(ids, rid)
    assert np.all(np.abs(w - rw) <= 2.0 ** -21 * np.abs(rw)), np.max(np.abs(w - rw) / np.maximum(np.abs(rw), 1e-300))
    assert flag == (q.QDG_FLAG_BAD_LOGIT if bad else 0)
    return ids, w


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("with_bias", [False, True])
@pytest.mark.parametrize("e,top_k", [(1, 1), (2, 2), (7, 3), (60, 4), (64, 8), (65, 8), (128, 6), (160, 6), (256, 8),
                                     (257, 32), (384, 8), (512, 10), (1000, 17), (1024, 32)])
def test_choice_and_weights(qdg, score, with_bias, e, top_k):
    rng = np.random.default_rng(1000 * e + top_k)
    bias = 0.1 * rng.standard_normal(e) if with_bias else None
    for i, (t, lt) in enumerate(((1, "bf16"), (5, "f16"), (37, "f32"))):
        x = 2.0 * rng.standard_normal((t, e))
        check(x, top_k, ltype=lt, score=score, bias=bias, renorm=bool((i + e) & 1), scale=(1.0, 2.5, -0.5)[i],
              pad=(0, 3, 8)[i])


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("with_bias", [False, True])
@pytest.mark.parametrize("group_score", ["max", "top2"])
@pytest.mark.parametrize("e,groups,topk_groups,top_k", [(256, 8, 4, 8), (256, 8, 1, 8), (96, 32, 3, 5), (64, 64, 8, 8),
                                                        (130, 2, 1, 6), (160, 8, 3, 6), (1024, 64, 7, 32),
                                                        (250, 5, 5, 9), (12, 4, 4, 12)])
def test_groups(qdg, score, with_bias, group_score, e, groups, topk_groups, top_k):
    rng = np.random.default_rng(e + 7 * groups + top_k)
    bias = 0.1 * rng.standard_normal(e) if with_bias else None
    check(2.0 * rng.standard_normal((21, e)), top_k, ltype="bf16", score=score, bias=bias, groups=groups,
          topk_groups=topk_groups, group_score=group_score, renorm=True, scale=2.5)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups", [1, 8])
def test_ties_take_the_lowest_index(qdg, score, groups):
    rng = np.random.default_rng(3)
    kw = dict(score=score, groups=groups, topk_groups=max(1, groups // 2), group_score="top2")
    ids, _ = check(np.zeros((3, 256)), 8, **kw)
    assert ids.tolist() == [list(range(8))] * 3
    coarse = rng.integers(-2, 3, (40, 256)).astype(np.float64)  # five values only
    check(coarse, 8, **kw)
    check(coarse, 8, bias=np.zeros(256), **kw)
    check(coarse, 8, bias=rng.integers(0, 2, 256) * 0.25, **kw)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups,topk_groups", [(1, 1), (8, 3)])
@pytest.mark.parametrize("with_bias", [False, True])
@pytest.mark.parametrize("renorm", [False, True])
def test_masks_infinities_nan(qdg, score, groups, topk_groups, with_bias, renorm):
    rng = np.random.default_rng(5)
    e = 64
    x = 2.0 * rng.standard_normal((12, e))
    x[0] = -np.inf                       # nothing left
    x[1, 3:] = -np.inf                   # fewer than top_k left
    x[2, :] = np.nan
    x[3, 5] = np.nan
    x[4, [7, 40]] = np.inf               # both, in order of the index
    x[5, ::2] = -np.inf
    x[6, :32] = -np.inf                  # whole groups masked
    x[7] = float(np.finfo(np.float32).min)   # the type's lowest finite value is not masked
    x[8, 1:] = float(np.finfo(np.float32).min)
    x[9] = 1000.0
    x[10, :8] = -1000.0
    bias = None
    if with_bias:
        bias = 0.1 * rng.standard_normal(e)
        bias[[2, 50]] = [-np.inf, np.nan]
        bias[9] = np.inf
    check(x, 6, score=score, bias=bias, groups=groups, topk_groups=topk_groups, group_score="top2", renorm=renorm)
    check(x, 6, score=score, bias=bias, groups=groups, topk_groups=topk_groups, group_score="max", renorm=renorm)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("with_bias", [False, True])
@pytest.mark.parametrize("renorm", [False, True])
def test_logits_far_apart(qdg, score, with_bias, renorm):
    """Differences past binary32's largest value, and scores past its smallest."""
    e, big = 48, float(np.finfo(np.float32).max)
    rng = np.random.default_rng(19)
    x = 2.0 * rng.standard_normal((8, e))
    x[0, 3], x[0, 9] = np.inf, -big
    x[1] = -big
    x[1, 5] = big
    x[2, ::2], x[2, 1::2] = 3e38, -3e38
    x[3] = -700.0 + np.arange(e)
    x[4] = -90.0 - 0.25 * np.arange(e)
    x[5] = -3000.0
    x[5, 7] = -2995.0
    x[6] = np.linspace(-120.0, 0.0, e)
    x[7] = np.linspace(80.0, 100.0, e)
    x = x.astype(np.float32).astype(np.float64)
    bias = np.where(np.arange(e) % 3 == 0, 1.5, 0.0) if with_bias else None
    ids, w, _, seen = run(x, 6, score=score, bias=bias, renorm=renorm)
    rid, rw, _ = ops.route(seen, 6, score=score, bias=bias, renorm=renorm)
    np.testing.assert_array_equal(ids, rid)
    # half a step of a subnormal binary32 more where the weight is one
    assert np.all(np.abs(w - rw) <= 2.0 ** -21 * np.abs(rw) + 2.0 ** -150), (w, rw)


@pytest.mark.parametrize("ltype", ["bf16", "f16"])
def test_lowest_value_of_the_type(qdg, ltype):
    x = np.full((2, 70), float(torch.finfo(DT[ltype][1]).min))
    x[1, 33] = 0.0
    check(x, 5, ltype=ltype, renorm=True)
    check(x, 5, ltype=ltype, score="sigmoid", bias=np.zeros(70))


@pytest.mark.parametrize("groups", [1, 4])
def test_keys_closer_than_binary32_tells(qdg, groups):
    """bias_e = f32(c - s_e) puts all keys of a row within about 2^-25 of c:
    their order is only visible in binary64."""
    rng = np.random.default_rng(11)
    e = 128
    x = rng.uniform(-1.0, 3.0, (1, e)).astype(np.float32).astype(np.float64)
    s = 1.0 / (1.0 + np.exp(-x[0]))
    bias = (1.0 - s).astype(np.float32)
    key = np.sort(s + bias.astype(np.float64))
    assert 0 < np.min(np.diff(key)) and key[-1] - key[0] < 2.0 ** -23  # distinct, and one or two binary32 steps in all
    check(np.repeat(x, 3, axis=0), 8, score="sigmoid", bias=bias, groups=groups, topk_groups=max(1, groups // 2),
          group_score="top2")
    # the same against rows whose other keys lie far below
    far = np.full(e, -4.0, np.float32)
    far[:24] = bias[:24]
    check(x, 8, score="sigmoid", bias=far, groups=groups, topk_groups=max(1, groups // 2), group_score="max")


def test_many_tokens(qdg):
    rng = np.random.default_rng(13)
    check(2.0 * rng.standard_normal((3001, 64)), 6, ltype="bf16", renorm=True)
    check(2.0 * rng.standard_normal((1025, 256)), 8, ltype="f32", score="sigmoid", bias=0.1 * rng.standard_normal(256),
          groups=8, topk_groups=4, group_score="top2", renorm=True, scale=2.5)


def test_replayed_graph_and_other_stream(qdg):
    rng = np.random.default_rng(17)
    x = torch.from_numpy(rng.standard_normal((9, 256)).astype(np.float32)).cuda()
    ids = torch.zeros((9, 8), dtype=torch.int32, device="cuda")
    w = torch.zeros((9, 8), dtype=torch.float32, device="cuda")
    cfg = q.route(256, 8, ltype=q.QDG_L_F32, renormalize=1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        q.qdg_moe_route(cfg, x.data_ptr(), 256, None, 9, ids.data_ptr(), w.data_ptr(), side.cuda_stream)
    torch.cuda.synchronize()
    want, _, _ = ops.route(x.cpu().numpy(), 8, renorm=True)
    np.testing.assert_array_equal(ids.cpu().numpy(), want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        q.qdg_moe_route(cfg, x.data_ptr(), 256, None, 9, ids.data_ptr(), w.data_ptr(), q.current_stream())
    for _ in range(4):
        y = rng.standard_normal((9, 256)).astype(np.float32)
        x.copy_(torch.from_numpy(y))
        g.replay()
        torch.cuda.synchronize()
        rid, rw, _ = ops.route(y, 8, renorm=True)
        np.testing.assert_array_equal(ids.cpu().numpy(), rid)
        assert np.all(np.abs(w.cpu().numpy() - rw) <= 2.0 ** -21 * rw)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("per", [2, 3, 20, 32])
def test_group_values_past_binary32(qdg, score, per):
    """Sums of two keys below (or above) binary32's range: finite in binary64, so ahead of a group whose experts are
    all masked, and in order among themselves."""
    low, inf = float(np.finfo(np.float32).min), np.inf
    rng = np.random.default_rng(per)
    for values in ([-inf, -3e38], [-3.2e38, -2e38], [low, -2.5e38], [-inf, low, -3e38, -inf], [low, low, low, -inf],
                   [2e38, 3e38], [low, -3e38, -1.8e38, -1e38, 0.0, 1.8e38, 3e38, -inf]):
        groups = len(values)
        bias = np.repeat(np.array(values), per)
        x = rng.standard_normal((5, groups * per))
        for topk_groups in range(1, groups):
            check(x, min(per, 4), score=score, bias=bias, groups=groups, topk_groups=topk_groups, group_score="top2")
    # one finite key of a pair next to a masked one
    bias = np.full(4 * per, -inf)
    bias[per:per + 2] = -3e38
    bias[2 * per] = low
    check(rng.standard_normal((5, 4 * per)), 1, score=score, bias=bias, groups=4, topk_groups=1, group_score="top2")
    check(rng.standard_normal((5, 4 * per)), 2, score=score, bias=bias, groups=4, topk_groups=2, group_score="top2")


@pytest.mark.parametrize("groups", [1, 4])
@pytest.mark.parametrize("group_score", ["max", "top2"])
def test_sigmoid_scores_below_the_smallest_normal(qdg, groups, group_score):
    """sigmoid(-725) = 2^-1046 is a binary64 number (a subnormal one with 28 bits): scores there have an order, group
    values and renormalised weights (28 bits in, one step of exp and half steps of sum and quotient: far below 2^-21)."""
    e = 32
    x = np.empty((3, e))
    x[0] = -725.0 + 0.25 * np.arange(e)
    x[1] = -711.0 - 0.25 * np.arange(e)
    x[2] = -718.0
    check(x, 6, score="sigmoid", groups=groups, topk_groups=max(1, groups // 2), group_score=group_score, renorm=True)
    check(x, 6, score="sigmoid", bias=np.zeros(e), groups=groups, topk_groups=max(1, groups // 2),
          group_score=group_score, renorm=True)


def test_largest_number_of_tokens(qdg):
    t = (1 << 26) - 4
    x = torch.zeros(t, dtype=torch.float16, device="cuda")
    x[-1] = 3.0
    ids = torch.full((t + 1,), -7, dtype=torch.int32, device="cuda")
    w = torch.full((t + 1,), -7.0, dtype=torch.float32, device="cuda")
    cfg = q.route(1, 1, ltype=q.QDG_L_F16, score=q.QDG_SCORE_SIGMOID)
    q.qdg_moe_route(cfg, x.data_ptr(), 1, None, t, ids.data_ptr(), w.data_ptr(), q.current_stream())
    torch.cuda.synchronize()
    assert int(ids[:t].abs().max()) == 0 and bool((w[:t - 1] == 0.5).all())
    assert abs(float(w[t - 1]) - 1 / (1 + np.exp(-3.0))) < 2.0 ** -21
    assert int(ids[t]) == -7 and float(w[t]) == -7.0
