"""Measured cases of the router and of the 8-bit integer products.

Four operators that stand around and inside one MoE (or dense) layer served
with 8-bit weights and activations:

  route          expert scores -> top-k expert ids and weights
  quantize_zp    bf16 activations -> int8 codes with one scale and one zero
                 point for each token
  gemm_i8        Y = a_scale * b_scale * sum_k (qa - za) * qb + bias over
                 operands as they are stored (row-major, strided), with an
                 optional SiLU * mul of a fused gate+up layer
  moe_gemm_i8    the same product, grouped by expert

``run`` computes a case in its plain form (elementary torch operations) or,
where ``own`` is true, through the library's entry points. ``exact`` is the
definition in 64 bits, written apart from the plain form.
"""

import math

import torch

own = False

OTYPES = {"bf16": torch.bfloat16, "f32": torch.float32, "i32": torch.int32}
LTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def listed():
    return [
        # one decoded token: 256 experts in 8 groups, 4 of them kept, top 8 by
        # sigmoid score + balance bias, weights renormalised and scaled
        _route("route 1 token 256 experts grouped", 1, 256, 8, "bf16", "sigmoid", True, 8, 4, "top2", True, 2.5),
        # a decode batch of a small softmax router, odd numbers of tokens and experts
        _route("route 333 tokens 60 experts", 333, 60, 4, "f16", "softmax", False, 1, 1, "max", False, 1.0),
        # a long prefill chunk of the grouped router, float32 logits
        _route("route 8192 tokens 256 experts grouped", 8192, 256, 8, "f32", "sigmoid", True, 8, 4, "top2", True, 2.5),
        # a prefill chunk of a plain renormalised softmax router
        _route("route 4096 tokens 256 experts", 4096, 256, 8, "bf16", "softmax", False, 1, 1, "max", True, 1.0),
        # the activations of a decode batch before a projection
        _quant("quantize 16 x 4096", 16, 4096),
        # the activations of a prefill chunk before a down projection
        _quant("quantize 4096 x 14336", 4096, 14336),
        # one decoded token through a square projection
        _gemm("gemm 1 x 4096 x 4096", 1, 4096, 4096, True, False, "bf16", "none"),
        # a decode batch through the up projection
        _gemm("gemm 16 x 14336 x 4096", 16, 14336, 4096, True, True, "bf16", "none"),
        # a ragged batch through a layer with odd sizes and padded rows
        _gemm("gemm 250 x 4100 x 4090", 250, 4100, 4090, True, True, "f32", "none"),
        # a prefill chunk through the up projection
        _gemm("gemm 4096 x 14336 x 4096", 4096, 14336, 4096, True, False, "bf16", "none"),
        # a decode batch of 64 tokens through the experts' down projection
        _moe("moe down 64 tokens", 64, 256, 8, 7168, 2048, 16, True, True, False, "bf16", "none"),
        # a prefill chunk of 4096 tokens through the experts' fused gate+up projection
        _moe("moe gate+up 4096 tokens", 4096, 256, 8, 4096, 7168, 64, False, True, False, "bf16", "silu_mul"),
    ]


def _route(name, T, E, top_k, ltype, score, bias, groups, topk_groups, group_score, renorm, scale):
    return {"name": name, "op": "route", "T": T, "E": E, "top_k": top_k, "ltype": ltype, "score": score, "bias": bias,
            "groups": groups, "topk_groups": topk_groups, "group_score": group_score, "renorm": renorm, "scale": scale}


def _quant(name, M, k):
    return {"name": name, "op": "quantize_zp", "M": M, "k": k}


def _gemm(name, M, n, k, zeros, bias, otype, epilogue):
    return {"name": name, "op": "gemm_i8", "M": M, "n": n, "k": k, "zeros": zeros, "bias": bias, "otype": otype,
            "epilogue": epilogue}


def _moe(name, T, E, top_k, n, k, block_m, a_per_pair, zeros, bias, otype, epilogue):
    return {"name": name, "op": "moe_gemm_i8", "T": T, "E": E, "top_k": top_k, "n": n, "k": k, "block_m": block_m,
            "a_per_pair": a_per_pair, "zeros": zeros, "bias": bias, "otype": otype, "epilogue": epilogue}


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["route", "quantize_zp", "gemm_i8", "gemm_i8", "moe_gemm_i8"])
    if op == "route":
        groups = rng.choice([1, 1, 2, 4, 8])
        E = groups * max(2, _log_int(rng, 8, 512) // groups)
        topk_groups = rng.randint(1, groups)
        top_k = rng.randint(1, min(16, topk_groups * (E // groups)))
        T = _log_int(rng, 1, min(8192, (8192 * 256) // E))
        case = _route("", T, E, top_k, rng.choice(sorted(LTYPES)), rng.choice(["softmax", "sigmoid"]),
                      rng.random() < 0.5, groups, topk_groups, rng.choice(["max", "top2"]), rng.random() < 0.5,
                      rng.choice([1.0, 2.5]))
    elif op == "quantize_zp":
        k = _log_int(rng, 64, 14336)
        case = _quant("", _log_int(rng, 1, 4096), k)
    elif op == "gemm_i8":
        M, n, k = _log_int(rng, 1, 4096), _log_int(rng, 64, 14336), _log_int(rng, 64, 14336)
        k = min(k, (4096 * 14336 * 4096) // (M * n))
        epilogue = rng.choice(["none", "none", "silu_mul"])
        n = n if epilogue == "none" else n // 2 * 2
        otype = rng.choice(["bf16", "bf16", "f32", "i32"] if epilogue == "none" else ["bf16", "f32"])
        case = _gemm("", M, n, k, rng.random() < 0.6, otype != "i32" and rng.random() < 0.5, otype, epilogue)
    else:
        E = _log_int(rng, 8, 256)
        top_k = rng.randint(1, 8)
        T = _log_int(rng, 1, 4096)
        n, k = 2 * _log_int(rng, 64, 2048), _log_int(rng, 128, 7168)
        epilogue = rng.choice(["none", "silu_mul"])
        rows = T * top_k / E
        block_m = 16 if rows <= 4 else 32 if rows <= 12 else 64 if rows <= 256 else 128
        case = _moe("", T, E, top_k, n, k, block_m, rng.random() < 0.5, rng.random() < 0.6, rng.random() < 0.3,
                    rng.choice(["bf16", "f32"]), epilogue)
    del case["name"]
    return case


# ------------------------------------------------------------------ inputs

def _round_up(x, m):
    return (x + m - 1) // m * m


def _codes(gen, rows, ld, spread):
    """int8 codes of normal values: bytes behind a row's end are codes too (the padding of a strided operand)."""
    out = torch.empty((rows, ld), dtype=torch.int8, device="cuda")
    step = max(1, (1 << 28) // ld)
    for r in range(0, rows, step):
        x = torch.randn((min(step, rows - r), ld), generator=gen, device="cuda")
        out[r:r + step] = x.mul_(spread).round_().clamp_(-127, 127)
    return out


def _a_operand(case, gen, rows, s):
    """Codes of asymmetrically quantized activations (values behind an
    activation function lie mostly on one side of zero) or of symmetric ones."""
    k = case["k"]
    s["lda"] = _round_up(k, 16)
    s["A"] = _codes(gen, rows, s["lda"], 40.0)
    s["a_scales"] = torch.rand(rows, generator=gen, device="cuda") * 0.02 + 0.01
    s["a_zeros"] = None
    if case["zeros"]:
        s["a_zeros"] = torch.randint(-128, 1, (rows,), generator=gen, device="cuda", dtype=torch.int32)


def _b_operand(case, gen, experts, s):
    n, k = case["n"], case["k"]
    s["ldb"] = _round_up(k, 16)
    s["B"] = _codes(gen, experts * n, s["ldb"], 30.0).view(experts, n, s["ldb"])
    s["b_scales"] = torch.rand((experts, n), generator=gen, device="cuda") * 4e-4 + 4e-4
    s["bias"] = torch.randn((experts, n), generator=gen, device="cuda") if case["bias"] else None


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op = case["op"]
    s = {"case": case}
    if op == "route":
        T, E = case["T"], case["E"]
        s["logits"] = (2.0 * torch.randn((T, E), generator=gen, device="cuda")).to(LTYPES[case["ltype"]])
        s["bias"] = 0.1 * torch.randn(E, generator=gen, device="cuda") if case["bias"] else None
        if own:
            import quantized_dequant_gemm_amd as q
            s["cfg"] = q.route(E, case["top_k"], ltype={"bf16": q.QDG_L_BF16, "f16": q.QDG_L_F16, "f32": q.QDG_L_F32}[case["ltype"]],
                               score=q.QDG_SCORE_SIGMOID if case["score"] == "sigmoid" else q.QDG_SCORE_SOFTMAX,
                               num_groups=case["groups"], topk_groups=case["topk_groups"],
                               group_score=q.QDG_GROUP_TOP2 if case["group_score"] == "top2" else q.QDG_GROUP_MAX,
                               renormalize=int(case["renorm"]), scale=case["scale"])
            s["ids"] = torch.empty((T, case["top_k"]), dtype=torch.int32, device="cuda")
            s["weights"] = torch.empty((T, case["top_k"]), dtype=torch.float32, device="cuda")
        return s
    if op == "quantize_zp":
        M, k = case["M"], case["k"]
        s["lda"], s["ldq"] = _round_up(k, 8), _round_up(k, 16)
        x = torch.randn((M, s["lda"]), generator=gen, device="cuda")
        s["x"] = (torch.nn.functional.silu(x) * (1.0 + torch.rand((M, 1), generator=gen, device="cuda"))).to(torch.bfloat16)
        if own:
            s["qa"] = torch.empty((M, s["ldq"]), dtype=torch.int8, device="cuda")
            s["a_scales"] = torch.empty(M, dtype=torch.float32, device="cuda")
            s["a_zeros"] = torch.empty(M, dtype=torch.int32, device="cuda")
        return s
    moe = op == "moe_gemm_i8"
    rows = case["M"] if not moe else case["T"] * (case["top_k"] if case["a_per_pair"] else 1)
    experts = case["E"] if moe else 1
    _a_operand(case, gen, rows, s)
    _b_operand(case, gen, experts, s)
    if moe:
        _routing(case, gen, s)
    out_rows = case["T"] * case["top_k"] if moe else case["M"]
    cols = case["n"] // 2 if case["epilogue"] == "silu_mul" else case["n"]
    if own:
        import quantized_dequant_gemm_amd as q
        s["Y"] = torch.empty((out_rows, cols), dtype=OTYPES[case["otype"]], device="cuda")
        s["cfg"] = q.gemm_i8(case["n"], case["k"], lda=s["lda"], ldb=s["ldb"], ldy=cols, num_experts=experts,
                             otype={"bf16": q.QDG_O_BF16, "f32": q.QDG_O_F32, "i32": q.QDG_O_I32}[case["otype"]],
                             epilogue=q.QDG_EPI_SILU_MUL if case["epilogue"] == "silu_mul" else q.QDG_EPI_NONE)
        if not moe:
            s["ws_bytes"] = q.qdg_gemm_i8_workspace(s["cfg"], case["M"])
            s["ws"] = torch.empty(max(1, s["ws_bytes"]), dtype=torch.uint8, device="cuda")
    return s


def _routing(case, gen, s):
    """The expert sort of a seeded softmax router's choice (top-k of the logits)."""
    T, E, top_k, bm = case["T"], case["E"], case["top_k"], case["block_m"]
    ids = torch.randn((T, E), generator=gen, device="cuda").topk(top_k, dim=1).indices.reshape(-1)
    order = torch.argsort(ids, stable=True)
    counts = torch.bincount(ids, minlength=E)
    padded = (counts + bm - 1) // bm * bm
    first, start = counts.cumsum(0) - counts, padded.cumsum(0) - padded
    expert = ids[order]
    capacity = _round_up(T * top_k + E * (bm - 1), bm)
    s["sorted_ids"] = torch.full((capacity,), T * top_k, dtype=torch.int32, device="cuda")
    s["sorted_ids"][start[expert] + torch.arange(T * top_k, device="cuda") - first[expert]] = order.to(torch.int32)
    s["blocks"] = int(padded.sum()) // bm
    s["block_expert"] = torch.full((capacity // bm,), -1, dtype=torch.int32, device="cuda")
    s["block_expert"][:s["blocks"]] = torch.repeat_interleave(torch.arange(E, device="cuda"), padded // bm).to(torch.int32)
    s["num_padded"] = padded.sum().to(torch.int32).reshape(1)
    s["expert_ids"] = ids


# ------------------------------------------------------------------ one pass

def _ptr(t):
    return None if t is None else t.data_ptr()


def run(s):
    if own:
        return _run_own(s)
    op = s["case"]["op"]
    if op == "route":
        return _route_plain(s)
    if op == "quantize_zp":
        return _quantize_plain(s)
    return _moe_plain(s) if op == "moe_gemm_i8" else _gemm_plain(s)


def _run_own(s):
    import quantized_dequant_gemm_amd as q
    case, stream = s["case"], q.current_stream()
    op = case["op"]
    if op == "route":
        q.qdg_moe_route(s["cfg"], s["logits"].data_ptr(), case["E"], _ptr(s["bias"]), case["T"], s["ids"].data_ptr(),
                        s["weights"].data_ptr(), stream)
        return s["ids"], s["weights"]
    if op == "quantize_zp":
        q.qdg_quantize_act_zp(s["x"].data_ptr(), s["lda"], case["M"], case["k"], s["qa"].data_ptr(), s["ldq"],
                              s["a_scales"].data_ptr(), s["a_zeros"].data_ptr(), stream)
        return s["qa"][:, :case["k"]], s["a_scales"], s["a_zeros"]
    if op == "gemm_i8":
        q.qdg_gemm_i8(s["cfg"], s["A"].data_ptr(), s["a_scales"].data_ptr(), _ptr(s["a_zeros"]), s["B"].data_ptr(),
                      s["b_scales"].data_ptr(), _ptr(s["bias"]), s["Y"].data_ptr(), case["M"], s["ws"].data_ptr(),
                      s["ws_bytes"], stream)
    else:
        q.qdg_moe_gemm_i8(s["cfg"], s["A"].data_ptr(), s["a_scales"].data_ptr(), _ptr(s["a_zeros"]),
                          s["B"].data_ptr(), s["b_scales"].data_ptr(), _ptr(s["bias"]), s["sorted_ids"].data_ptr(),
                          s["block_expert"].data_ptr(), s["num_padded"].data_ptr(), case["T"], case["top_k"],
                          case["block_m"], int(case["a_per_pair"]), s["Y"].data_ptr(), stream)
    return s["Y"]


def _first(key, count):
    """The `count` largest of each row, equal ones in ascending index (a stable sort)."""
    return torch.sort(key, dim=1, descending=True, stable=True).indices[:, :count]


def _route_plain(s):
    """Scores and keys in 64 bits: two keys may lie closer than 32 bits tell."""
    case = s["case"]
    T, E, G = case["T"], case["E"], case["groups"]
    x = s["logits"].double()
    if case["score"] == "sigmoid":
        score = 1.0 / (1.0 + torch.exp(-x))
    else:
        e = torch.exp(x - x.amax(dim=1, keepdim=True))
        score = e / e.sum(dim=1, keepdim=True)
    key = x if s["bias"] is None else score + s["bias"].double()
    if G > 1:
        value = (score if s["bias"] is None else key).view(T, G, E // G)
        if case["group_score"] == "top2":
            value = torch.sort(value, dim=2, descending=True).values[:, :, :2].sum(dim=2)
        else:
            value = value.amax(dim=2)
        kept = torch.zeros((T, G), dtype=torch.bool, device=x.device)
        kept.scatter_(1, _first(value, case["topk_groups"]), True)
        key = key.masked_fill(~kept.repeat_interleave(E // G, dim=1), -math.inf)
    ids = _first(key, case["top_k"])
    w = score.gather(1, ids)
    if case["renorm"]:
        w = w / w.sum(dim=1, keepdim=True)
    return ids.to(torch.int32), (w * case["scale"]).float()


def _quantize_plain(s):
    """The codes are whole numbers that the product multiplies; each decision
    is taken in 64 bits, since a value next to a border goes one way only."""
    x = s["x"][:, :s["case"]["k"]].double()
    lo, hi = x.amin(dim=1).clamp(max=0.0), x.amax(dim=1).clamp(min=0.0)
    scale = ((hi - lo) / 255.0).float().clamp(min=2.0 ** -126)
    scale = torch.where(hi > lo, scale, torch.ones_like(scale))
    inv = 1.0 / scale.double()
    zero = torch.where(hi > lo, torch.round(-128.0 - lo * inv).clamp(-128.0, 127.0), torch.zeros_like(lo))
    codes = (torch.round(x * inv[:, None]) + zero[:, None]).clamp(-128.0, 127.0)
    return codes.to(torch.int8), scale, zero.to(torch.int32)


def _product(case, a, a_scales, a_zeros, b, b_scales, bias):
    """The integer sums need more than the 24 bits of a float32: 64 bits."""
    a, b = a[:, :case["k"]].double(), b[:, :case["k"]].double()
    if a_zeros is not None:
        a = a - a_zeros[:, None]
    y = a @ b.t()
    if case["otype"] == "i32":
        return y.to(torch.int32)
    y = y * a_scales.double()[:, None] * b_scales.double()
    if bias is not None:
        y = y + bias
    if case["epilogue"] == "silu_mul":
        g, u = y[:, :case["n"] // 2], y[:, case["n"] // 2:]
        y = g / (1.0 + torch.exp(-g)) * u
    return y.to(OTYPES[case["otype"]])


def _gemm_plain(s):
    return _product(s["case"], s["A"], s["a_scales"], s["a_zeros"], s["B"][0], s["b_scales"][0],
                    None if s["bias"] is None else s["bias"][0])


def _moe_plain(s):
    """Block by block of the expert-sorted rows; padding goes to a last row that is cut off."""
    case = s["case"]
    pairs, bm = case["T"] * case["top_k"], case["block_m"]
    cols = case["n"] // 2 if case["epilogue"] == "silu_mul" else case["n"]
    out = torch.empty((pairs + 1, cols), dtype=OTYPES[case["otype"]], device="cuda")
    for blk in range(s["blocks"]):
        ids = s["sorted_ids"][blk * bm:(blk + 1) * bm].long()
        rows = ids.clamp(max=pairs - 1)
        if not case["a_per_pair"]:
            rows = rows // case["top_k"]
        e = s["block_expert"][blk:blk + 1].long()
        out[ids] = _product(case, s["A"][rows], s["a_scales"][rows], None if s["a_zeros"] is None else s["a_zeros"][rows],
                            s["B"].index_select(0, e)[0], s["b_scales"].index_select(0, e)[0],
                            None if s["bias"] is None else s["bias"].index_select(0, e)[0])
    return out[:pairs]


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    op = case["op"]
    if op == "route":
        T, E, k = case["T"], case["E"], case["top_k"]
        size = 4 if case["ltype"] == "f32" else 2
        return {"bytes": T * E * size + (4 * E if case["bias"] else 0) + T * k * 8, "flops": T * E * 4}
    if op == "quantize_zp":
        return {"bytes": case["M"] * (case["k"] * 3 + 8), "flops": case["M"] * case["k"] * 4}
    n, k = case["n"], case["k"]
    esz = 2 if case["otype"] == "bf16" else 4
    cols = n // 2 if case["epilogue"] == "silu_mul" else n
    per_row = k + 4 + (4 if case["zeros"] else 0)
    per_col = k + 4 + (4 if case["bias"] else 0)
    if op == "gemm_i8":
        M = case["M"]
        return {"bytes": M * per_row + n * per_col + M * cols * esz, "flops": 2 * M * n * k}
    T, E, top_k = case["T"], case["E"], case["top_k"]
    pairs = T * top_k
    # experts that a token reaches: E (1 - (1 - top_k / E)^T) of them on average
    experts = max(1.0, E * (1.0 - (1.0 - min(1.0, top_k / E)) ** T))
    rows = pairs if case["a_per_pair"] else T
    return {"bytes": int(rows * per_row + experts * n * per_col + pairs * cols * esz + pairs * 4),
            "flops": 2 * pairs * n * k}


# ------------------------------------------------------------------ the definition in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "route":
        return _route_exact(s, case)
    if op == "quantize_zp":
        return _quantize_exact(s, case)
    if op == "gemm_i8":
        rows = torch.arange(case["M"], device="cuda")
        return _rows_exact(s, case, rows, rows, 0)
    top_k = case["top_k"]
    cols = case["n"] // 2 if case["epilogue"] == "silu_mul" else case["n"]
    out = torch.empty((case["T"] * top_k, cols), dtype=torch.float64, device="cuda")
    for e in range(case["E"]):
        pairs = (s["expert_ids"] == e).nonzero().reshape(-1)
        if pairs.numel():
            out[pairs] = _rows_exact(s, case, pairs, pairs if case["a_per_pair"] else pairs // top_k, e)
    return out


def _rows_exact(s, case, out_rows, a_rows, e):
    """Integer sums over K in pieces (each exact in 64 bits), then the scales."""
    n, k = case["n"], case["k"]
    total = torch.zeros((out_rows.numel(), n), dtype=torch.int64, device="cuda")
    sums = torch.zeros(n, dtype=torch.int64, device="cuda")
    for k0 in range(0, k, 4096):
        k1 = min(k, k0 + 4096)
        a, b = s["A"][a_rows, k0:k1].double(), s["B"][e, :, k0:k1]
        total += torch.matmul(b.double(), a.t().contiguous()).t().to(torch.int64)
        sums += b.sum(dim=1, dtype=torch.int64)
    if s["a_zeros"] is not None:
        total -= s["a_zeros"][a_rows].long()[:, None] * sums[None, :]
    if case["otype"] == "i32":
        return total.to(torch.int32)
    y = total.double() * (s["a_scales"][a_rows].double()[:, None] * s["b_scales"][e].double()[None, :])
    if s["bias"] is not None:
        y += s["bias"][e].double()
    if case["epilogue"] == "silu_mul":
        gate, up = y.split(n // 2, dim=1)
        y = gate * up / (1.0 + torch.exp(-gate))
    return y


def _route_exact(s, case):
    import numpy as np
    x = s["logits"].double().cpu().numpy()
    T, E, G, top_k = case["T"], case["E"], case["groups"], case["top_k"]
    if case["score"] == "sigmoid":
        score = 1.0 / (1.0 + np.exp(-x))
    else:
        score = np.exp(x - x.max(axis=1, keepdims=True))
        score /= score.sum(axis=1, keepdims=True)
    biased = s["bias"] is not None
    key = score + s["bias"].double().cpu().numpy() if biased else x
    allowed = np.ones((T, E), dtype=bool)
    if G > 1:
        ordered = np.sort((key if biased else score).reshape(T, G, E // G), axis=2)
        value = ordered[:, :, -2:].sum(axis=2) if case["group_score"] == "top2" else ordered[:, :, -1]
        best = np.argsort(-value, axis=1, kind="stable")[:, :case["topk_groups"]]
        in_group = np.zeros((T, G), dtype=bool)
        np.put_along_axis(in_group, best, True, axis=1)
        allowed = np.repeat(in_group, E // G, axis=1)
    ids = np.argsort(np.where(allowed, -key, np.inf), axis=1, kind="stable")[:, :top_k]
    w = np.take_along_axis(score, ids, axis=1)
    if case["renorm"]:
        w = w / w.sum(axis=1, keepdims=True)
    return ids.astype(np.int32), w * case["scale"]


def _quantize_exact(s, case):
    import numpy as np
    x = s["x"][:, :case["k"]].float().cpu().numpy().astype(np.float64)
    codes = np.empty(x.shape, dtype=np.int8)
    lo, hi = np.minimum(x.min(axis=1), 0.0), np.maximum(x.max(axis=1), 0.0)
    scale = np.maximum(((hi - lo) / 255.0).astype(np.float32), np.float32(2.0 ** -126))
    scale[hi == lo] = 1.0
    inv = 1.0 / scale.astype(np.float64)
    zero = np.clip(np.rint(-128.0 - lo * inv), -128, 127)
    zero[hi == lo] = 0.0
    for r in range(x.shape[0]):
        codes[r] = np.clip(np.rint(x[r] * inv[r]) + zero[r], -128, 127).astype(np.int8)
    return codes, scale.astype(np.float64), zero.astype(np.int32)
