"""Measured cases of what surrounds a quantized projection in a served layer.

  norm    a block's output joins the residual stream (norm behind the block,
          gate, residual scale), the stream is normed for the next block and
          leaves as bf16 rows and / or as codes of the quantized products
  gated   act(gate) * up of a gate+up projection, as bf16 rows and / or codes
  lora    Y += scale * (X A^T) B^T with each row's own low-rank adapter,
          beside the product that all rows share

``run`` computes a case in its plain form (elementary torch operations) or,
where ``own`` is true, through the library's entry points. ``exact`` is the
definition in 64 bits, written apart from the plain form.

Norms and activations are defined to round once to binary32 and from there to
bf16; codes follow from the bf16 values by the rules of the activation
quantizers. All of these are whole decisions, so the plain forms take them in
64 bits: a value next to a border goes one way only.
"""

import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZES = {"bf16": 2, "f32": 4}


def listed():
    return [
        # one decoded token between two blocks: the codes for the products, the rows for the adapters beside them
        _norm("norm 1 x 4096 int8", 1, 4096, "rms", False, "bf16", "bf16", "none", True, "int8"),
        # a ragged batch of a model with norms on both sides of a block and a gate for each token
        _norm("norm 333 x 7168 both sides fp8", 333, 7168, "rms", True, "f32", "f32", "rows", False, "fp8"),
        # a prefill chunk, asymmetric codes beside the rows
        _norm("norm 4096 x 4096 int8 zp", 4096, 4096, "rms", False, "bf16", "bf16", "none", True, "int8_zp"),
        # a long prefill of a wide model: layer norm, channel gate, residual stream in binary32, 4-bit codes
        _norm("norm 8192 x 8192 layer mxfp4", 8192, 8192, "layer", False, "bf16", "f32", "channels", False, "mxfp4"),
        # rows of an odd length, nothing quantized
        _norm("norm 77 x 1001", 77, 1001, "layer", True, "bf16", "bf16", "channels", True, "none"),
        # a decode batch before the down projection
        _gated("gated 16 x 14336 int8", 16, 14336, "silu", "bf16", False, "int8"),
        # a prefill chunk before the down projection
        _gated("gated 4096 x 14336 fp8", 4096, 14336, "silu", "bf16", False, "fp8"),
        # one decoded token with its adapter, a square projection
        _lora("lora 1 token", 1, 4096, 4096, 1, 16, 8, False, "bf16"),
        # a decode batch of many adapters beside a stacked q, k and v projection (4096 + 1024 + 1024 columns)
        _lora("lora 64 tokens q k v", 64, 6144, 4096, 3, 16, 48, False, "bf16"),
        # a ragged batch, odd sizes, adapters of different ranks, binary32 rows
        _lora("lora 250 tokens odd", 250, 4100, 4090, 1, 64, 12, True, "f32"),
        # a prefill of several requests beside a stacked gate+up projection
        _lora("lora 4096 tokens gate up", 4096, 28672, 4096, 2, 16, 8, False, "bf16"),
        # a prefill of several requests beside the down projection, large ranks
        _lora("lora 2048 tokens down", 2048, 4096, 14336, 1, 64, 12, True, "bf16"),
    ]


def _norm(name, M, n, kind, post, xtype, rtype, gate, rows, quant):
    return {"name": name, "op": "norm", "M": M, "n": n, "kind": kind, "post": post, "xtype": xtype, "rtype": rtype,
            "gate": gate, "rows": rows, "quant": quant}


def _gated(name, M, n, act, ytype, rows, quant):
    return {"name": name, "op": "gated", "M": M, "n": n, "act": act, "ytype": ytype, "rows": rows, "quant": quant}


def _lora(name, M, n, k, slices, rank, adapters, mixed, otype):
    return {"name": name, "op": "lora", "M": M, "n": n, "k": k, "slices": slices, "rank": rank, "adapters": adapters,
            "mixed": mixed, "otype": otype}


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["norm", "norm", "gated", "lora", "lora"])
    if op == "lora":
        M, k = _log_int(rng, 1, 4096), _log_int(rng, 64, 14336)
        n = min(_log_int(rng, 64, 28672), max(64, (2048 * 28672) // M))
        slices = rng.randint(1, 3)
        case = _lora("", M, n, k, slices, rng.choice([4, 8, 16, 16, 24, 32, 64]), _log_int(rng, 1, 24 // slices),
                     rng.random() < 0.5, rng.choice(["bf16", "bf16", "f32"]))
    else:
        quant = rng.choice(["none", "int8", "int8_zp", "fp8", "mxfp4"])
        n = _log_int(rng, 64, 8192 if op == "norm" else 14336)
        unit = {"fp8": 128, "mxfp4": 32}.get(quant, 1)
        n = max(unit, n // unit * unit)
        rows = quant == "none" or rng.random() < 0.5
        M = min(_log_int(rng, 1, 8192), (4096 * 8192) // n)
        if op == "norm":
            case = _norm("", M, n, rng.choice(["rms", "rms", "layer"]), rng.random() < 0.4, rng.choice(["bf16", "f32"]),
                         rng.choice(["bf16", "f32"]), rng.choice(["none", "none", "channels", "rows"]), rows, quant)
        else:
            case = _gated("", M, n, rng.choice(["silu", "silu", "gelu"]), rng.choice(["bf16", "f32"]), rows, quant)
    del case["name"]
    return case


# ------------------------------------------------------------------ inputs

EPS, OFFSET, RESIDUAL_SCALE = 1e-5, 0.0, 0.875


def _round_up(x, m):
    return (x + m - 1) // m * m


def _slice_ends(case):
    """One slice; gate and up; or q and two smaller ones (4 : 1 : 1)."""
    n, s = case["n"], case["slices"]
    return [n] if s == 1 else [n // 2, n] if s == 2 else [n - 2 * (n // 6), n - n // 6, n]


def _codes_buffer(case):
    """Codes as the products read them: rows of whole 16-byte pieces."""
    n, quant = case["n"], case["quant"]
    return _round_up(n // 2 if quant == "mxfp4" else n, 16)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def normal(*shape, dtype=torch.float32, spread=1.0):
        return (spread * torch.randn(shape, generator=gen, device="cuda")).to(dtype)

    s = {"case": case}
    M, n, op = case["M"], case["n"], case["op"]
    if op == "norm":
        # outputs of a block are small beside the stream they join; a few channels of the stream are large
        s["x"] = normal(M, n, dtype=TYPES[case["xtype"]], spread=0.5)
        stream = normal(M, n)
        stream[:, ::97] *= 8.0
        s["residual"] = stream.to(TYPES[case["rtype"]])
        del stream
        s["weight"] = (1.0 + normal(n, spread=0.2)).to(torch.bfloat16)
        s["bias"] = normal(n, dtype=torch.bfloat16, spread=0.1) if case["kind"] == "layer" else None
        s["post_weight"] = (1.0 + normal(n, spread=0.2)).to(torch.bfloat16) if case["post"] else None
        s["gate"] = {"none": None, "channels": normal(1, n, dtype=torch.bfloat16),
                     "rows": normal(M, n, dtype=torch.bfloat16)}[case["gate"]] if case["gate"] != "none" else None
    elif op == "gated":
        s["y"] = normal(M, 2 * n, dtype=TYPES[case["ytype"]], spread=1.5)
    else:
        k, S, R, E = case["k"], case["slices"], case["rank"], case["adapters"]
        s["x"] = normal(M, k, dtype=torch.bfloat16)
        s["A"] = normal(E, S, R, k, dtype=torch.bfloat16, spread=1.0 / math.sqrt(k))
        s["B"] = normal(E, n, R, dtype=torch.bfloat16, spread=0.3)
        s["scales"] = torch.rand(E, generator=gen, device="cuda") + 0.5
        s["ranks"] = torch.randint(1, R + 1, (E,), generator=gen, device="cuda", dtype=torch.int32) if case["mixed"] else None
        s["Y"] = normal(M, n, dtype=TYPES[case["otype"]])
        s["ends"] = _slice_ends(case)
        # tokens of one request follow each other: runs of ids; a run in eight has no adapter
        runs = max(1, min(M, 2 * E))
        ids = torch.randint(0, E, (runs,), generator=gen, device="cuda", dtype=torch.int32)
        ids[7::8] = -1
        s["ids"] = ids[torch.arange(M, device="cuda") * runs // M].contiguous()
    if own:
        _prepare_own(case, s)
    return s


def _prepare_own(case, s):
    """Output buffers, configs, and the grouping of a step's rows by adapter,
    which serves every projection of every layer in that step."""
    import quantized_dequant_gemm_amd as q
    M, n, op = case["M"], case["n"], case["op"]
    types = {"bf16": q.QDG_O_BF16, "f32": q.QDG_O_F32}
    if op == "lora":
        E, rows_each = case["adapters"], M / case["adapters"]
        s["block_m"] = 16 if rows_each <= 32 else 64
        capacity = q.qdg_moe_align_capacity(M, 1, E, s["block_m"])
        s["sorted_ids"] = torch.empty(capacity, dtype=torch.int32, device="cuda")
        s["block_adapter"] = torch.empty(capacity // s["block_m"], dtype=torch.int32, device="cuda")
        s["num_padded"] = torch.empty(1, dtype=torch.int32, device="cuda")
        q.qdg_moe_align(s["ids"].data_ptr(), M, 1, E, s["block_m"], s["sorted_ids"].data_ptr(),
                        s["block_adapter"].data_ptr(), s["num_padded"].data_ptr(), q.current_stream())
        s["cfg"] = q.lora(n, case["k"], case["rank"], num_adapters=E, slice_ends=s["ends"], otype=types[case["otype"]])
        s["ws_bytes"] = q.qdg_lora_workspace(s["cfg"], M, s["block_m"])
        s["ws"] = torch.empty(max(16, s["ws_bytes"]), dtype=torch.uint8, device="cuda")
        return
    quant = case["quant"]
    code = {"none": q.QDG_Q_NONE, "int8": q.QDG_Q_INT8, "int8_zp": q.QDG_Q_INT8_ZP, "fp8": q.QDG_Q_FP8E4M3,
            "mxfp4": q.QDG_Q_MXFP4}[quant]
    s["out"] = torch.empty((M, n), dtype=torch.bfloat16, device="cuda") if case["rows"] else None
    s["qa"] = s["a_scales"] = s["a_zeros"] = None
    ldq = _codes_buffer(case)
    if quant != "none":
        s["qa"] = torch.empty((M, ldq), dtype=torch.uint8, device="cuda")
        shape = {"fp8": (M, n // 128), "mxfp4": (M, n // 32)}.get(quant, (M,))
        s["a_scales"] = torch.empty(shape, dtype=torch.uint8 if quant == "mxfp4" else torch.float32, device="cuda")
        s["a_zeros"] = torch.empty(M, dtype=torch.int32, device="cuda") if quant == "int8_zp" else None
    if op == "gated":
        s["cfg"] = q.gated_act(n, ytype=types[case["ytype"]], quant=code, ldq=ldq,
                               act=q.QDG_ACT_SILU if case["act"] == "silu" else q.QDG_ACT_GELU_TANH)
    else:
        s["new_residual"] = torch.empty((M, n), dtype=TYPES[case["rtype"]], device="cuda")
        s["cfg"] = q.norm(n, kind=q.QDG_NORM_RMS if case["kind"] == "rms" else q.QDG_NORM_LAYER,
                          xtype=types[case["xtype"]], rtype=types[case["rtype"]], wtype=q.QDG_O_BF16,
                          post_norm=int(case["post"]), quant=code, ldq=ldq, ldg=n if case["gate"] == "rows" else 0,
                          eps=EPS, residual_scale=RESIDUAL_SCALE, weight_offset=OFFSET)


# ------------------------------------------------------------------ one pass

def _ptr(t):
    return None if t is None else t.data_ptr()


def run(s):
    if own:
        return _run_own(s)
    return {"norm": _norm_plain, "gated": _gated_plain, "lora": _lora_plain}[s["case"]["op"]](s)


def _run_own(s):
    import quantized_dequant_gemm_amd as q
    case, stream = s["case"], q.current_stream()
    M, op = case["M"], case["op"]
    if op == "lora":
        q.qdg_lora(s["cfg"], s["x"].data_ptr(), s["A"].data_ptr(), s["B"].data_ptr(), _ptr(s["ranks"]),
                   s["scales"].data_ptr(), s["sorted_ids"].data_ptr(), s["block_adapter"].data_ptr(),
                   s["num_padded"].data_ptr(), M, s["block_m"], s["Y"].data_ptr(), s["ws"].data_ptr(), s["ws_bytes"],
                   stream)
        return s["Y"]
    if op == "gated":
        q.qdg_gated_act(s["cfg"], s["y"].data_ptr(), M, _ptr(s["out"]), _ptr(s["qa"]), _ptr(s["a_scales"]),
                        _ptr(s["a_zeros"]), stream)
        return _rows(case, s["out"], s["qa"], s["a_scales"], s["a_zeros"])
    q.qdg_norm(s["cfg"], s["x"].data_ptr(), s["residual"].data_ptr(), _ptr(s["gate"]), _ptr(s["post_weight"]), None,
               s["weight"].data_ptr(), _ptr(s["bias"]), M, s["new_residual"].data_ptr(), _ptr(s["out"]),
               _ptr(s["qa"]), _ptr(s["a_scales"]), _ptr(s["a_zeros"]), stream)
    return {"residual": s["new_residual"], **_rows(case, s["out"], s["qa"], s["a_scales"], s["a_zeros"])}


def _rows(case, out, qa, a_scales, a_zeros):
    """What leaves: int8 codes and fp8 codes as their values, two 4-bit codes
    as the byte that holds them (equal bytes are equal values)."""
    got = {"out": out, "a_scales": a_scales, "a_zeros": a_zeros}
    n, quant = case["n"], case["quant"]
    if quant != "none":
        got["codes"] = qa[:, :n // 2] if quant == "mxfp4" else qa[:, :n].view(
            torch.float8_e4m3fn if quant == "fp8" else torch.int8)
    return {key: t for key, t in got.items() if t is not None}


def _to(y, dtype):
    """Rounded to binary32, then to the type."""
    return y.float().to(dtype)


def _norm_rows(v, kind, weight, bias):
    if kind == "layer":
        v = v - v.mean(dim=1, keepdim=True)
    v = v / torch.sqrt((v * v).mean(dim=1, keepdim=True) + float(torch.tensor(EPS)))
    v = v * (weight.double() + OFFSET)
    return v if bias is None else v + bias.double()


def _norm_plain(s):
    case = s["case"]
    t = s["x"].double()
    if case["post"]:
        t = _norm_rows(t, case["kind"], s["post_weight"], None)
    if s["gate"] is not None:
        t = t * s["gate"].double()
    t = _to(t + RESIDUAL_SCALE * s["residual"].double(), TYPES[case["rtype"]])
    out = _to(_norm_rows(t.double(), case["kind"], s["weight"], s["bias"]), torch.bfloat16)
    return {"residual": t, **_quantize_plain(case, out)}


def _gated_plain(s):
    case = s["case"]
    g, u = s["y"][:, :case["n"]].double(), s["y"][:, case["n"]:].double()
    if case["act"] == "silu":
        g = g / (1.0 + torch.exp(-g))
    else:
        # 0.5 (1 + tanh z) = 1 / (1 + exp(-2 z)), which keeps its digits where tanh z is near -1
        g = g / (1.0 + torch.exp(-2.0 * math.sqrt(2.0 / math.pi) * (g + 0.044715 * g * g * g)))
    return _quantize_plain(case, _to(g * u, torch.bfloat16))


def _quantize_plain(case, out):
    M, n, quant = case["M"], case["n"], case["quant"]
    x = out.float()
    got = {"out": out if case["rows"] else None}
    if quant == "int8" or quant == "fp8":
        most = 127.0 if quant == "int8" else 448.0
        x = x.view(M, -1, n if quant == "int8" else 128)
        amax = x.abs().amax(dim=2, keepdim=True)
        inv = torch.where(amax > 0, (most / amax.double()).float(), torch.zeros_like(amax))
        code = (x * inv).clamp(-most, most)
        code = torch.round(code).to(torch.int8) if quant == "int8" else code.to(torch.float8_e4m3fn)
        scale = torch.where(amax > 0, (amax.double() / most).float(), torch.ones_like(amax))
        got |= {"codes": code.view(M, n), "a_scales": scale.view(M) if quant == "int8" else scale.view(M, n // 128)}
    elif quant == "int8_zp":
        x = x.double()
        lo, hi = x.amin(dim=1).clamp(max=0.0), x.amax(dim=1).clamp(min=0.0)
        scale = ((hi - lo) / 255.0).float().clamp(min=2.0 ** -126)
        scale = torch.where(hi > lo, scale, torch.ones_like(scale))
        inv = 1.0 / scale.double()
        zero = torch.where(hi > lo, torch.round(-128.0 - lo * inv).clamp(-128.0, 127.0), torch.zeros_like(lo))
        codes = (torch.round(x * inv[:, None]) + zero[:, None]).clamp(-128.0, 127.0)
        got |= {"codes": codes.to(torch.int8), "a_scales": scale, "a_zeros": zero.to(torch.int32)}
    elif quant == "mxfp4":
        x = x.view(M, n // 32, 32)
        amax = x.abs().amax(dim=2, keepdim=True)
        e = (torch.frexp(amax).exponent - 3).clamp(min=-127)  # floor(log2(amax)) - 2
        v = torch.ldexp(x.abs().double(), -e)
        code = ((v > 0.25).int() + (v >= 0.75).int() + (v > 1.25).int() + (v >= 1.75).int() + (v > 2.5).int()
                + (v >= 3.5).int() + (v > 5.0).int() + 8 * torch.signbit(x).int())
        code = torch.where(amax > 0, code, torch.zeros_like(code)).to(torch.uint8).view(M, n // 2, 2)
        scale = torch.where(amax > 0, e + 127, torch.zeros_like(e)).to(torch.uint8)
        got |= {"codes": code[:, :, 0] | code[:, :, 1] << 4, "a_scales": scale.view(M, n // 32)}
    return {key: t for key, t in got.items() if t is not None}


def _lora_plain(s):
    """Every row meets every adapter; what is not its own is taken out between the two products."""
    case = s["case"]
    M, n, S, R, E = case["M"], case["n"], case["slices"], case["rank"], case["adapters"]
    t = (s["x"].float() @ s["A"].float().view(E * S * R, -1).t()).view(M, E, S, R)
    mine = (s["ids"][:, None] == torch.arange(E, device="cuda"))[:, :, None, None]
    if s["ranks"] is not None:
        mine = mine & (torch.arange(R, device="cuda") < s["ranks"][:, None])[None, :, None, :]
    t = torch.where(mine, t * s["scales"][None, :, None, None], 0.0)
    ends = torch.tensor(s["ends"], device="cuda")
    of = torch.searchsorted(ends, torch.arange(n, device="cuda"), right=True)
    b = s["B"].float().transpose(1, 2)[:, None] * (of == torch.arange(S, device="cuda")[:, None])[None, :, None, :]
    y = s["Y"].float() + t.view(M, E * S * R) @ b.reshape(E * S * R, n)
    s["Y"].copy_(y)
    return s["Y"]


# ------------------------------------------------------------------ what a pass cannot do without

def _row_bytes(case):
    n, quant = case["n"], case["quant"]
    out = 2 * n if case["rows"] else 0
    return out + {"none": 0, "int8": n + 4, "int8_zp": n + 8, "fp8": n + n // 32, "mxfp4": n // 2 + n // 32}[quant]


def work(case):
    M, n, op = case["M"], case["n"], case["op"]
    if op == "norm":
        row = n * (SIZES[case["xtype"]] + 2 * SIZES[case["rtype"]] + (2 if case["gate"] == "rows" else 0))
        return {"bytes": M * (row + _row_bytes(case)) + 4 * n, "flops": M * n * (16 if case["post"] else 10)}
    if op == "gated":
        return {"bytes": M * (2 * n * SIZES[case["ytype"]] + _row_bytes(case)), "flops": M * n * 10}
    k, S, R, E = case["k"], case["slices"], case["rank"], case["adapters"]
    runs = max(1, min(M, 2 * E))
    rows = M * (runs - runs // 8) / runs  # those with an adapter
    met = E * (1.0 - (1.0 - 1.0 / E) ** (runs - runs // 8))
    mean_rank = (R + 1) / 2 if case["mixed"] else R
    return {"bytes": int(rows * (2 * k + 2 * n * SIZES[case["otype"]]) + met * mean_rank * 2 * (S * k + n)),
            "flops": int(2 * rows * mean_rank * (S * k + n))}


# ------------------------------------------------------------------ the definition in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "lora":
        return _lora_exact(s, case)
    if case["op"] == "gated":
        gate, up = s["y"].double().split(case["n"], dim=1)
        if case["act"] == "silu":
            y = up * gate * torch.sigmoid(gate)
        else:
            y = up * gate * torch.sigmoid(2.0 * math.sqrt(2.0 / math.pi) * gate * (1.0 + 0.044715 * gate.square()))
        return _quantize_exact(case, y)
    t = s["x"].double()
    if case["post"]:
        t = _norm_exact(t, case["kind"], s["post_weight"], None)
    if s["gate"] is not None:
        t.mul_(s["gate"])
    t.add_(s["residual"], alpha=RESIDUAL_SCALE)
    stream = t.to(torch.float32).to(TYPES[case["rtype"]]).double()
    return {"residual": stream, **_quantize_exact(case, _norm_exact(stream, case["kind"], s["weight"], s["bias"]))}


def _norm_exact(v, kind, weight, bias):
    eps = float(torch.tensor(EPS, dtype=torch.float32))
    n = v.shape[1]
    mean = v.sum(dim=1, keepdim=True) / n if kind == "layer" else 0.0
    centred = v - mean
    length = torch.linalg.vector_norm(centred, dim=1, keepdim=True)
    y = centred * torch.rsqrt(length.square() / n + eps) * (OFFSET + weight.double())
    return y if bias is None else y.add_(bias)


def _quantize_exact(case, y):
    """Codes and scales from the bf16 values, products and quotients of binary32 numbers rounded from 64 bits."""
    M, n, quant = case["M"], case["n"], case["quant"]
    x = y.to(torch.float32).to(torch.bfloat16).double()
    got = {"out": x} if case["rows"] else {}
    f32 = lambda v: v.to(torch.float32).double()  # noqa: E731
    if quant in ("int8", "fp8"):
        top, group = (127.0, n) if quant == "int8" else (448.0, 128)
        x = x.reshape(M, n // group, group)
        amax = x.abs().max(dim=2).values
        some = amax > 0
        one = torch.ones_like(amax)
        v = f32(x * torch.where(some, f32(top / torch.where(some, amax, one)), 0.0 * one)[:, :, None]).clamp_(-top, top)
        if quant == "int8":
            codes = v.round_().reshape(M, n).to(torch.int8)
        else:
            step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3.0)
            codes = ((v / step).round_() * step).reshape(M, n)
        scales = torch.where(some, f32(amax / top), one)
        got |= {"codes": codes, "a_scales": scales.reshape(M) if quant == "int8" else scales}
    elif quant == "int8_zp":
        zero_in = torch.cat([x, torch.zeros((M, 1), dtype=x.dtype, device=x.device)], dim=1)
        lo, hi = zero_in.min(dim=1).values, zero_in.max(dim=1).values
        some = hi > lo
        scale = torch.where(some, f32((hi - lo) / 255.0).clamp(min=2.0 ** -126), torch.ones_like(lo))
        zero = torch.where(some, (-128.0 - lo * (1.0 / scale)).round().clamp(-128, 127), torch.zeros_like(lo))
        codes = ((x * (1.0 / scale)[:, None]).round_() + zero[:, None]).clamp_(-128, 127)
        got |= {"codes": codes.to(torch.int8), "a_scales": scale, "a_zeros": zero.to(torch.int32)}
    elif quant == "mxfp4":
        x = x.reshape(M, n // 32, 32)
        amax = x.abs().max(dim=2).values
        e = torch.floor(torch.log2(amax.clamp(min=2.0 ** -127))).clamp(min=-125.0) - 2.0
        v = (x.abs() * torch.exp2(-e)[:, :, None]).clamp_(max=6.0)
        # steps of 1/2 below 2, 1 below 4, 2 below 6; an even number of steps is an even code
        step = torch.where(v < 2.0, 0.5, torch.where(v < 4.0, 1.0, 2.0))
        v = (v / step).round_() * step
        code = torch.where(v <= 2.0, 2.0 * v, torch.where(v <= 4.0, v + 2.0, v / 2.0 + 4.0)).to(torch.int32)
        code = torch.where(amax[:, :, None] > 0, code + 8 * torch.signbit(x).to(torch.int32), 0).reshape(M, n // 2, 2)
        got |= {"codes": (code[..., 0] + 16 * code[..., 1]).to(torch.uint8),
                "a_scales": torch.where(amax > 0, e + 127.0, torch.zeros_like(e)).to(torch.uint8)}
    return got


def _lora_exact(s, case):
    y = s["Y"].double()
    ends, R = [0] + s["ends"], case["rank"]
    for a in range(case["adapters"]):
        rows = (s["ids"] == a).nonzero().reshape(-1)
        if not rows.numel():
            continue
        r = R if s["ranks"] is None else int(s["ranks"][a])
        x = s["x"][rows].double()
        for i in range(case["slices"]):
            down = x @ s["A"][a, i, :r].double().t()
            y[rows, ends[i]:ends[i + 1]] += float(s["scales"][a]) * (down @ s["B"][a, ends[i]:ends[i + 1], :r].double().t())
    return y
