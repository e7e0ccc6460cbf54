"""Products in microscaled 4-bit floating point and of ragged groups, measured: MXFP4 quantisation (``quant``), the MXFP4
product (``mx``), products grouped by expert (``grouped``), and those as experts of an FFN behind a routing (``experts``).

``run`` computes a case in its plain form, elementary torch operations in 32 bits, or, where ``own`` is true, by the
library's entry points.

quant    blocks of 32 along a row share a scale 2^e, e = floor(log2(largest magnitude)) - 2 ("floor"), or one more where
         the largest magnitude is past 6 * 2^e ("fit"), at least -127; the values divided by it become E2M1 numbers
         (0, 0.5, 1, 1.5, 2, 3, 4, 6), round to nearest, ties to the even code, magnitudes past 6 become 6.  What comes
         back is the numbers times their scales, in the input's type.
mx       out = act(x W^T + bias) + residual, or act(x W^T + bias, x U^T + bias_up) + residual, of MXFP4 rows x, W, U.
grouped  out[r] = act(x[rows[r]] W_g^T + bias_g (, x[rows[r]] U_g^T)) for the rows r of group g, offsets[g] <= r <
         offsets[g + 1]; rows from offsets[G] on stay as they are.  16-bit operands or MXFP4 ones.
experts  the choices of each token (ids, weights) sorted by expert, h = act of the grouped products with W, U, y of the
         one with D, out[t] = residual[t] + sum_j weights[t][j] y[place of choice (t, j)]; an id of -1 is no choice.
"""
import math

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
_GATED = ("situ_glu", "swiglu")
_ACTS = ("none", "relu", "silu", "gelu", "gelu_tanh")
_B1, _B2 = 4.0, 25.0  # SiTU's two bounds
_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ---------------------------------------------------------------------------------------------------------- the cases

def _named(name, c):
    return dict(c, name=name) if name else c


def _quant(name, T, K, type="bf16", rule="floor", pad=0):
    return _named(name, dict(op="quant", T=T, K=K, type=type, rule=rule, pad=pad))


def _mx(name, T, K, N, act="none", bias=False, residual="none", type="bf16", out="half"):
    return _named(name, dict(op="mx", T=T, K=K, N=N, act=act, bias=bias, residual=residual, type=type, out=out))


def _grouped(name, T, k, E, K, N, act="none", bias=False, type="bf16", mx=False, gather=True, out="half", pad=0, masked=0.0):
    return _named(name, dict(op="grouped", T=T, k=k, E=E, K=K, N=N, act=act, bias=bias, type=type, mx=mx, gather=gather,
                             out=out, pad=pad, masked=masked))


def _experts(name, T, k, E, K, F, act="swiglu", residual="none", type="bf16", masked=0.0):
    return _named(name, dict(op="experts", T=T, k=k, E=E, K=K, F=F, act=act, residual=residual, type=type, masked=masked))


def listed():
    return [
        # one token's activations before a 4-bit product, where the latency counts
        _quant("quant-1x7168", 1, 7168),
        # ragged rows inside wider ones, a last block that is not full, scales that fit
        _quant("quant-777x1117", 777, 1117, type="f16", rule="fit", pad=6),
        # a set of experts' 16-bit weights made into the 4-bit ones that the layer reads
        _quant("quant-28672x3584", 28672, 3584, rule="fit"),
        # one token through a 4-bit projection whose output is added to the stream
        _mx("mx-1x7168x3584", 1, 7168, 3584, bias=True, residual="same"),
        # a chunk of a prompt, sizes no tile divides, scale rows of 35 bytes, an activation
        _mx("mx-200x1120x2049", 200, 1120, 2049, act="gelu", bias=True, residual="f32", type="f16"),
        # a prompt through a wide 4-bit projection whose output is added to the stream
        _mx("mx-4096x7168x7168", 4096, 7168, 7168, bias=True, residual="same"),
        # one token's gate and up products: eight of 128 experts, each read for one row
        _grouped("grouped-1-of-128", 1, 8, 128, 3584, 2048, act="swiglu"),
        # a served batch's down products: a few rows for each expert
        _grouped("grouped-64-of-64", 64, 8, 64, 2048, 3584, type="f16", gather=False, out="f32"),
        # few experts with ragged sizes, rows that no wide load reaches, choices that are dropped
        _grouped("grouped-333-of-7", 333, 3, 7, 1117, 515, act="gelu", bias=True, type="f16", pad=5, masked=0.2),
        # a prompt's gate and up products with 4-bit experts and activations
        _grouped("grouped-mx-2048-of-64", 2048, 8, 64, 3584, 2048, act="situ_glu", mx=True),
        # one token through sixteen of 896 small experts: every launch counts
        _experts("experts-1-of-896", 1, 16, 896, 1024, 512),
        # a prompt through 16-bit experts, added to the stream, some padding tokens: the most work of all
        _experts("experts-4096-of-64", 4096, 8, 64, 2048, 1408, residual="same", masked=0.05),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _steps(rng, step, lo, hi):
    return step * max(1, _log(rng, lo, hi) // step)


def draw(rng):
    op = rng.choice(["quant", "mx", "mx", "grouped", "grouped", "grouped", "experts"])
    if op == "quant":
        K = _log(rng, 1, 7168)
        T = _log(rng, 1, min(65536, 28672 * 3584 // K))
        return _quant(None, T, K, rng.choice(["bf16", "f16", "f32"]), rng.choice(["floor", "fit"]), rng.choice([0, 0, 3, 8]))
    if op == "mx":
        act = rng.choice(_ACTS + _GATED)
        K, N, T = _steps(rng, rng.choice([32, 128]), 32, 7168), _log(rng, 16, 7168), _log(rng, 1, 4096)
        if act in _GATED:
            N = max(1, N // 2)
        return _mx(None, T, K, N, act, rng.random() < 0.5, rng.choice(["none", "same", "f32"]), rng.choice(["bf16", "f16"]),
                   rng.choice(["half", "half", "f32"]))
    E = _log(rng, 1, 256)
    k, T = rng.randint(1, min(E, 8)), _log(rng, 1, 2048)
    if op == "grouped":
        mx = rng.random() < 0.35
        act = rng.choice(_ACTS + _GATED)
        K = _steps(rng, 128 if mx else rng.choice([1, 8, 64]), 64, 3584)
        N = _log(rng, 16, min(3584, (1 << 30) // (E * K)))
        if act in _GATED:
            N = max(1, N // 2)
        return _grouped(None, T, k, E, K, N, act, rng.random() < 0.4, rng.choice(["bf16", "f16"]), mx, rng.random() < 0.6,
                        rng.choice(["half", "half", "f32"]), 0 if mx else rng.choice([0, 0, 8, 5]), rng.choice([0.0, 0.0, 0.2]))
    K = _steps(rng, rng.choice([1, 8, 64]), 64, 2048)
    F = _steps(rng, rng.choice([1, 8, 64]), 32, min(1408, (1 << 29) // (E * K)))
    return _experts(None, T, k, E, K, F, rng.choice(_GATED), rng.choice(["none", "same", "f32"]), rng.choice(["bf16", "f16"]),
                    rng.choice([0.0, 0.1]))


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape, std=1.0, dtype=torch.float32):
        return torch.randn(*shape, device="cuda", generator=g, dtype=dtype) * std

    def rows(T, K, pad, dtype, values):
        wide = torch.full((T, K + pad), math.nan, dtype=dtype, device="cuda")
        wide[:, :K] = values
        return wide[:, :K]

    def packed(v):
        """MXFP4 codes and scales of rows v, ties to the even code, scales that fit."""
        flat = v.reshape(-1, v.shape[-1])
        codes = torch.empty(flat.shape[0], flat.shape[1] // 2, dtype=torch.uint8, device="cuda")
        scales = torch.empty(flat.shape[0], flat.shape[1] // 32, dtype=torch.uint8, device="cuda")
        step = max(1, (1 << 26) // flat.shape[1])
        for a in range(0, flat.shape[0], step):
            n, e = _blocks(flat[a:a + step].float(), "fit")
            q = n.abs()
            c = torch.where(q < 2, q * 2, torch.where(q < 4, q + 2, q * 0.5 + 4)).to(torch.uint8)
            c = (c | (torch.signbit(n).to(torch.uint8) << 3)).view(c.shape[0], -1)
            codes[a:a + step] = c[:, 0::2] | (c[:, 1::2] << 4)
            scales[a:a + step] = (e[:, :, 0] + 127).to(torch.uint8)
        return codes.view(*v.shape[:-1], -1), scales.view(*v.shape[:-1], -1)

    op, t = case["op"], _TYPES[case["type"]]
    s = dict(case=case)
    T, K = case["T"], case["K"]
    # activations: tokens of different sizes, some channels larger than the rest
    size = 0.5 + torch.rand(T, 1, device="cuda", generator=g)
    channel = torch.where(torch.rand(1, K, device="cuda", generator=g) < 0.01, 8.0, 1.0)
    x = normal(T, K) * size * channel
    if op == "quant":
        s["x"] = rows(T, K, case["pad"], t, x)
        if own:
            import quantized_expert_gemv_sigmoid_amd as moe
            blocks = (K + 31) // 32
            s["codes"] = torch.empty(T, 16 * blocks, dtype=torch.uint8, device="cuda")
            s["scales"] = torch.empty(T, blocks, dtype=torch.uint8, device="cuda")
            s["rule"] = moe.MX_FLOOR if case["rule"] == "floor" else moe.MX_FIT
            s["out"] = torch.empty(T, K, dtype=t, device="cuda")
        return s
    gated = case["act"] in _GATED
    if op == "mx":
        N = case["N"]
        s["x"], s["x_s"] = packed(x)
        s["w"], s["w_s"] = packed(normal(N, K, std=K ** -0.5))
        s["w_up"], s["w_up_s"] = packed(normal(N, K, std=K ** -0.5)) if gated else (None, None)
        s["bias"] = normal(N, std=0.3).to(t) if case["bias"] else None
        s["bias_up"] = normal(N, std=0.3).to(t) if case["bias"] and gated else None
        s["residual"] = None if case["residual"] == "none" else normal(T, N).to(t if case["residual"] == "same" else torch.float32)
        if own:
            import quantized_expert_gemv_sigmoid_amd as moe
            s["desc"] = moe.make_mx_linear_desc(
                s["w"], s["w_s"], w_up=s["w_up"], w_up_s=s["w_up_s"], bias=s["bias"], bias_up=s["bias_up"],
                type=moe.F16 if case["type"] == "f16" else moe.BF16, act=getattr(moe, "LINEAR_" + case["act"].upper()),
                situ_b1=_B1, situ_b2=_B2, residual_type=moe.F32 if case["residual"] == "f32" else None)
            s["ws"] = moe.mx_linear_workspace(s["desc"], T)
            s["out"] = torch.empty(T, N, dtype=torch.float32 if case["out"] == "f32" else t, device="cuda")
        return s
    # a routing with experts liked by all; tokens of padding choose none
    E, k = case["E"], case["k"]
    liked = normal(T, E) + normal(1, E, std=0.7)
    top = liked.topk(k, dim=1)
    ids = top.indices.int()
    if case["masked"]:
        ids[torch.rand(T, device="cuda", generator=g) < case["masked"]] = -1
    R = T * k
    if op == "grouped":
        N = case["N"]
        flat = torch.where(ids < 0, E, ids).view(-1).long()
        order = torch.argsort(flat, stable=True)
        counts = torch.bincount(flat, minlength=E + 1)[:E]
        s["offsets"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).int()
        s["rows"] = torch.div(order, k, rounding_mode="floor").int() if case["gather"] else None
        if not case["gather"]:  # every row of its own
            x = normal(R, K) * (0.5 + torch.rand(R, 1, device="cuda", generator=g))
        for n in ("w", "w_up") if gated else ("w",):
            w = normal(E, N, K, dtype=t).mul_(K ** -0.5)
            s[n], s[n + "_s"] = packed(w) if case["mx"] else (w, None)
        s["x"], s["x_s"] = packed(x) if case["mx"] else (rows(x.shape[0], K, case["pad"], t, x), None)
        s["bias"] = normal(E, N, std=0.3).to(t) if case["bias"] else None
        s["bias_up"] = normal(E, N, std=0.3).to(t) if case["bias"] and gated else None
        s["out"] = torch.zeros(R, N, dtype=torch.float32 if case["out"] == "f32" else t, device="cuda")
        if own:
            import quantized_expert_gemv_sigmoid_amd as moe
            s["desc"] = moe.make_grouped_desc(
                s["w"], w_up=s.get("w_up"), w_s=s["w_s"], w_up_s=s.get("w_up_s"), bias=s["bias"], bias_up=s["bias_up"],
                type=moe.F16 if case["type"] == "f16" else moe.BF16, act=getattr(moe, "LINEAR_" + case["act"].upper()),
                situ_b1=_B1, situ_b2=_B2)
        return s
    F = case["F"]
    s["ids"] = ids
    s["weights"] = torch.softmax(top.values, 1).contiguous()
    s["x"] = x.to(t)
    s["w"], s["w_up"] = normal(E, F, K, dtype=t).mul_(K ** -0.5), normal(E, F, K, dtype=t).mul_(K ** -0.5)
    s["down"] = normal(E, K, F, dtype=t).mul_(F ** -0.5)
    s["residual"] = None if case["residual"] == "none" else normal(T, K).to(t if case["residual"] == "same" else torch.float32)
    if own:
        import quantized_expert_gemv_sigmoid_amd as moe
        s["up_desc"] = moe.make_grouped_desc(s["w"], w_up=s["w_up"], act=getattr(moe, "LINEAR_" + case["act"].upper()),
                                             situ_b1=_B1, situ_b2=_B2)
        s["down_desc"] = moe.make_grouped_desc(s["down"])
        s["ws"] = moe.group_workspace(T, k, E)
        s["offsets"] = torch.empty(E + 1, dtype=torch.int32, device="cuda")
        s["tokens"] = torch.empty(R, dtype=torch.int32, device="cuda")
        s["places"] = torch.empty(T, k, dtype=torch.int32, device="cuda")
        s["h"] = torch.empty(R, F, dtype=t, device="cuda")
        s["y"] = torch.empty(R, K, device="cuda")  # 32 bits until the rows of a token are added up
        s["out"] = torch.empty(T, K, dtype=t, device="cuda")
    return s


def _active(case):
    """Expected number of groups that get a row, and of rows."""
    E, R = case["E"], case["T"] * case["k"] * (1.0 - case["masked"])
    return E * (1.0 - (1.0 - case["k"] / E) ** (case["T"] * (1.0 - case["masked"]))) if E > case["k"] else E, R


def work(case):
    T, K = case["T"], case["K"]
    if case["op"] == "quant":
        size = 4 if case["type"] == "f32" else 2
        return {"bytes": T * K * 2 * size + T * ((K + 31) // 32) * 17, "flops": 4 * T * K}
    m = 2 if case["act"] in _GATED else 1
    if case["op"] == "mx":
        N = case["N"]
        b = (T + m * N) * K * 17 // 32 + (2 * m * N if case["bias"] else 0) + T * N * (4 if case["out"] == "f32" else 2)
        return {"bytes": b + T * N * {"none": 0, "same": 2, "f32": 4}[case["residual"]], "flops": 2 * m * T * N * K}
    active, R = _active(case)
    if case["op"] == "grouped":
        N, row = case["N"], K * (17 / 32 if case["mx"] else 2)
        b = ((T if case["gather"] else R) + active * m * N) * row + R * N * (4 if case["out"] == "f32" else 2)
        return {"bytes": int(b + (2 * m * active * N if case["bias"] else 0)), "flops": int(2 * m * R * N * K)}
    F = case["F"]
    b = 3 * active * F * K * 2 + T * K * (4 + {"none": 0, "same": 2, "f32": 4}[case["residual"]]) + T * case["k"] * 8
    return {"bytes": int(b), "flops": int(6 * R * F * K)}


# ---------------------------------------------------------------------------------------------------------- the calls

def run(s):
    case = s["case"]
    if own:
        return _own(s, case)
    return {"quant": _plain_quant, "mx": _plain_mx, "grouped": _plain_grouped, "experts": _plain_experts}[case["op"]](s, case)


def _own(s, case):
    import quantized_expert_gemv_sigmoid_amd as moe
    T, f32 = case["T"], case.get("out") == "f32"
    if case["op"] == "quant":
        moe.mx_quantize(s["x"], T, s["codes"], s["scales"], rule=s["rule"])
        moe.mx_dequantize(s["codes"], s["scales"], T, s["out"])
        return s["out"]
    half, full, mode = (None, s["out"], moe.OUT_F32) if f32 else (s["out"], None, moe.OUT_HALF)
    if case["op"] == "mx":
        moe.mx_linear(s["desc"], s["x"], s["x_s"], T, half, full, mode, s["ws"], residual=s["residual"])
        return s["out"]
    R = T * case["k"]
    if case["op"] == "grouped":
        moe.grouped_linear(s["desc"], s["x"], s["offsets"], R, half, full, mode, rows=s["rows"], x_s=s["x_s"])
        return s["out"]
    moe.group(s["ids"], T, case["E"], s["offsets"], s["tokens"], s["places"], s["ws"])
    moe.grouped_linear(s["up_desc"], s["x"], s["offsets"], R, s["h"], None, moe.OUT_HALF, rows=s["tokens"])
    moe.grouped_linear(s["down_desc"], s["h"], s["offsets"], R, None, s["y"], moe.OUT_F32)
    moe.combine(s["y"], R, s["places"], s["weights"], T, s["out"], residual=s["residual"])
    return {"out": s["out"], "offsets": s["offsets"], "places": s["places"]}


def _scaled(x, e):
    """x 2^e, the powers made from their bits (pow may be off by a bit), in two steps that hold any exponent."""
    h = e.int() >> 1
    return x * ((h + 127) << 23).view(torch.float32) * ((e.int() - h + 127) << 23).view(torch.float32)


def _blocks(x, rule):
    """E2M1 numbers of rows x [T][K] in blocks [T][K / 32][32], and the exponents of their scales."""
    b = x.reshape(x.shape[0], -1, 32)
    top = b.abs().amax(2, keepdim=True)
    m, e = torch.frexp(top)  # top = m 2^e, m in [0.5, 1)
    e = e - 3
    if rule == "fit":
        e = e + (m > 0.75).int()
    e = torch.where(top > 0, e, -127).clamp_min(-127)
    v = _scaled(b, -e)
    a = v.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    return torch.copysign((torch.round(a / step) * step).clamp_max(6.0), v), e


def _plain_quant(s, case):
    T, K = case["T"], case["K"]
    x = torch.zeros(T, (K + 31) // 32 * 32, device=s["x"].device)
    x[:, :K] = s["x"].float()
    n, e = _blocks(x, case["rule"])
    return _scaled(n, e).view(T, -1)[:, :K].to(_TYPES[case["type"]])


def _values(codes, scales):
    """The fp32 values of MXFP4 rows."""
    table = torch.tensor(_E2M1 + tuple(-v for v in _E2M1), device=codes.device)
    n = table[torch.stack([codes & 15, codes >> 4], -1).long()].view(*scales.shape, 32)
    return _scaled(n, scales[..., None].int() - 127).view(*codes.shape[:-1], -1)


def _act(act, a, u):
    if act in _GATED:
        sig = 1.0 / (1.0 + torch.exp(-a))
        return a * sig * u if act == "swiglu" else _B1 * torch.tanh(a / _B1) * sig * (_B2 * torch.tanh(u / _B2))
    if act == "relu":
        return torch.where(a > 0, a, 0.0)
    if act == "silu":
        return a / (1.0 + torch.exp(-a))
    if act == "gelu":
        return 0.5 * a * (1.0 + torch.erf(a * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * a * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (a + 0.044715 * a * a * a)))
    return a


def _product(x, w, bias):
    a = x @ w.t()
    return a if bias is None else a + bias.float()


def _plain_mx(s, case):
    x = _values(s["x"], s["x_s"])
    a = _product(x, _values(s["w"], s["w_s"]), s["bias"])
    u = _product(x, _values(s["w_up"], s["w_up_s"]), s["bias_up"]) if case["act"] in _GATED else None
    a = _act(case["act"], a, u)
    if s["residual"] is not None:
        a = a + s["residual"].float()
    return a if case["out"] == "f32" else a.to(_TYPES[case["type"]])


def _plain_grouped(s, case):
    out, gated = s["out"], case["act"] in _GATED
    x = _values(s["x"], s["x_s"]) if case["mx"] else s["x"].float()
    if s["rows"] is not None:
        x = x[s["rows"].long()]

    def weights(n, e):
        return _values(s[n][e], s[n + "_s"][e]) if case["mx"] else s[n][e].float()

    ends = s["offsets"].tolist()
    for e in range(case["E"]):
        a, b = ends[e], ends[e + 1]
        if a == b:
            continue
        v = _product(x[a:b], weights("w", e), None if s["bias"] is None else s["bias"][e])
        u = _product(x[a:b], weights("w_up", e), None if s["bias_up"] is None else s["bias_up"][e]) if gated else None
        out[a:b] = _act(case["act"], v, u).to(out.dtype)
    return out


def _sorted(ids, E):
    """Offsets of the experts' choices, sorted by expert, their order, and the place of each choice (-1: no choice)."""
    flat = torch.where(ids < 0, E, ids).view(-1).long()
    by, order = torch.sort(flat, stable=True)
    offsets = torch.searchsorted(by, torch.arange(E + 1, device=ids.device)).int()
    places = torch.empty_like(flat).scatter_(0, order, torch.arange(flat.numel(), device=ids.device))
    return offsets, order, torch.where(flat < E, places, -1).int().view(ids.shape)


def _plain_experts(s, case):
    T, k, E = case["T"], case["k"], case["E"]
    offsets, order, places = _sorted(s["ids"], E)
    x, w = s["x"].float(), s["weights"].view(-1)
    out = torch.zeros(T, case["K"], device=x.device) if s["residual"] is None else s["residual"].float()
    ends = offsets.tolist()
    for e in range(E):
        if ends[e] == ends[e + 1]:
            continue
        at = order[ends[e]:ends[e + 1]]
        token = torch.div(at, k, rounding_mode="floor")
        xe = x[token]
        h = _act(case["act"], xe @ s["w"][e].float().t(), xe @ s["w_up"][e].float().t())
        # (a token chooses an expert once: no index twice)
        out[token] += w[at, None] * (h @ s["down"][e].float().t())
    return {"out": out.to(_TYPES[case["type"]]), "offsets": offsets, "places": places}


# ------------------------------------------------------------------------------------------------------ in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"quant": _exact_quant, "mx": _exact_mx, "grouped": _exact_grouped, "experts": _exact_experts}[case["op"]](s, case)


def _exact_quant(s, case):
    T, K = case["T"], case["K"]
    blocks = (K + 31) // 32
    step = max(1, (1 << 24) // K)
    parts = []
    for a in range(0, T, step):
        x = s["x"][a:a + step].double()
        b = torch.nn.functional.pad(x, (0, blocks * 32 - K)).view(-1, blocks, 32)
        top = b.abs().max(2).values
        # the power of two at or below the largest magnitude: that over its fraction in [1, 2)
        fraction = 2 * torch.frexp(top).mantissa
        power = torch.where(top > 0, top / torch.where(top > 0, fraction, 1.0), 0.0)
        scale = power / 4
        if case["rule"] == "fit":
            scale = torch.where(top > 6 * scale, 2 * scale, scale)
        scale = scale.clamp_min(2.0 ** -127)[:, :, None]
        v = b.abs() / scale
        # halfway points between neighbours go to the even code: the upper one where it is the even one
        q = torch.zeros_like(v)
        for mid, up, even in ((0.25, 0.5, False), (0.75, 1.0, True), (1.25, 1.5, False), (1.75, 2.0, True), (2.5, 3.0, False),
                              (3.5, 4.0, True), (5.0, 6.0, False)):
            q = torch.where(v >= mid if even else v > mid, up, q)
        parts.append((torch.where(b < 0, -q, q) * scale).view(-1, blocks * 32)[:, :K])
    return torch.cat(parts)


def _values64(codes, scales):
    high = codes.long() >> 4
    c = torch.stack([codes.long() - 16 * high, high], -1).view(*codes.shape[:-1], -1)
    e, m, neg = (c >> 1) & 3, (c & 1).double(), c > 7
    v = torch.where(e == 0, m / 2, (1 + m / 2) * torch.exp2((e - 1).double()))
    v = torch.where(neg, -v, v)
    power = ((scales.long() + (1023 - 127)) << 52).view(torch.float64)
    return v * power.repeat_interleave(32, dim=-1)


def _act64(act, a, u):
    sig = torch.sigmoid(a)
    if act == "swiglu":
        return a * sig * u
    if act == "situ_glu":
        return _B1 * _B2 * torch.tanh(a / _B1) * torch.tanh(u / _B2) * sig
    if act == "relu":
        return a.clamp_min(0.0)
    if act == "silu":
        return a * sig
    if act == "gelu":
        return 0.5 * a * torch.erfc(-a * math.sqrt(0.5))
    if act == "gelu_tanh":
        return a * torch.sigmoid(2.0 * math.sqrt(2.0 / math.pi) * (a + 0.044715 * a ** 3))
    return a


def _sum64(x, w, bias):
    v = x @ w.transpose(0, 1)
    return v if bias is None else v + bias.double()


def _exact_mx(s, case):
    x = _values64(s["x"], s["x_s"])
    a = _sum64(x, _values64(s["w"], s["w_s"]), s["bias"])
    u = _sum64(x, _values64(s["w_up"], s["w_up_s"]), s["bias_up"]) if case["act"] in _GATED else None
    v = _act64(case["act"], a, u)
    return v if s["residual"] is None else v + s["residual"].double()


def _exact_grouped(s, case):
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    group = torch.bucketize(torch.arange(out.shape[0], device="cuda"), s["offsets"][1:].contiguous(), right=True)
    for e in range(case["E"]):
        at = torch.nonzero(group == e)[:, 0]
        if not at.numel():
            continue
        src = at if s["rows"] is None else s["rows"][at].long()
        x = _values64(s["x"][src], s["x_s"][src]) if case["mx"] else s["x"][src].double()
        r = []
        for n, b in (("w", "bias"), ("w_up", "bias_up")) if case["act"] in _GATED else (("w", "bias"),):
            w = _values64(s[n][e], s[n + "_s"][e]) if case["mx"] else s[n][e].double()
            r.append(_sum64(x, w, None if s[b] is None else s[b][e]))
        out[at] = _act64(case["act"], r[0], r[-1])
    return out


def _exact_experts(s, case):
    x = s["x"].double()
    out = torch.zeros(x.shape, dtype=torch.float64, device="cuda") if s["residual"] is None else s["residual"].double()
    for e in range(case["E"]):
        chosen = s["ids"] == e
        at = torch.nonzero(chosen.any(1))[:, 0]
        if not at.numel():
            continue
        weight = torch.where(chosen, s["weights"].double(), 0.0).sum(1)[at, None]
        h = _act64(case["act"], _sum64(x[at], s["w"][e].double(), None), _sum64(x[at], s["w_up"][e].double(), None))
        out[at] = out[at] + weight * _sum64(h, s["down"][e].double(), None)
    return {"out": out, "offsets": None, "places": None}
