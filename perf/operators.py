"""The operators around the experts, measured: routing from router logits (``gate``) and the dense product with its
epilogue (``linear``; with a second weight matrix, a gated product).

``run`` computes a case in its plain form, elementary torch operations in 32 bits (routing scores in 64, where two
experts may lie next to each other), or, where ``own`` is true, by the library's entry points.

gate    s = sigmoid(logit) or softmax(logits); chosen by s + bias among the experts of the best groups (a group's
        score: its largest s + bias, or the sum of its two largest), ties to the lower index; weights: the chosen
        experts' s, divided by their sum where they are renormalised, times a scale.  An expert whose logit or bias is
        -inf takes no part; a row with fewer experts than it may choose has id -1 and weight 0 in the places left.
linear  out = act(x W^T + bias) + residual, or act(x W^T + bias, x U^T + bias_up) + residual for a gated act.
"""
import math

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
_GATED = ("situ_glu", "swiglu")
_ACTS = ("none", "relu", "silu", "gelu", "gelu_tanh")
_B1, _B2 = 4.0, 25.0  # SiTU's two bounds


# ---------------------------------------------------------------------------------------------------------- the cases

def _gate(name, T, E, k, score, bias, groups=1, top_groups=1, group_score="max", renorm=True, scale=1.0, type="f32",
          masked=0.0, pad=0):
    c = dict(op="gate", T=T, E=E, k=k, score=score, bias=bias, groups=groups, top_groups=top_groups,
             group_score=group_score, renorm=renorm, scale=scale, type=type, masked=masked, pad=pad)
    return dict(c, name=name) if name else c


def _linear(name, T, K, N, act="none", bias=False, residual="none", type="bf16", out="half", pad=0):
    c = dict(op="linear", T=T, K=K, N=N, act=act, bias=bias, residual=residual, type=type, out=out, pad=pad)
    return dict(c, name=name) if name else c


def listed():
    return [
        # one token of a served sequence: 16 of 896 experts by biased sigmoid scores, where the latency counts
        _gate("gate-1x896", 1, 896, 16, "sigmoid", True),
        # a served batch with softmax scores kept as they are, logits from a bf16 product: equal logits do occur
        _gate("gate-64x128-softmax", 64, 128, 8, "softmax", False, renorm=False, type="bf16"),
        # a ragged batch, logits inside wider rows, six groups of ten, experts switched off and padding rows without any
        _gate("gate-1000x60-groups", 1000, 60, 4, "softmax", True, groups=6, top_groups=3, type="f16", masked=0.1, pad=4),
        # a prompt's tokens with experts spread over eight devices: the best half of the groups by their two best experts
        _gate("gate-4096x256-groups", 4096, 256, 8, "sigmoid", True, groups=8, top_groups=4, group_score="top2", scale=2.5),
        # several prompts at once over the largest router
        _gate("gate-16384x896", 16384, 896, 16, "sigmoid", True),
        # one token through a projection whose output is added to the stream
        _linear("linear-1x7168x3584", 1, 7168, 3584, bias=True, residual="same"),
        # a served batch through a gated product
        _linear("glu-24x3584x6144", 24, 3584, 6144, act="swiglu", type="f16"),
        # sizes no tile divides, rows that no wide load reaches, an activation
        _linear("linear-333x1117x2049", 333, 1117, 2049, act="gelu", bias=True, residual="f32", type="f16", pad=6),
        # several hundred tokens of a chunked prompt: between the served batch and the whole prompt
        _linear("linear-200x3584x7168", 200, 3584, 7168, bias=True, act="silu"),
        # a prompt's router logits, kept in 32 bits
        _linear("logits-4096x7168x896", 4096, 7168, 896, out="f32"),
        # a prompt through a gated product
        _linear("glu-4096x3584x6144", 4096, 3584, 6144, act="situ_glu", bias=True),
        # a prompt through a wide projection whose output is added to the stream: the most work of all
        _linear("linear-4096x7168x7168", 4096, 7168, 7168, bias=True, residual="same"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    if rng.random() < 0.45:
        groups = rng.choice([1, 1, 1, 2, 4, 6, 8])
        E = groups * max(1, _log(rng, 8, 896) // groups)
        T = _log(rng, 1, 16384)
        top_groups = rng.randint(1, groups)
        k = min(_log(rng, 1, 32), E // groups * top_groups)
        return _gate(None, T, E, k, rng.choice(["sigmoid", "softmax"]), rng.random() < 0.6, groups, top_groups,
                     rng.choice(["max", "top2"]), rng.random() < 0.7, rng.choice([1.0, 2.5]),
                     rng.choice(["f32", "f32", "bf16", "f16"]), rng.choice([0.0, 0.0, 0.1]), rng.choice([0, 0, 3]))
    step = rng.choice([1, 8, 32, 64])
    K, N = step * max(1, _log(rng, 64, 7168) // step), step * max(1, _log(rng, 32, 7168) // step)
    act = rng.choice(_ACTS + _GATED)
    T = _log(rng, 1, 4096)
    if act in _GATED:
        N = max(1, N // 2)
    return _linear(None, T, K, N, act, rng.random() < 0.5, rng.choice(["none", "same", "f32"]),
                   rng.choice(["bf16", "f16"]), rng.choice(["half", "half", "f32"]), rng.choice([0, 0, 8, 5]))


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape, std=1.0):
        return torch.randn(*shape, device="cuda", generator=g) * std

    s = dict(case=case)
    t = _TYPES[case["type"]]
    if case["op"] == "gate":
        T, E, k = case["T"], case["E"], case["k"]
        # a trained router's logits: a spread of their own for each token, some experts liked by all
        logits = normal(T, E) * (0.5 + torch.rand(T, 1, device="cuda", generator=g) * 2.0) + normal(1, E, std=0.7)
        if case["masked"]:
            logits[:, torch.rand(E, device="cuda", generator=g) < case["masked"]] = -math.inf
            logits[T - T // 8:] = -math.inf  # padding tokens
        wide = torch.empty(T, E + case["pad"], dtype=t, device="cuda")
        wide[:, :E] = logits
        wide[:, E:] = math.nan
        s["logits"] = wide[:, :E]
        # balance biases: small next to the scores
        s["bias"] = normal(E, std=0.05 if case["score"] == "sigmoid" else 0.2 / E) if case["bias"] else None
        if own:
            import quantized_expert_gemv_sigmoid_amd as moe
            s["desc"] = moe.make_gate_desc(
                E, k, score=moe.SCORE_SIGMOID if case["score"] == "sigmoid" else moe.SCORE_SOFTMAX, bias=s["bias"],
                n_groups=case["groups"], top_groups=case["top_groups"],
                group_score=moe.GROUP_MAX if case["group_score"] == "max" else moe.GROUP_TOP2,
                renorm=int(case["renorm"]), routed_scale=case["scale"])
            s["ids"] = torch.empty(T, k, dtype=torch.int32, device="cuda")
            s["weights"] = torch.empty(T, k, device="cuda")
            s["counts"] = torch.empty(E, dtype=torch.int32, device="cuda")
        return s
    T, K, N = case["T"], case["K"], case["N"]
    gated = case["act"] in _GATED
    wide = torch.empty(T, K + case["pad"], dtype=t, device="cuda")
    wide[:, :K] = normal(T, K)
    wide[:, K:] = math.nan
    s["x"] = wide[:, :K]
    s["w"] = normal(N, K, std=K ** -0.5).to(t)
    s["w_up"] = normal(N, K, std=K ** -0.5).to(t) if gated else None
    s["bias"] = normal(N, std=0.3).to(t) if case["bias"] else None
    s["bias_up"] = normal(N, std=0.3).to(t) if case["bias"] and gated else None
    s["residual"] = None if case["residual"] == "none" else normal(T, N).to(t if case["residual"] == "same" else torch.float32)
    if own:
        import quantized_expert_gemv_sigmoid_amd as moe
        s["desc"] = moe.make_linear_desc(s["w"], w_up=s["w_up"], bias=s["bias"], bias_up=s["bias_up"],
                                         act=getattr(moe, "LINEAR_" + case["act"].upper()), situ_b1=_B1, situ_b2=_B2,
                                         residual_type=moe.F32 if case["residual"] == "f32" else None)
        s["ws"] = moe.linear_workspace(s["desc"], T)
        s["out"] = torch.empty(T, N, dtype=torch.float32 if case["out"] == "f32" else t, device="cuda")
    return s


def work(case):
    if case["op"] == "gate":
        T, E, k = case["T"], case["E"], case["k"]
        size = 4 if case["type"] == "f32" else 2
        return {"bytes": T * E * size + T * k * 8 + E * 4 + (E * 4 if case["bias"] else 0), "flops": 10 * T * E}
    T, K, N = case["T"], case["K"], case["N"]
    m = 2 if case["act"] in _GATED else 1
    b = 2 * (T * K + m * N * K) + (2 * m * N if case["bias"] else 0) + T * N * (4 if case["out"] == "f32" else 2)
    b += T * N * {"none": 0, "same": 2, "f32": 4}[case["residual"]]
    return {"bytes": b, "flops": 2 * m * T * N * K}


# ---------------------------------------------------------------------------------------------------------- the calls

def run(s):
    case = s["case"]
    if own:
        import quantized_expert_gemv_sigmoid_amd as moe
        if case["op"] == "gate":
            moe.gate(s["desc"], s["logits"], case["T"], s["ids"], s["weights"], s["counts"])
            return {"ids": s["ids"], "weights": s["weights"], "counts": s["counts"]}
        f32 = case["out"] == "f32"
        moe.linear(s["desc"], s["x"], case["T"], None if f32 else s["out"], s["out"] if f32 else None,
                   moe.OUT_F32 if f32 else moe.OUT_HALF, s["ws"], residual=s["residual"])
        return s["out"]
    return _plain_gate(s, case) if case["op"] == "gate" else _plain_linear(s, case)


def _plain_gate(s, case):
    T, E, k, groups = case["T"], case["E"], case["k"], case["groups"]
    logits = s["logits"].double()
    off = logits == -math.inf
    if case["score"] == "sigmoid":
        score = 1.0 / (1.0 + torch.exp(-logits))
    else:
        top = logits.amax(1, keepdim=True)
        e = torch.where(off, 0.0, torch.exp(logits - torch.where(top == -math.inf, 0.0, top)))
        score = e / e.sum(1, keepdim=True).clamp_min(1e-300)
    by = score if s["bias"] is None else score + s["bias"].double()
    by = torch.where(off, -math.inf, by)
    if groups > 1:
        g = by.view(T, groups, E // groups)
        best = g.sort(dim=2, descending=True)[0][:, :, :2]
        value = best[:, :, 0]
        if case["group_score"] == "top2" and E // groups > 1:
            value = value + torch.where(best[:, :, 1] == -math.inf, 0.0, best[:, :, 1])
        order = value.sort(dim=1, descending=True, stable=True)[1][:, :case["top_groups"]]
        kept = torch.zeros(T, groups, dtype=torch.bool, device=by.device).scatter(1, order, True)
        by = torch.where(kept[:, :, None], g, -math.inf).view(T, E)
    by, order = by.sort(dim=1, descending=True, stable=True)
    by, order = by[:, :k], order[:, :k]
    there = by > -math.inf
    w = torch.where(there, score.gather(1, order), 0.0)
    if case["renorm"]:
        total = w.sum(1, keepdim=True)
        w = w / torch.where(total > 0, total, 1.0)
    ids = torch.where(there, order, -1).int()
    counts = torch.zeros(E + 1, dtype=torch.int32, device=by.device)
    counts.scatter_add_(0, torch.where(there, order, E).view(-1), torch.ones(T * k, dtype=torch.int32, device=by.device))
    return {"ids": ids, "weights": (w * case["scale"]).float(), "counts": counts[:E]}


def _plain_linear(s, case):
    x = s["x"].float()
    a = x @ s["w"].float().t()
    if s["bias"] is not None:
        a = a + s["bias"].float()
    act = case["act"]
    if act in _GATED:
        u = x @ s["w_up"].float().t()
        if s["bias_up"] is not None:
            u = u + s["bias_up"].float()
        sig = 1.0 / (1.0 + torch.exp(-a))
        a = a * sig * u if act == "swiglu" else _B1 * torch.tanh(a / _B1) * sig * (_B2 * torch.tanh(u / _B2))
    elif act == "relu":
        a = torch.where(a > 0, a, 0.0)
    elif act == "silu":
        a = a / (1.0 + torch.exp(-a))
    elif act == "gelu":
        a = 0.5 * a * (1.0 + torch.erf(a * math.sqrt(0.5)))
    elif act == "gelu_tanh":
        a = 0.5 * a * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (a + 0.044715 * a * a * a)))
    if s["residual"] is not None:
        a = a + s["residual"].float()
    return a if case["out"] == "f32" else a.to(_TYPES[case["type"]])


# ------------------------------------------------------------------------------------------------------ in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return _exact_gate(s, case) if case["op"] == "gate" else _exact_linear(s, case)


def _first_max(v):
    """The largest value of each row and the lowest index that has it."""
    m = v.amax(1, keepdim=True)
    at = torch.arange(v.shape[1], device=v.device)
    return m, torch.where(v == m, at, v.shape[1]).amin(1, keepdim=True)


def _exact_gate(s, case):
    T, E, k, groups = case["T"], case["E"], case["k"], case["groups"]
    size = E // groups
    z = s["logits"].double()
    on = z > -math.inf
    if case["score"] == "sigmoid":
        p = 0.5 + 0.5 * torch.tanh(0.5 * z)
    else:
        p = torch.where(on.any(1, keepdim=True), torch.exp(z - torch.logsumexp(z, 1, keepdim=True)), 0.0)
    pick = torch.where(on, p + (0.0 if s["bias"] is None else s["bias"].double()), -math.inf)
    if groups > 1:
        value = torch.empty(T, groups, dtype=torch.float64, device=z.device)
        for j in range(groups):
            part = pick[:, j * size:(j + 1) * size].clone()
            m, at = _first_max(part)
            if case["group_score"] == "top2" and size > 1:
                m2 = part.scatter(1, at, -math.inf).amax(1, keepdim=True)
                m = m + torch.where(m2 == -math.inf, 0.0, m2)
            value[:, j] = m[:, 0]
        kept = torch.zeros(T, groups, dtype=torch.bool, device=z.device)
        for _ in range(case["top_groups"]):
            _, at = _first_max(torch.where(kept, -math.inf, value))
            # (groups without an expert left are all -inf: which of them is kept makes no difference)
            kept = kept.scatter(1, at, True)
        pick = torch.where(kept.repeat_interleave(size, 1), pick, -math.inf)
    w = torch.zeros(T, k, dtype=torch.float64, device=z.device)
    for j in range(k):
        m, at = _first_max(pick)
        w[:, j:j + 1] = torch.where(m > -math.inf, p.gather(1, at), 0.0)
        pick = pick.scatter(1, at, -math.inf)
    if case["renorm"]:
        total = w.sum(1, keepdim=True)
        w = torch.where(total > 0, w / total, w)
    return {"ids": None, "weights": w * case["scale"], "counts": None}


def _exact_linear(s, case):
    def product(w, b):
        v = s["x"].double() @ w.double().t()
        return v if b is None else v + b.double()

    v, act = product(s["w"], s["bias"]), case["act"]
    sig = torch.sigmoid(v)
    if act == "swiglu":
        v = v * sig * product(s["w_up"], s["bias_up"])
    elif act == "situ_glu":
        u = product(s["w_up"], s["bias_up"])
        v = _B1 * _B2 * torch.tanh(v / _B1) * torch.tanh(u / _B2) * sig
    elif act == "relu":
        v = v.clamp_min(0.0)
    elif act == "silu":
        v = v * sig
    elif act == "gelu":
        v = 0.5 * v * torch.erfc(-v * math.sqrt(0.5))
    elif act == "gelu_tanh":
        v = v * torch.sigmoid(2.0 * math.sqrt(2.0 / math.pi) * (v + 0.044715 * v ** 3))
    return v if s["residual"] is None else v + s["residual"].double()
