"""moe_grouped_linear, moe_group and moe_combine on the GPU against their formulas in 64 bits.

Bounds as in test_gpu_linear.py and test_gpu_mx_linear.py; whole numbers have to be equal.  What no row or group covers
has to keep its sentinels.
"""
import pytest

import quantized_expert_gemv_sigmoid_amd as moe
from mx_support import pack, unpack
from test_gpu_linear import B1, B2, GATED, HALF, PLAIN
from test_gpu_mx_linear import close, finish, product

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def sizes_of(E, R, kind, g):
    """How many rows each group gets."""
    if kind == "one":            # all in one group
        c = [0] * E
        c[E // 2] = R
        return c
    if kind == "even":
        return [R // E + (e < R % E) for e in range(E)]
    if kind == "short":          # rows that are in no group, at both ends
        return [max(0, R // E - 1)] * E
    w = torch.rand(E, generator=g) ** 3 * (torch.rand(E, generator=g) < 0.6) + 1e-9   # ragged, many empty
    cuts = torch.sort(torch.multinomial(w, R, replacement=True, generator=g))[0]
    return torch.bincount(cuts, minlength=E).tolist()


def make(E, R, K, N, type=torch.bfloat16, act="none", bias=None, gather=0, kind="ragged", mx=False, whole=False, padx=0, padw=0,
         seed=0):
    """gather: rows of x (0: row r is x's own).  Matrices and rows apart by padw, rows of x by padx, NaN between them."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    gc = torch.Generator().manual_seed(seed)

    def values(*shape, std=1.0):
        if whole:
            return torch.randint(-3, 4, shape, device="cuda", generator=g).float()
        return torch.randn(*shape, device="cuda", generator=g) * std

    def apart(t, pad):
        if not pad:
            return t.contiguous()
        wide = torch.full((*t.shape[:-1], t.shape[-1] + pad), float("nan"), device="cuda", dtype=t.dtype)
        wide[..., :t.shape[-1]] = t
        return wide[..., :t.shape[-1]]

    X = gather or R
    s = dict(E=E, R=R, K=K, N=N, type=type, act=act, mx=mx, rows=None, bias=None, bias_up=None, w_up=None, w_s=None, w_up_s=None,
             x_s=None, x_rows=X)
    c = sizes_of(E, R, kind, gc)
    first = 1 if kind == "short" and R > sum(c) else 0
    s["offsets"] = torch.tensor([first + sum(c[:e]) for e in range(E + 1)], dtype=torch.int32, device="cuda")
    x = values(X, K)
    names = ("w", "w_up") if act in GATED else ("w",)
    if mx:
        s["x"], s["x_s"] = pack(x, "fit")
        for n in names:
            s[n], s[n + "_s"] = pack(values(E, N, K, std=K ** -0.5), "fit")
    else:
        s["x"] = apart(x.to(type), padx)
        for n in names:
            s[n] = apart(values(E, N, K, std=K ** -0.5).to(type), padw)
    if gather:
        s["rows"] = torch.randint(0, X, (R,), device="cuda", generator=g, dtype=torch.int32)
    if bias is not None:
        s["bias"] = values(E, N, std=0.5).to(bias)
        s["bias_up"] = values(E, N, std=0.5).to(bias) if act in GATED else None
    return s


def descriptor(s):
    return moe.make_grouped_desc(s["w"], w_up=s["w_up"], bias=s["bias"], bias_up=s["bias_up"], w_s=s["w_s"], w_up_s=s["w_up_s"],
                                 act=getattr(moe, "LINEAR_" + s["act"].upper()), situ_b1=B1, situ_b2=B2,
                                 type=moe.F16 if s["type"] == torch.float16 else moe.BF16)


def call(s, mode=moe.OUT_BOTH, pad=0, stream=None):
    R, N = s["R"], s["N"]
    h = torch.full((R + 2, N + pad), 99.0, device="cuda").to(s["type"])
    f = torch.full((R + 2, N + pad), 99.0, device="cuda")
    moe.grouped_linear(descriptor(s), s["x"], s["offsets"], R, h[:, :N], f[:, :N], mode, rows=s["rows"], x_s=s["x_s"], stream=stream)
    torch.cuda.synchronize()
    a, b = covered(s)
    for o, written in ((h, mode != moe.OUT_F32), (f, mode != moe.OUT_HALF)):
        assert (o[:a] == 99.0).all() and (o[b:] == 99.0).all() and (o[:, N:] == 99.0).all()
        if not written:
            assert (o == 99.0).all()
    return h[:R, :N], f[:R, :N]


def covered(s):
    o = s["offsets"].tolist()
    return max(0, o[0]), max(0, min(o[-1], s["R"]))


def reference(s):
    """(values, bound) of the rows that groups cover."""
    x = unpack(s["x"], s["x_s"]) if s["mx"] else s["x"].double()
    if s["rows"] is not None:
        r = s["rows"].long()
        ok = (r >= 0) & (r < s["x_rows"])
        x = torch.where(ok[:, None], x[r.clamp(0, s["x_rows"] - 1)], 0.0)
    o = s["offsets"].tolist()
    v = torch.full((s["R"], s["N"]), 99.0, dtype=torch.float64, device="cuda")
    e = torch.zeros_like(v)

    def weights(n, g):
        return unpack(s[n][g], s[n + "_s"][g]) if s["mx"] else s[n][g].double()

    for g in range(s["E"]):
        a, b = o[g], o[g + 1]
        if a >= b:
            continue
        p, ep = product(x[a:b], weights("w", g), None if s["bias"] is None else s["bias"][g])
        u, eu = (None, None) if s["act"] not in GATED else product(x[a:b], weights("w_up", g),
                                                                   None if s["bias_up"] is None else s["bias_up"][g])
        v[a:b], e[a:b] = finish(s["act"], p, ep, u, eu, None)
    return v, e


def check(s, mode=moe.OUT_BOTH, pad=0):
    h, f = call(s, mode, pad)
    v, e = reference(s)
    a, b = covered(s)
    if mode != moe.OUT_HALF:
        close(f[a:b], v[a:b], e[a:b])
    if mode != moe.OUT_F32:
        close(h[a:b], v[a:b], e[a:b])
    return h, f


SIZES = [(1, 1, 64, 8), (8, 1, 256, 40), (128, 8, 512, 96), (3, 2, 1024, 33), (7, 50, 192, 65), (64, 512, 256, 128),
         (16, 300, 640, 200), (896, 1000, 128, 48), (1000, 64, 64, 16), (5, 700, 320, 515), (2, 1500, 512, 770), (4, 2600, 256, 4096)]


@pytest.mark.parametrize("E,R,K,N", SIZES)
@pytest.mark.parametrize("form", ["bf16", "f16", "mx"])
@pytest.mark.parametrize("gated", [0, 1])
@pytest.mark.parametrize("gather", [0, 1])
def test_sizes(E, R, K, N, form, gated, gather):
    print(f"case: {E} {R}x{K}x{N} {form} gated {gated} gather {gather}", flush=True)
    if form == "mx":
        K = (K + 127) // 128 * 128
    s = make(E, R, K, N // (1 + gated), torch.float16 if form == "f16" else torch.bfloat16, act="swiglu" if gated else "none",
             bias=torch.float32 if R % 2 else None, gather=R // 3 + 1 if gather else 0, mx=form == "mx", seed=E + R)
    check(s, pad=3)


@pytest.mark.parametrize("E,R,K,N", [(1, 1, 1, 1), (3, 5, 7, 9), (7, 999, 1117, 515), (128, 16, 333, 65), (30, 400, 61, 100), (2, 900, 515, 1030)])
@pytest.mark.parametrize("gather", [0, 1])
@pytest.mark.parametrize("gated", [0, 1])
def test_odd_sizes_and_rows_apart(E, R, K, N, gather, gated):
    for pads in ((0, 0), (5, 3), (8, 8)):
        s = make(E, R, K, N, torch.float16, act="situ_glu" if gated else "gelu", bias=torch.float16, gather=R if gather else 0,
                 padx=pads[0], padw=pads[1], seed=R + pads[0])
        check(s)


@pytest.mark.parametrize("kind", ["one", "even", "short"])
@pytest.mark.parametrize("E,R,K,N", [(9, 30, 256, 64), (64, 640, 128, 72), (6, 1400, 128, 520)])
@pytest.mark.parametrize("mx", [0, 1])
def test_groups(kind, E, R, K, N, mx):
    s = make(E, R, K, N, act="silu", kind=kind, mx=bool(mx), seed=E)
    check(s)


@pytest.mark.parametrize("E,R,K,N", SIZES)
@pytest.mark.parametrize("gather", [0, 1])
def test_whole_numbers_are_exact(E, R, K, N, gather):
    s = make(E, R, K, N, bias=torch.float32, whole=True, gather=7 if gather else 0, seed=R)
    h, f = call(s)
    v = reference(s)[0]
    a, b = covered(s)
    assert torch.equal(f[a:b].double(), v[a:b]) and torch.equal(h[a:b], f[a:b].to(s["type"]))


@pytest.mark.parametrize("act", PLAIN + GATED)
@pytest.mark.parametrize("mx", [0, 1])
def test_activations(act, mx):
    for R in (3, 90, 900):
        s = make(4, R, 384, 200, torch.float16, act=act, bias=torch.float16, mx=bool(mx), gather=20, seed=R)
        for mode in (moe.OUT_HALF, moe.OUT_F32):
            check(s, mode)


@pytest.mark.parametrize("form", ["half", "unaligned", "mx"])
@pytest.mark.parametrize("R", [12, 200, 1200])
def test_rows_without_a_source_are_zeros(form, R):
    s = make(3, R, 256 if form != "unaligned" else 203, 150, bias=torch.float32, gather=50, mx=form == "mx", seed=R)
    s["rows"][::5] = -1
    s["rows"][1::7] = 50
    s["rows"][2::9] = 2 ** 31 - 1
    s["rows"][3::11] = -2 ** 31
    check(s)


@pytest.mark.parametrize("R", [40, 1000])
def test_offsets_past_the_rows(R):
    """They count as the rows' end; before the first row, as its start."""
    s = make(4, R, 128, 64, kind="even", seed=1)
    far = s["offsets"].clone()
    far[0], far[-1] = -5, R + 1000
    want = call(s)[1]
    s["offsets"] = far
    h = torch.full((R + 2, 64), 99.0, device="cuda")
    moe.grouped_linear(descriptor(s), s["x"], far, R, None, h, moe.OUT_F32)
    torch.cuda.synchronize()
    assert torch.equal(h[:R], want) and (h[R:] == 99.0).all()
    s["offsets"] = torch.tensor([0, R, 0, R, R], dtype=torch.int32, device="cuda")   # not in order: whatever, inside the rows
    moe.grouped_linear(descriptor(s), s["x"], s["offsets"], R, None, h, moe.OUT_F32)
    torch.cuda.synchronize()
    assert (h[R:] == 99.0).all()


def test_no_rows_and_empty_groups():
    s = make(5, 6, 128, 32, seed=2)
    s["offsets"].zero_()
    h, f = call(s)
    assert (f == 99.0).all() and (h == 99.0).all()
    moe.grouped_linear(descriptor(s), s["x"], s["offsets"], 0, h, None, moe.OUT_HALF)


def test_matrices_apart():
    """Experts' matrices inside larger ones, in another order of dimensions, and one shared by every group."""
    g = torch.Generator(device="cuda").manual_seed(3)
    E, R, K, N = 6, 200, 128, 96
    s = make(E, R, K, N, seed=3)
    both = torch.randn(N, E, 2 * K, device="cuda", generator=g).bfloat16() * 0.1
    s["w"] = both.transpose(0, 1)[:, :, K:]
    check(s)
    s["w"] = both[:, :1, :K].transpose(0, 1).expand(E, N, K)
    check(s)


def test_captured_and_on_another_stream():
    for mx in (False, True):
        s = make(16, 300, 256, 200, gather=64, mx=mx, seed=4)
        d = descriptor(s)
        want = call(s)[0].clone()
        out = torch.full((300, 200), 99.0, dtype=torch.bfloat16, device="cuda")
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        moe.grouped_linear(d, s["x"], s["offsets"], 300, out, None, moe.OUT_HALF, rows=s["rows"], x_s=s["x_s"], stream=side)
        side.synchronize()
        assert torch.equal(out, want)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            moe.grouped_linear(d, s["x"], s["offsets"], 300, out, None, moe.OUT_HALF, rows=s["rows"], x_s=s["x_s"])
        # other groups by the time of the replay
        s["offsets"].copy_(make(16, 300, 256, 200, seed=5)["offsets"])
        want = call(s)[0].clone()
        for _ in range(3):
            out.fill_(99.0)
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, want)


# ------------------------------------------------------------------ the groups themselves

def group_reference(ids, E):
    flat = ids.view(-1).long().cpu()
    k = ids.shape[1]
    flat = torch.where((flat < 0) | (flat >= E), E, flat)
    order = torch.sort(flat, stable=True)[1]
    offsets = torch.cat([torch.zeros(1, dtype=torch.long), torch.bincount(flat, minlength=E + 1)[:E].cumsum(0)])
    n = int(offsets[-1])
    places = torch.full_like(flat, -1)
    places[order[:n]] = torch.arange(n)
    return offsets.int(), (order[:n] // k).int(), places.int().view(ids.shape)


@pytest.mark.parametrize("T,k,E", [(1, 1, 1), (1, 16, 896), (1, 64, 1024), (3, 2, 5), (64, 8, 64), (100, 7, 1000), (1000, 3, 7), (512, 8, 128),
                                   (513, 8, 128), (4096, 8, 64), (4096, 16, 896), (5000, 1, 2), (70000, 4, 1024), (9000, 64, 300)])
@pytest.mark.parametrize("kind", ["distinct", "repeated", "none", "one"])
def test_group(T, k, E, kind):
    print(f"case: {T}x{k} of {E} {kind}", flush=True)
    g = torch.Generator(device="cuda").manual_seed(T + k)
    if kind == "distinct" and k <= E and T * E < 2 ** 24:
        ids = torch.rand(T, E, device="cuda", generator=g).topk(k, dim=1)[1].int()
        ids[torch.rand(T, k, device="cuda", generator=g) < 0.1] = -1
    elif kind == "none":
        ids = torch.full((T, k), -1, dtype=torch.int32, device="cuda")
        ids[::2] = E
    elif kind == "one":
        ids = torch.full((T, k), E - 1, dtype=torch.int32, device="cuda")
    else:
        ids = torch.randint(-2 if E > 3 else 0, E + 2, (T, k), device="cuda", generator=g, dtype=torch.int32)
        ids[0, 0], ids[-1, -1] = -2 ** 31, 2 ** 31 - 1
    offsets = torch.full((E + 2,), 77, dtype=torch.int32, device="cuda")
    tokens = torch.full((T * k + 2,), 77, dtype=torch.int32, device="cuda")
    places = torch.full((T + 1, k), 77, dtype=torch.int32, device="cuda")
    ws = moe.group_workspace(T, k, E).fill_(255)
    moe.group(ids, T, E, offsets, tokens, places, ws)
    torch.cuda.synchronize()
    o, t, p = group_reference(ids, E)
    n = int(o[-1])
    assert torch.equal(offsets.cpu()[:E + 1], o) and offsets[E + 1] == 77
    assert torch.equal(tokens.cpu()[:n], t) and (tokens[n:] == 77).all()
    assert torch.equal(places.cpu()[:T], p) and (places[T:] == 77).all()


def test_group_of_no_tokens():
    ids = torch.zeros(1, 4, dtype=torch.int32, device="cuda")
    offsets = torch.full((9,), 77, dtype=torch.int32, device="cuda")
    t, p = torch.full((4,), 77, dtype=torch.int32, device="cuda"), torch.full((1, 4), 77, dtype=torch.int32, device="cuda")
    moe.group(ids, 0, 8, offsets, t, p, moe.group_workspace(0, 4, 8))
    torch.cuda.synchronize()
    assert (offsets == 0).all() and (t == 77).all() and (p == 77).all()


def test_group_captured():
    T, k, E = 2000, 8, 64
    ids = torch.randint(-1, E, (T, k), dtype=torch.int32, device="cuda")
    offsets, tokens = torch.empty(E + 1, dtype=torch.int32, device="cuda"), torch.empty(T * k, dtype=torch.int32, device="cuda")
    places, ws = torch.empty(T, k, dtype=torch.int32, device="cuda"), moe.group_workspace(T, k, E)
    moe.group(ids, T, E, offsets, tokens, places, ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.group(ids, T, E, offsets, tokens, places, ws)
    for i in range(3):
        ids.copy_(torch.randint(-1, E, (T, k), dtype=torch.int32, device="cuda"))
        offsets.fill_(-7), places.fill_(-7), ws.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        o, t, p = group_reference(ids, E)
        assert torch.equal(offsets.cpu(), o) and torch.equal(tokens.cpu()[:int(o[-1])], t) and torch.equal(places.cpu(), p)


TYPES = (torch.bfloat16, torch.float16, torch.float32)


@pytest.mark.parametrize("T,k,n,R", [(1, 1, 1, 1), (1, 16, 3584, 16), (5, 3, 33, 15), (100, 8, 2048, 800), (333, 4, 1001, 1000), (70000, 2, 8, 64),
                                     (3, 64, 2049, 100)])
@pytest.mark.parametrize("yt", TYPES, ids=str)
@pytest.mark.parametrize("residual", [None, "rows", "one"])
def test_combine(T, k, n, R, yt, residual):
    g = torch.Generator(device="cuda").manual_seed(T + n)
    wide = torch.full((R, n + 3), float("nan"), device="cuda", dtype=yt)
    wide[:, :n] = torch.randn(R, n, device="cuda", generator=g)
    y = wide[:, :n]
    places = torch.randint(-1, R, (T, k), device="cuda", generator=g, dtype=torch.int32)
    places[0, 0] = R if T > 1 else 0
    w = torch.randn(T, k, device="cuda", generator=g)
    for ot, rt, weighted in ((torch.bfloat16, torch.float32, True), (torch.float32, torch.float16, False), (torch.float16, torch.bfloat16, True)):
        res = None
        if residual is not None:
            res = torch.randn(T if residual == "rows" else 1, n, device="cuda", generator=g).to(rt).expand(T, n)
        out = torch.full((T + 1, n + 5), 99.0, device="cuda", dtype=ot)
        moe.combine(y, R, places, w if weighted else None, T, out[:, :n], residual=res)
        torch.cuda.synchronize()
        ok = ((places >= 0) & (places < R)).double()
        ww = (w.double() if weighted else 1.0) * ok
        v = torch.zeros(T, n, dtype=torch.float64, device="cuda")
        m = torch.zeros_like(v)
        for j in range(k):
            term = ww[:, j:j + 1] * y[places[:, j].long().clamp(0, R - 1)].double()
            v, m = v + term, m + term.abs()
        e = (k + 1) * 2.0 ** -23 * m   # k steps of fp32, none worse than the sum of magnitudes' step
        if res is not None:
            v = v + res.double()
            e = e + 2.0 ** -23 * v.abs()
        bound = e + HALF[ot] * (v.abs() + e) + (2.0 ** -25 if ot == torch.float16 else 1e-37)
        assert ((out[:T, :n].double() - v).abs() <= bound).all()
        assert (out[T:] == 99.0).all() and (out[:, n:] == 99.0).all()


def test_combine_in_place_and_dropped_rows_of_nan():
    """A row that no choice names may hold anything; out may be the residual."""
    y = torch.full((10, 64), float("nan"), device="cuda")
    y[:4] = 1.0
    places = torch.tensor([[0, 1], [-1, 3], [-1, -1]], dtype=torch.int32, device="cuda")
    w = torch.tensor([[0.5, 0.25], [float("nan"), 2.0], [float("inf"), 1.0]], device="cuda")
    out = torch.arange(3.0, device="cuda")[:, None].repeat(1, 64)
    moe.combine(y, 10, places, w, 3, out, residual=out)
    assert out[:, 0].tolist() == [0.75, 3.0, 2.0] and (out == out[:, :1]).all()
    moe.combine(y, 0, places, w, 3, out)
    assert (out == 0).all()
    moe.combine(y, 0, places, w, 0, out.fill_(3))
    assert (out == 3).all()


@pytest.mark.parametrize("T,E,k", [(1, 32, 4), (40, 32, 4), (700, 16, 2)])
@pytest.mark.parametrize("type", [torch.bfloat16, torch.float16])
def test_an_ffn_of_16_bit_experts(T, E, k, type):
    """moe_gate, moe_group, the products and moe_combine as they are used together."""
    g = torch.Generator(device="cuda").manual_seed(T)
    d, F = 256, 192
    x = torch.randn(T, d, device="cuda", generator=g).to(type)
    logits = torch.randn(T, E, device="cuda", generator=g) * 2
    logits[T // 2:T // 2 + T // 10] = -float("inf")   # padding: no choice
    w1, w3 = ((torch.randn(E, F, d, device="cuda", generator=g) * d ** -0.5).to(type) for _ in range(2))
    w2 = (torch.randn(E, d, F, device="cuda", generator=g) * F ** -0.5).to(type)
    i32 = torch.int32
    ids, wt = torch.empty(T, k, dtype=i32, device="cuda"), torch.empty(T, k, device="cuda")
    moe.gate(moe.make_gate_desc(E, k, score=moe.SCORE_SOFTMAX), logits, T, ids, wt)
    offsets, tokens, places = (torch.empty(*n, dtype=i32, device="cuda") for n in ((E + 1,), (T * k,), (T, k)))
    moe.group(ids, T, E, offsets, tokens, places, moe.group_workspace(T, k, E))
    h, y = torch.empty(T * k, F, dtype=type, device="cuda"), torch.empty(T * k, d, device="cuda")
    out = torch.empty(T, d, dtype=type, device="cuda")
    moe.grouped_linear(moe.make_grouped_desc(w1, w_up=w3, act=moe.LINEAR_SWIGLU), x, offsets, T * k, h, None, moe.OUT_HALF, rows=tokens)
    moe.grouped_linear(moe.make_grouped_desc(w2), h, offsets, T * k, None, y, moe.OUT_F32)
    moe.combine(y, T * k, places, wt, T, out, residual=x)
    torch.cuda.synchronize()
    v, e = x.double(), torch.zeros(T, d, dtype=torch.float64, device="cuda")
    half = HALF[type]
    for j in range(k):
        for ex in range(E):
            at = (ids[:, j] == ex).nonzero()[:, 0]
            if not at.numel():
                continue
            a, ea = product(x[at].double(), w1[ex].double(), None)
            u, eu = product(x[at].double(), w3[ex].double(), None)
            hv, eh = finish("swiglu", a, ea, u, eu, None)
            eh = eh + half * (hv.abs() + eh)
            yv, ey = product(hv, w2[ex].double(), None)
            ey = ey + eh @ w2[ex].double().abs().t() * 1.01
            c = wt[at, j:j + 1].double()
            v[at] += c * yv
            e[at] += c * (ey + 2.0 ** -22 * yv.abs())
    close(out, v, e + 2.0 ** -22 * v.abs())


def test_an_ffn_of_4_bit_experts():
    """Quantised rows, products of groups, and the hidden rows quantised between them."""
    g = torch.Generator(device="cuda").manual_seed(6)
    T, E, k, d, F = 90, 8, 2, 256, 384
    x = torch.randn(T, d, device="cuda", generator=g).bfloat16()
    ids = torch.rand(T, E, device="cuda", generator=g).topk(k, dim=1)[1].int()
    i32, u8 = torch.int32, torch.uint8
    offsets, tokens, places = (torch.empty(*n, dtype=i32, device="cuda") for n in ((E + 1,), (T * k,), (T, k)))
    moe.group(ids, T, E, offsets, tokens, places, moe.group_workspace(T, k, E))
    w1, w3, w2 = (pack(torch.randn(E, *n, device="cuda", generator=g) * n[1] ** -0.5, "fit") for n in ((F, d), (F, d), (d, F)))
    xq, xs = torch.empty(T, d // 2, dtype=u8, device="cuda"), torch.empty(T, d // 32, dtype=u8, device="cuda")
    moe.mx_quantize(x, T, xq, xs)
    h, y = torch.empty(T * k, F, dtype=torch.bfloat16, device="cuda"), torch.empty(T * k, d, device="cuda")
    moe.grouped_linear(moe.make_grouped_desc(w1[0], w_s=w1[1], w_up=w3[0], w_up_s=w3[1], act=moe.LINEAR_SITU_GLU), xq, offsets, T * k,
                       h, None, moe.OUT_HALF, rows=tokens, x_s=xs)
    hq, hs = torch.empty(T * k, F // 2, dtype=u8, device="cuda"), torch.empty(T * k, F // 32, dtype=u8, device="cuda")
    moe.mx_quantize(h, T * k, hq, hs, rule=moe.MX_FIT)
    moe.grouped_linear(moe.make_grouped_desc(w2[0], w_s=w2[1]), hq, offsets, T * k, None, y, moe.OUT_F32, x_s=hs)
    out = torch.empty(T, d, device="cuda")
    moe.combine(y, T * k, places, None, T, out)
    torch.cuda.synchronize()
    xv = unpack(*pack(x))
    hv = unpack(*pack(h, "fit"))    # (of the hidden rows as they came out: a value next to a border may go either way)
    v, e = torch.zeros(T, d, dtype=torch.float64, device="cuda"), torch.zeros(T, d, dtype=torch.float64, device="cuda")
    for j in range(k):
        for t in range(T):
            ex, r = int(ids[t, j]), int(places[t, j])
            a, ea = product(xv[t:t + 1], unpack(w1[0][ex], w1[1][ex]), None)
            u, eu = product(xv[t:t + 1], unpack(w3[0][ex], w3[1][ex]), None)
            want, bound = finish("situ_glu", a, ea, u, eu, None)
            close(h[r:r + 1], want, bound)
            yv, ey = product(hv[r:r + 1], unpack(w2[0][ex], w2[1][ex]), None)
            v[t] += yv[0]
            e[t] += ey[0] + 2.0 ** -22 * yv[0].abs()
    close(out, v, e)
