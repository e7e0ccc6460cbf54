"""moe_gate and moe_route_gated on the GPU against a plain 64-bit implementation.

Ids and counts have to be equal.  Weights are computed in 64 bits and rounded to fp32 once: within half a step, 2^-24 of
the value, and the 2^-50 or so that the order of the 64-bit sums moves it by.
"""
import numpy as np
import pytest

import quantized_expert_gemv_sigmoid_amd as moe

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

HALF_STEP = 2.0 ** -24 * (1 + 2.0 ** -20)


def plain(logits, k, score=0, bias=None, groups=1, top_groups=1, group_score=0, renorm=1, scale=1.0):
    """Row by row, in 64 bits: (ids, weights, counts)."""
    logits = np.asarray(logits, np.float64)
    T, E = logits.shape
    b = np.zeros(E) if bias is None else np.asarray(bias, np.float64)
    ids, wts = np.full((T, k), -1, np.int32), np.zeros((T, k))
    for t in range(T):
        l = logits[t]
        on = (l != -np.inf) & (b != -np.inf)
        s = np.full(E, np.nan)
        with np.errstate(over="ignore", invalid="ignore"):
            if score == 0:
                s[on] = 1.0 / (1.0 + np.exp(-l[on]))
            elif on.any():
                m = np.nanmax(np.where(np.isnan(l[on]), -np.inf, l[on]))
                e = np.exp(np.where(l[on] == m, 0.0, l[on] - m))
                s[on] = e / e.sum()
            c = np.where(on, s + b, -np.inf)
        c = np.where(on & np.isnan(c), np.inf, c)
        if groups > 1:
            g = np.sort(c.reshape(groups, -1), axis=1)[:, ::-1]
            v = g[:, 0].copy()
            if group_score == 1 and g.shape[1] > 1:
                v += np.where(g[:, 1] == -np.inf, 0.0, g[:, 1])
            kept = sorted(range(groups), key=lambda i: (-v[i], i))[:top_groups]
            keep = np.zeros(groups, bool)
            keep[kept] = True
            c = np.where(np.repeat(keep, E // groups), c, -np.inf)
        order = [e for e in sorted(range(E), key=lambda i: (-c[i], i)) if c[e] > -np.inf][:k]
        w = s[order]
        tot = w.sum()
        if renorm:
            w = w / tot if tot != 0 else w
        ids[t, :len(order)] = order
        wts[t, :len(order)] = w * scale
    counts = np.bincount(ids[ids >= 0].ravel(), minlength=E)
    return ids, wts, counts


def run(logits, k, bias=None, counts=True, **kw):
    T, E = logits.shape
    ids = torch.full((T, k), 77, dtype=torch.int32, device="cuda")
    w = torch.full((T, k), 7.0, device="cuda")
    c = torch.full((E,), 99, dtype=torch.int32, device="cuda") if counts else None
    bd = None if bias is None else torch.as_tensor(bias, dtype=torch.float32).cuda()
    moe.gate(moe.make_gate_desc(E, k, bias=bd, **kw), logits, T, ids, w, c)
    torch.cuda.synchronize()
    return ids.cpu().numpy(), w.cpu().numpy(), None if c is None else c.cpu().numpy()


def check(logits, k, bias=None, **kw):
    """logits: a CUDA tensor; kw as make_gate_desc's."""
    ids, w, c = run(logits, k, bias, **kw)
    names = dict(score="score", n_groups="groups", top_groups="top_groups", group_score="group_score", renorm="renorm",
                 routed_scale="scale")
    rid, rw, rc = plain(logits.double().cpu().numpy(), k, bias=bias, **{names[n]: v for n, v in kw.items()})
    assert np.array_equal(ids, rid)
    assert np.array_equal(c, rc)
    assert np.array_equal(np.isnan(w), np.isnan(rw))
    ok = ~np.isnan(rw)
    assert (np.abs(w[ok] - rw[ok]) <= HALF_STEP * np.abs(rw[ok]) + 2.0 ** -150).all()


def logits_of(T, E, seed, dtype=torch.float32, pad=0, spread=1.5):
    g = torch.Generator().manual_seed(seed)
    wide = torch.full((T, E + pad), float("nan"))
    wide[:, :E] = torch.randn(T, E, generator=g) * spread
    return wide.to(dtype).cuda()[:, :E]


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 2, 2), (3, 8, 1), (5, 63, 6), (4, 64, 64), (7, 65, 64), (1, 896, 16),
                                   (33, 128, 8), (130, 200, 12), (257, 384, 8), (65, 896, 16), (40, 1000, 33),
                                   (9, 1024, 64), (2000, 60, 4)])
@pytest.mark.parametrize("score", [moe.SCORE_SIGMOID, moe.SCORE_SOFTMAX])
def test_sizes(T, E, k, score):
    print(f"case: T={T} E={E} k={k} score={score}", flush=True)
    rng = np.random.default_rng(T * 1000 + E + k)
    bias = (rng.standard_normal(E) * 0.05).astype(np.float32)
    logits = logits_of(T, E, E + k)
    check(logits, k, bias, score=score)
    check(logits, k, None, score=score, renorm=0, routed_scale=2.5)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("pad", [0, 1, 8])
def test_types_and_strides(dtype, pad):
    # 16-bit logits of 300 experts hold equal ones: the lower id comes first
    check(logits_of(21, 300, 5, dtype, pad), 10, score=moe.SCORE_SOFTMAX)
    check(logits_of(21, 300, 6, dtype, pad), 10, np.linspace(-0.1, 0.1, 300).astype(np.float32))


@pytest.mark.parametrize("E,G,top,k", [(256, 8, 4, 8), (60, 6, 3, 4), (64, 64, 7, 7), (896, 2, 1, 16), (896, 56, 20, 16),
                                       (1024, 4, 2, 64), (12, 3, 1, 4), (320, 5, 5, 8)])
@pytest.mark.parametrize("group_score", [moe.GROUP_MAX, moe.GROUP_TOP2])
def test_groups(E, G, top, k, group_score):
    print(f"case: E={E} G={G} top={top} k={k} group_score={group_score}", flush=True)
    bias = (np.random.default_rng(E + G).standard_normal(E) * 0.1).astype(np.float32)
    for score in (moe.SCORE_SIGMOID, moe.SCORE_SOFTMAX):
        check(logits_of(50, E, G + k), k, bias, score=score, n_groups=G, top_groups=top, group_score=group_score)


def test_ties_go_to_the_lower_id_and_group():
    logits = torch.zeros(3, 130, device="cuda")
    logits[1, 77] = logits[1, 129] = 1.0
    logits[2] = torch.arange(130, device="cuda") % 3
    for score in (moe.SCORE_SIGMOID, moe.SCORE_SOFTMAX):
        check(logits, 20, score=score)
        for gs in (moe.GROUP_MAX, moe.GROUP_TOP2):
            check(logits, 20, score=score, n_groups=13, top_groups=4, group_score=gs)


def test_scores_that_fp32_would_make_equal():
    # sigmoid(17 + i / 8) rounds to 1 in fp32; in 64 bits the larger logit wins
    logits = (17.0 + torch.arange(96, device="cuda").float().view(1, 96) / 8).repeat(2, 1)
    check(logits, 7)
    # c differs in the 40th bit
    bias = np.full(96, 0.25, np.float32)
    base = torch.zeros(1, 96, device="cuda")
    base[0, 50] = 2.0 ** -30
    check(base, 3, bias)
    check(base, 3, bias, score=moe.SCORE_SOFTMAX)


@pytest.mark.parametrize("score", [moe.SCORE_SIGMOID, moe.SCORE_SOFTMAX])
@pytest.mark.parametrize("groups", [1, 4])
def test_masked_experts_and_empty_rows(score, groups):
    logits = logits_of(6, 96, 11)
    logits[0, :] = -float("inf")                 # nothing left
    logits[1, 1:] = -float("inf")                # one expert
    logits[2, 5:] = -float("inf")                # fewer than k
    logits[3, ::2] = -float("inf")
    logits[4, 3] = torch.finfo(torch.float32).min  # a finite logit takes part
    bias = np.zeros(96, np.float32)
    bias[40:60] = -np.inf                        # experts switched off ...
    logits[5, 41] = float("nan")                 # ... whatever their logit is
    logits[5, 42] = float("inf")
    kw = dict(score=score, n_groups=groups, top_groups=max(1, groups // 2), group_score=moe.GROUP_TOP2)
    check(logits, 8, bias, **kw)
    check(logits, 8, bias, renorm=0, **kw)
    check(logits[:5], 8, None, **kw)


@pytest.mark.parametrize("score", [moe.SCORE_SIGMOID, moe.SCORE_SOFTMAX])
def test_infinities_and_nan(score):
    logits = logits_of(5, 70, 3)
    logits[0, 9] = float("inf")
    logits[1, 9] = logits[1, 69] = float("inf")
    logits[2, 33] = float("nan")
    logits[3, :] = float("nan")
    logits[4] = torch.linspace(-3e38, 3e38, 70)
    check(logits, 4, score=score)
    check(logits, 4, score=score, renorm=0)
    bias = np.zeros(70, np.float32)
    bias[7], bias[8] = np.inf, np.nan
    check(logits, 4, bias, score=score, renorm=0)


def test_scores_that_vanish():
    # every chosen sigmoid is 0 in 64 bits: the weights are 0, not 0 / 0
    logits = torch.full((2, 40), -800.0, device="cuda")
    logits[1, 3] = -3.0e38
    check(logits, 5)
    check(logits, 5, score=moe.SCORE_SOFTMAX)


def test_rows_behind_stay_and_same_bits():
    logits = logits_of(40, 256, 8)
    d = moe.make_gate_desc(256, 8, n_groups=8, top_groups=4, group_score=moe.GROUP_TOP2)
    got = []
    for _ in range(3):
        ids = torch.full((40, 8), 77, dtype=torch.int32, device="cuda")
        w = torch.full((40, 8), 7.0, device="cuda")
        c = torch.empty(256, dtype=torch.int32, device="cuda")
        moe.gate(d, logits, 23, ids, w, c)
        torch.cuda.synchronize()
        assert (ids[23:] == 77).all() and (w[23:] == 7.0).all()
        assert int(c.sum()) == 23 * 8
        got.append((ids.cpu(), w.cpu(), c.cpu()))
    for g in got[1:]:
        assert all(torch.equal(a, b) for a, b in zip(g, got[0]))


def test_no_tokens():
    ids = torch.full((1, 2), 5, dtype=torch.int32, device="cuda")
    w = torch.full((1, 2), 5.0, device="cuda")
    c = torch.full((8,), 5, dtype=torch.int32, device="cuda")
    moe.gate(moe.make_gate_desc(8, 2), torch.zeros(1, 8, device="cuda"), 0, ids, w, c)
    torch.cuda.synchronize()
    assert (ids == 5).all() and (w == 5.0).all() and (c == 5).all()


@pytest.mark.parametrize("T", [1, 300])
def test_captured_and_replayed_on_another_stream(T):
    d = moe.make_gate_desc(256, 8, n_groups=8, top_groups=3)
    logits = logits_of(T, 256, 1)
    ids = torch.empty(T, 8, dtype=torch.int32, device="cuda")
    w, c = torch.empty(T, 8, device="cuda"), torch.empty(256, dtype=torch.int32, device="cuda")
    moe.gate(d, logits, T, ids, w, c)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        moe.gate(d, logits, T, ids, w, c)
    for seed in range(4):
        logits.copy_(logits_of(T, 256, 50 + seed))
        g.replay()
        torch.cuda.synchronize()
        a = [v.clone() for v in (ids, w, c)]
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            moe.gate(d, logits, T, ids, w, c)
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(a, (ids, w, c)))


# ------------------------------------------------------------------ from x, with the experts

@pytest.mark.parametrize("T", [1, 2, 9, 40])
def test_route_gated_and_experts(T):
    """The logits moe_route works on, this routing, and the experts on it, against the oracle's experts."""
    import oracle
    import synth
    import synth.device as sdev
    from support import assert_close, make_gpu_layer, tokens
    shape = synth.LayerShape(n_experts=40, top_k=6, n_shared=2, d_model=512, d_ffn=256)
    gl = make_gpu_layer(shape, 21)
    x, rw, _ = tokens(gl, T)
    xd = sdev.tokens_to_device(x)
    ws = moe.workspace(gl.desc, T)
    # logits as the oracle has them: 64-bit sums of the bf16 tokens and the fp32 router
    xf = (x.astype(np.uint32) << 16).view(np.float32).astype(np.float64)
    ref = xf @ np.asarray(rw, np.float64).reshape(40, 512).T
    bias = torch.zeros(40, device="cuda")
    bias[3] = -float("inf")
    for kw in (dict(score=moe.SCORE_SOFTMAX), dict(score=moe.SCORE_SIGMOID, n_groups=5, top_groups=2, group_score=1),
               dict(score=moe.SCORE_SOFTMAX, n_groups=4, top_groups=2, renorm=0, routed_scale=2.5)):
        names = dict(score="score", n_groups="groups", top_groups="top_groups", group_score="group_score",
                     renorm="renorm", routed_scale="scale")
        rid, rwt, rc = plain(ref, 6, bias=bias.cpu().numpy(), **{names[n]: v for n, v in kw.items()})
        ids = torch.empty(T, 6, dtype=torch.int32, device="cuda")
        w = torch.empty(T, 6, device="cuda")
        c = torch.empty(40, dtype=torch.int32, device="cuda")
        moe.route_gated(gl.desc, moe.make_gate_desc(40, 6, bias=bias, **kw), xd, T, ids, w, c, ws)
        torch.cuda.synchronize()
        # (the fp32 logits are off by at most 512 roundings of sums below 8, 512 * 8 * 2^-24 = 2.5e-4;
        # these tokens' choices are wider apart: the sets are equal, the weights off by e^(2 * 2.5e-4))
        same = [sorted(a) == sorted(b) for a, b in zip(ids.cpu().numpy().tolist(), rid.tolist())]
        assert all(same)
        got = np.take_along_axis(w.cpu().numpy(), np.argsort(ids.cpu().numpy(), 1), 1)
        want = np.take_along_axis(rwt, np.argsort(rid, 1), 1)
        assert (np.abs(got - want) <= 6e-4 * np.abs(want)).all()
        assert np.array_equal(c.cpu().numpy(), rc)
        out = torch.empty(T, 512, device="cuda")
        moe.expert_forward(gl.desc, xd, T, ids, w, 1, None, out, moe.OUT_F32, ws)
        torch.cuda.synchronize()
        h = gl.host
        o = oracle.forward(x, ids.cpu().numpy(), w.cpu().numpy(), oracle.held_arrays(h), oracle.shared_arrays(h))
        assert_close(out.cpu().numpy(), o, f"experts T={T}")


def test_calls_of_two_streams_at_once():
    """Two streams' calls of different sizes, several deep, each with its own outputs: each as alone."""
    g = torch.Generator(device="cuda").manual_seed(17)
    sides = []
    for T, E, k, kw in ((700, 896, 16, {}), (1900, 60, 4, dict(score=moe.SCORE_SOFTMAX, n_groups=6, top_groups=3))):
        l = torch.randn(T, E, device="cuda", generator=g)
        sides.append((moe.make_gate_desc(E, k, **kw), l, T, [torch.empty(T, k, dtype=torch.int32, device="cuda") for _ in range(2)],
                      [torch.empty(T, k, device="cuda") for _ in range(2)],
                      [torch.empty(E, dtype=torch.int32, device="cuda") for _ in range(2)]))
    for d, l, T, ids, w, c in sides:
        moe.gate(d, l, T, ids[0], w[0], c[0])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sides]
    for _ in range(10):
        for s, (d, l, T, ids, w, c) in zip(streams, sides):
            moe.gate(d, l, T, ids[1], w[1], c[1], stream=s)
    torch.cuda.synchronize()
    for _, _, _, ids, w, c in sides:
        assert torch.equal(ids[0], ids[1]) and torch.equal(w[0], w[1]) and torch.equal(c[0], c[1])


def test_rows_past_two_gib():
    """Rows a wide distance apart, the last ones past 2^31 and 2^32 bytes."""
    T, E, ld = 520, 64, 1 << 21
    buf = torch.zeros(T * ld, device="cuda")
    l = torch.randn(T, E, device="cuda")
    rows = buf.view(T, ld)[:, :E]
    rows.copy_(l)
    d = moe.make_gate_desc(E, 6)
    out = [(torch.empty(T, 6, dtype=torch.int32, device="cuda"), torch.empty(T, 6, device="cuda")) for _ in range(2)]
    for (ids, w), logits in zip(out, (l, rows)):
        moe.gate(d, logits, T, ids, w)
    torch.cuda.synchronize()
    assert torch.equal(out[0][0], out[1][0]) and torch.equal(out[0][1], out[1][1])
