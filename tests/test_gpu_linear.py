"""moe_linear on the GPU against the formula in 64 bits.

Two kinds of checks:
- inputs that are small whole numbers: every product and sum is exact in fp32, so outputs without an activation have to
  be equal bit for bit, whatever the order of the sums;
- normal inputs, every output within a bound derived from the arithmetic (`bound`): a sum of K products in fp32 is off
  by at most (K + 2) 2^-23 sum |x w| (a step of 2^-23, not half of one: the matrix cores may cut instead of round), an
  activation passes that on with its largest slope and adds its own error, and the output's rounding adds half a step.
"""
import math

import pytest

import quantized_expert_gemv_sigmoid_amd as moe

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

PLAIN = ("none", "relu", "silu", "gelu", "gelu_tanh")
GATED = ("situ_glu", "swiglu")
B1, B2 = 4.0, 25.0
HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}


def act64(name, a, u):
    if name == "relu":
        return torch.where(a < 0, 0.0, a)
    if name == "silu":
        return a * torch.sigmoid(a)
    if name == "gelu":
        return 0.5 * a * torch.erfc(-a * math.sqrt(0.5))
    if name == "gelu_tanh":
        return 0.5 * a * (1 + torch.tanh(math.sqrt(2 / math.pi) * (a + 0.044715 * a ** 3)))
    if name == "swiglu":
        return a * torch.sigmoid(a) * u
    if name == "situ_glu":
        return B1 * torch.tanh(a / B1) * torch.sigmoid(a) * B2 * torch.tanh(u / B2)
    return a


def make(T, K, N, dtype, act="none", bias=None, residual=None, whole=False, seed=0, padx=0, padw=0, padr=0):
    """Inputs on the GPU; rows of x, w, residual apart by the pads, NaN between them."""
    g = torch.Generator(device="cuda").manual_seed(seed)

    def values(r, c, std):
        if whole:
            return torch.randint(-3, 4, (r, c), device="cuda", generator=g).float()
        return torch.randn(r, c, device="cuda", generator=g) * std

    def rows(r, c, pad, std, dt):
        t = torch.full((r, c + pad), float("nan"), device="cuda").to(dt)
        t[:, :c] = values(r, c, std)
        return t[:, :c]

    s = dict(T=T, K=K, N=N, dtype=dtype, act=act, w_up=None, bias=None, bias_up=None, residual=None)
    s["x"] = rows(T, K, padx, 1.0, dtype)
    s["w"] = rows(N, K, padw, K ** -0.5, dtype)
    if act in GATED:
        s["w_up"] = rows(N, K, padw, K ** -0.5, dtype)
    if bias is not None:
        s["bias"] = values(1, N, 0.5)[0].to(bias)
        if act in GATED:
            s["bias_up"] = values(1, N, 0.5)[0].to(bias)
    if residual is not None:
        s["residual"] = rows(T, N, padr, 1.0, residual)
    return s


def call(s, mode, ldo_pad=0, ws=None, stream=None, T=None):
    """(16-bit output, fp32 output) with sentinels between rows and behind them checked."""
    T, N = s["T"] if T is None else T, s["N"]
    d = moe.make_linear_desc(s["w"], w_up=s["w_up"], bias=s["bias"], bias_up=s["bias_up"],
                             act=getattr(moe, "LINEAR_" + s["act"].upper()), situ_b1=B1, situ_b2=B2,
                             residual_type=None if s["residual"] is None or s["residual"].dtype != torch.float32 else moe.F32)
    h = torch.full((T + 2, N + ldo_pad), 99.0, device="cuda").to(s["dtype"])
    f = torch.full((T + 2, N + ldo_pad), 99.0, device="cuda")
    ws = moe.linear_workspace(d, T) if ws is None else ws
    moe.linear(d, s["x"], T, h[:, :N], f[:, :N], mode, ws, residual=s["residual"], stream=stream)
    torch.cuda.synchronize()
    for o, written in ((h, mode != moe.OUT_F32), (f, mode != moe.OUT_HALF)):
        assert (o[T:] == 99.0).all() and (o[:, N:] == 99.0).all()
        if not written:
            assert (o == 99.0).all()
    return h[:T, :N], f[:T, :N]


def reference(s):
    """(output in 64 bits, bound on an fp32 result's error before its rounding)."""
    K = s["K"]
    x = s["x"].double()

    def product(w, b):
        w = w.double()
        v, m = x @ w.t(), x.abs() @ w.abs().t()
        if b is not None:
            v, m = v + b.double(), m + b.double().abs()
        return v, (K + 2) * 2.0 ** -23 * m

    a, ea = product(s["w"], s["bias"])
    u, eu = product(s["w_up"], s["bias_up"]) if s["w_up"] is not None else (None, None)
    v = act64(s["act"], a, u)
    # exp(z) from 2^(z log2 e) in fp32 is off by (|z| + 4) 2^-23 of itself; a few more operations of 2^-23 each
    own = 2.0 ** -23
    if s["act"] in ("none", "relu"):
        e = ea
    elif s["act"] in PLAIN:   # slopes up to 1.13
        e = 1.13 * ea + (2 * a.abs() ** 3 * 0.1 + 2 * a.abs() + 16) * own * torch.maximum(v.abs(), a.abs() * torch.sigmoid(-a.abs()))
        if s["act"] == "gelu":  # erfc: 16 steps of itself, and its argument's rounding times a^2
            e = e + (16 + a * a) * own * v.abs()
    else:
        silu = a * torch.sigmoid(a)
        if s["act"] == "swiglu":
            e = 1.13 * ea * (u.abs() + eu) + silu.abs() * eu + (2 * a.abs() + 16) * own * v.abs()
        else:  # both tanh have slopes up to 1; below 1/16 their polynomial, above it 1 - e with e up to 0.9: 32 steps
            e = 1.13 * ea * (u.abs() + eu) + silu.abs() * eu + (2 * a.abs() + 2 * u.abs() + 64) * own * v.abs()
    if s["residual"] is not None:
        r = s["residual"].double()
        v = v + r
        e = e + own * v.abs()
    return v, e


def check(s, out, dtype):
    v, e = reference(s)
    assert torch.isfinite(out).all()
    off = (out.double() - v).abs()
    tiny = 2.0 ** -25 if dtype == torch.float16 else 2.0 ** -140   # half a step of the type's subnormal numbers
    lim = e * (1 + HALF[dtype]) + HALF[dtype] * v.abs() + tiny
    worst = (off / lim).max()
    assert worst <= 1.0, f"off by {worst:.3g} of the bound"


SIZES = [(1, 1, 1), (1, 7, 3), (2, 8, 16), (3, 32, 33), (1, 640, 512), (5, 64, 64), (16, 256, 130), (17, 264, 130),
         (31, 100, 257), (33, 520, 48), (64, 512, 96), (65, 1024, 256), (130, 72, 640), (200, 448, 512),
         (256, 256, 256), (300, 520, 1032), (257, 129, 391), (513, 640, 768), (100, 2056, 40)]


@pytest.mark.parametrize("T,K,N", SIZES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_whole_numbers_are_exact(T, K, N, dtype):
    print(f"case: T={T} K={K} N={N} {dtype}", flush=True)
    s = make(T, K, N, dtype, bias=dtype, residual=torch.float32, whole=True, seed=T + K + N)
    v, _ = reference(s)
    h, f = call(s, moe.OUT_BOTH)
    assert torch.equal(f.double(), v)
    assert torch.equal(h, v.float().to(dtype))


# sizes at which the rule takes each of its kernels, with and without a split of K: served batches of up to 8, 16 and 32
# tokens a block, tiles of 64 x 32 to 256 x 256, and the tiles for rows that are not 16-byte aligned
KERNELS = [(5, 1000, 700), (13, 1000, 5000), (70, 4104, 1000), (30, 2056, 3000), (40, 1000, 4000), (260, 4104, 500),
           (100, 2056, 4000), (600, 4104, 512), (200, 2056, 4000), (1000, 8200, 260), (400, 1032, 4000), (200, 7176, 900),
           (1000, 1032, 2500), (140, 7176, 7000), (1000, 1160, 4000), (2060, 520, 4104), (1030, 6152, 6000), (300, 1025, 2001),
           (24, 4097, 300), (500, 1025, 2001), (60, 3585, 3587), (700, 2049, 1000), (1500, 1025, 2001)]
KERNELS_GATED = [(5, 1000, 700), (13, 1000, 3000), (30, 2056, 1500), (100, 2056, 2000), (400, 1032, 2000), (520, 1032, 1800),
                 (1000, 1160, 2000), (1000, 4104, 2052), (2060, 520, 2052), (500, 1025, 1001), (700, 2049, 500), (9, 4097, 150)]


@pytest.mark.parametrize("T,K,N", KERNELS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_every_kernel_is_exact(T, K, N, dtype):
    print(f"case: T={T} K={K} N={N} {dtype}", flush=True)
    s = make(T, K, N, dtype, bias=torch.float32, residual=dtype, whole=True, seed=T + K + N)
    v, _ = reference(s)
    h, f = call(s, moe.OUT_BOTH)
    assert torch.equal(f.double(), v)
    assert torch.equal(h, v.float().to(dtype))


@pytest.mark.parametrize("T,K,N", KERNELS_GATED)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_every_gated_kernel(T, K, N, dtype):
    print(f"case: T={T} K={K} N={N} {dtype}", flush=True)
    s = make(T, K, N, dtype, act="swiglu", bias=dtype, residual=torch.float32, seed=T + K + N)
    h, f = call(s, moe.OUT_BOTH)
    check(s, f, torch.float32)
    assert torch.equal(h, f.to(dtype))
    # gates of 30 and more: sigmoid is 1 in fp32, so whole numbers make whole numbers
    s = make(T, K, N, dtype, act="swiglu", whole=True, seed=T)
    s["bias"] = torch.full((N,), 4096.0, device="cuda")
    s["bias_up"] = torch.zeros(N, device="cuda")
    s["x"].clamp_(-1, 1)
    s["w"].mul_(0).add_(1)       # gate: 4096 + the sum of a row of -1 .. 1, above 4096 - 5 sqrt(K)
    v, _ = reference(s)
    keep = v.abs() < 2 ** 24     # (whole numbers that fp32 holds)
    _, f = call(s, moe.OUT_F32)
    assert torch.equal(f.double()[keep], v[keep].round())


@pytest.mark.parametrize("T,K,N", SIZES)
@pytest.mark.parametrize("act", GATED)
def test_gated_sizes(T, K, N, act):
    print(f"case: T={T} K={K} N={N} {act}", flush=True)
    dtype = torch.bfloat16 if (T + N) % 2 else torch.float16
    s = make(T, K, N, dtype, act=act, bias=torch.float32, residual=dtype, seed=T + K + N)
    h, f = call(s, moe.OUT_BOTH)
    check(s, f, torch.float32)
    assert torch.equal(h, f.to(dtype))   # one rounding of the fp32 output


@pytest.mark.parametrize("act", PLAIN + GATED)
@pytest.mark.parametrize("T,K,N", [(1, 256, 192), (24, 256, 192), (150, 256, 192), (600, 264, 384)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_activations(act, T, K, N, dtype):
    print(f"case: {act} T={T} {dtype}", flush=True)
    s = make(T, K, N, dtype, act=act, bias=dtype, seed=T)
    s["x"].mul_(3.0)   # sums up to about 15: both tails of each activation
    h, f = call(s, moe.OUT_BOTH)
    check(s, f, torch.float32)
    check(s, h, dtype)


@pytest.mark.parametrize("T", [1, 12, 70, 400])
@pytest.mark.parametrize("padx,padw,padr,ldo", [(0, 0, 0, 0), (8, 16, 4, 8), (1, 3, 5, 7), (6, 2, 0, 2), (0, 8, 1, 0)])
def test_strides(T, padx, padw, padr, ldo):
    print(f"case: T={T} pads {padx} {padw} {padr} {ldo}", flush=True)
    for K in (256, 250):
        s = make(T, K, 264, torch.bfloat16, bias=torch.bfloat16, residual=torch.bfloat16, whole=True, seed=T, padx=padx,
                 padw=padw, padr=padr)
        v, _ = reference(s)
        h, f = call(s, moe.OUT_BOTH, ldo_pad=ldo)
        assert torch.equal(f.double(), v)
        h, _ = call(s, moe.OUT_HALF, ldo_pad=ldo)
        assert torch.equal(h, v.float().bfloat16())
        _, f = call(s, moe.OUT_F32, ldo_pad=ldo)
        assert torch.equal(f.double(), v)


@pytest.mark.parametrize("T", [1, 20, 300])
@pytest.mark.parametrize("shift", [1, 2, 4])
def test_rows_that_start_anywhere(T, shift):
    """Elements of 2 bytes need no more alignment than that: x, w and the output start `shift` elements into a buffer."""
    print(f"case: T={T} shift={shift}", flush=True)
    s = make(T, 512, 192, torch.float16, whole=True, seed=T)
    for n in ("x", "w"):
        t = s[n]
        flat = torch.zeros(t.numel() + 16, dtype=t.dtype, device="cuda")
        s[n] = flat[shift:shift + t.numel()].view(t.shape)
        s[n].copy_(t)
    v, _ = reference(s)
    d = moe.make_linear_desc(s["w"])
    out = torch.zeros(T * 192 + 16, dtype=torch.float16, device="cuda")[shift:shift + T * 192].view(T, 192)
    moe.linear(d, s["x"], T, out, None, moe.OUT_HALF, moe.linear_workspace(d, T))
    torch.cuda.synchronize()
    assert torch.equal(out, v.half())


@pytest.mark.parametrize("T", [1, 9, 70, 300])
def test_broadcast_and_in_place_residual(T):
    print(f"case: T={T}", flush=True)
    s = make(T, 384, 320, torch.bfloat16, whole=True, seed=3)
    s["residual"] = torch.randint(-9, 9, (1, 320), device="cuda").float().expand(T, 320)
    v, _ = reference(s)
    _, f = call(s, moe.OUT_F32)
    assert torch.equal(f.double(), v)
    for dt, mode in ((torch.bfloat16, moe.OUT_HALF), (torch.float32, moe.OUT_F32)):
        s["residual"] = torch.randint(-9, 9, (T, 320), device="cuda").to(dt)
        v, _ = reference(s)
        d = moe.make_linear_desc(s["w"], residual_type=moe.F32 if dt == torch.float32 else None)
        o = s["residual"]
        moe.linear(d, s["x"], T, o if mode == moe.OUT_HALF else None, o if mode == moe.OUT_F32 else None, mode,
                   moe.linear_workspace(d, T), residual=o)
        torch.cuda.synchronize()
        assert torch.equal(o, v.to(dt))


def test_fewer_tokens_than_rows():
    s = make(40, 256, 128, torch.bfloat16, whole=True)
    v, _ = reference(s)
    for T in (0, 1, 23):
        _, f = call(s, moe.OUT_F32, T=T)
        assert torch.equal(f.double(), v[:T])


@pytest.mark.parametrize("T", [1, 16, 200, 600])
def test_infinities_and_nan_stay_in_their_rows(T):
    print(f"case: T={T}", flush=True)
    s = make(T, 264, 160, torch.float16, seed=9)
    ref, _ = call(s, moe.OUT_F32)
    _, ref = call(s, moe.OUT_F32)
    ref = ref.clone()
    s["x"][T - 1, 263] = float("inf")
    s["w"][159, 0] = float("nan")
    _, f = call(s, moe.OUT_F32)
    assert torch.equal(f[:T - 1, :159], ref[:T - 1, :159])
    assert torch.isnan(f[:, 159]).all()
    assert torch.isinf(f[T - 1, :159]).all()


def test_no_overflow_between_fp16_and_output():
    # sums past fp16's range: inf in the 16-bit output, the value in the fp32 one
    s = make(3, 64, 8, torch.float16)
    s["x"].fill_(100.0)
    s["w"].fill_(100.0)
    h, f = call(s, moe.OUT_BOTH)
    assert (f == 640000.0).all() and torch.isinf(h).all()


@pytest.mark.parametrize("T,K,N,act", [(1, 1024, 512, "none"), (30, 1024, 512, "swiglu"), (200, 2048, 320, "silu"),
                                       (700, 1536, 640, "situ_glu"), (64, 4096, 64, "none"), (90, 1117, 513, "gelu"),
                                       (2060, 520, 4104, "none"), (1030, 6152, 6000, "relu")])
def test_captured_and_replayed(T, K, N, act):
    """Replays between eager work equal the eager call, two graphs in turn on one workspace among them."""
    print(f"case: T={T} K={K} N={N} {act}", flush=True)
    sets = [make(T, K, N, torch.bfloat16, act=act, bias=torch.float32, residual=torch.bfloat16, seed=i) for i in (1, 2)]
    descs = [moe.make_linear_desc(s["w"], w_up=s["w_up"], bias=s["bias"], bias_up=s["bias_up"],
                                  act=getattr(moe, "LINEAR_" + act.upper())) for s in sets]
    ws = moe.linear_workspace(descs[0], T)
    outs = [torch.zeros(T, N, device="cuda") for _ in sets]

    def go(i):
        moe.linear(descs[i], sets[i]["x"], T, None, outs[i], moe.OUT_F32, ws, residual=sets[i]["residual"])

    want = []
    for i in (0, 1):
        go(i)
        torch.cuda.synchronize()
        want.append(outs[i].clone())
        check(sets[i], outs[i], torch.float32)
    graphs = []
    for i in (0, 1):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            go(i)
        graphs.append(g)
    for n in range(4):
        for i in (0, 1):
            outs[i].zero_()
            graphs[i].replay()
        ws.fill_(n)   # nothing in the workspace is kept between calls
        torch.cuda.synchronize()
        for i in (0, 1):
            assert torch.equal(outs[i], want[i])


def test_two_streams_with_their_own_workspaces():
    sets = [make(T, 2048, 256, torch.bfloat16, act="silu", seed=T) for T in (8, 150)]
    descs = [moe.make_linear_desc(s["w"], act=moe.LINEAR_SILU) for s in sets]
    ws = [moe.linear_workspace(d, s["T"]) for d, s in zip(descs, sets)]
    outs = [torch.zeros(s["T"], 256, device="cuda") for s in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    for _ in range(8):
        for i in (0, 1):
            moe.linear(descs[i], sets[i]["x"], sets[i]["T"], None, outs[i], moe.OUT_F32, ws[i], stream=streams[i])
    torch.cuda.synchronize()
    for s, o in zip(sets, outs):
        check(s, o, torch.float32)


def test_long_sums_and_rows_past_two_gib():
    """Offsets past 2^31 bytes: the last rows of a wide x and of the output."""
    T, K, N, ld = 300, 64, 136, 1 << 22
    x = torch.zeros(T * ld, dtype=torch.bfloat16, device="cuda").view(T, ld)[:, :K]
    s = make(T, K, N, torch.bfloat16, whole=True)
    x.copy_(s["x"])
    s["x"] = x
    v, _ = reference(s)
    d = moe.make_linear_desc(s["w"])
    o = torch.zeros(T * ld, device="cuda").view(T, ld)[:, :N]
    moe.linear(d, x, T, None, o, moe.OUT_F32, moe.linear_workspace(d, T))
    torch.cuda.synchronize()
    assert torch.equal(o.double(), v)
    s = make(9, 1 << 17, 20, torch.bfloat16, seed=4)
    check(s, call(s, moe.OUT_F32)[1], torch.float32)


# ------------------------------------------------------------------ the operators together

@pytest.mark.parametrize("T", [1, 6, 50])
def test_router_product_gate_experts_and_dense_layer(T):
    """A block as it is served: router logits by moe_linear, moe_gate, the MXFP4 experts on that routing, and a dense
    gated FFN (shared by all tokens) whose down product adds the experts' output and the stream."""
    import numpy as np
    import oracle
    import synth
    import synth.device as sdev
    from support import make_gpu_layer, tokens
    from test_gpu_gate import plain
    shape = synth.LayerShape(n_experts=40, top_k=6, n_shared=0, d_model=512, d_ffn=256)
    gl = make_gpu_layer(shape, 33)
    bits, _, _ = tokens(gl, T)
    x = sdev.tokens_to_device(bits).view(torch.bfloat16).view(T, 512)
    g = torch.Generator(device="cuda").manual_seed(T)
    wr, w1, w3 = (torch.randn(n, 512, device="cuda", generator=g).mul_(512 ** -0.5).bfloat16() for n in (40, 768, 768))
    w2 = (torch.randn(512, 768, device="cuda", generator=g) * 768 ** -0.5).bfloat16()
    router = moe.make_linear_desc(wr)
    logits = torch.empty(T, 40, device="cuda")
    moe.linear(router, x, T, None, logits, moe.OUT_F32, moe.linear_workspace(router, T))
    ids, wts = torch.empty(T, 6, dtype=torch.int32, device="cuda"), torch.empty(T, 6, device="cuda")
    moe.gate(moe.make_gate_desc(40, 6, score=moe.SCORE_SOFTMAX, n_groups=5, top_groups=3, routed_scale=2.0), logits, T, ids, wts)
    routed = torch.empty(T, 512, device="cuda")
    moe.expert_forward(gl.desc, x, T, ids, wts, 0, None, routed, moe.OUT_F32, moe.workspace(gl.desc, T))
    gate_up = moe.make_linear_desc(w1, w_up=w3, act=moe.LINEAR_SWIGLU)
    h = torch.empty(T, 768, dtype=torch.bfloat16, device="cuda")
    moe.linear(gate_up, x, T, h, None, moe.OUT_HALF, moe.linear_workspace(gate_up, T))
    down = moe.make_linear_desc(w2, residual_type=moe.F32)
    moe.linear(down, h, T, None, routed, moe.OUT_F32, moe.linear_workspace(down, T), residual=routed)
    torch.cuda.synchronize()

    rid, rwt, _ = plain(logits.double().cpu().numpy(), 6, score=1, groups=5, top_groups=3, scale=2.0)
    assert np.array_equal(ids.cpu().numpy(), rid)
    assert (np.abs(wts.cpu().numpy() - rwt) <= 2.0 ** -24 * 1.001 * rwt).all()
    xd = x.double()
    assert ((logits.double() - xd @ wr.double().t()).abs() <= 514 * 2.0 ** -23 * (xd.abs() @ wr.double().abs().t())).all()
    experts = torch.as_tensor(oracle.forward(bits, rid, rwt.astype(np.float32), oracle.held_arrays(gl.host), oracle.shared_arrays(gl.host), False)).double().cuda()
    a = xd @ w1.double().t()
    ref = experts + (a * torch.sigmoid(a) * (xd @ w3.double().t())) @ w2.double().t()
    # the experts' tolerance (2e-3 of their norm) and the dense FFN's bf16 H, 2^-8 of it at most
    dense = ref - experts
    assert (routed.double() - ref).norm() <= 2e-3 * experts.norm() + 2.0 ** -8 * dense.norm()
