"""moe_mx_linear on the GPU against the formula in 64 bits.

Operands are exact MXFP4 rows.  With whole numbers of equal scales every sum is exact and outputs without an activation
have to be equal; with normal rows the bound is moe_linear's (test_gpu_linear.py): a term that a matrix product of 128
cuts off is below 2^-23 of the largest one or of the sum so far, so K of them are within (K + 2) 2^-23 sum |x w|.
"""
import math

import pytest

import quantized_expert_gemv_sigmoid_amd as moe
from mx_support import pack, unpack
from test_gpu_linear import B1, B2, GATED, HALF, PLAIN, act64

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def rows_apart(t, pad, shift=0):
    """The rows of a uint8 tensor `pad` bytes apart, the first one `shift` bytes behind an aligned address; 255 between them."""
    T, n = t.shape
    flat = torch.full((T * (n + pad) + shift + 64,), 255, dtype=torch.uint8, device=t.device)
    v = flat[shift:shift + T * (n + pad)].view(T, n + pad)[:, :n]
    v.copy_(t)
    return v


def make(T, K, N, type=torch.bfloat16, act="none", bias=None, residual=None, whole=False, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def operand(r, std):
        if whole:   # whole numbers -4 .. 4 in blocks of scale 1, some of 2
            c = torch.tensor([0, 2, 4, 5, 6, 10, 12, 13, 14], dtype=torch.uint8, device="cuda")  # 0 1 2 3 4 -1 -2 -3 -4
            v = c[torch.randint(0, 9, (r, K), device="cuda", generator=g)]
            s = torch.randint(127, 129, (r, K // 32), device="cuda", generator=g).to(torch.uint8)
            return (v[:, 0::2] | (v[:, 1::2] << 4)).contiguous(), s
        x = torch.randn(r, K, device="cuda", generator=g) * std
        x = x * torch.exp2(torch.randint(-3, 4, (r, 1), device="cuda", generator=g).float())
        return pack(x, "fit")

    def values(*shape, std=0.5):
        if whole:
            return torch.randint(-3, 4, shape, device="cuda", generator=g).float()
        return torch.randn(*shape, device="cuda", generator=g) * std

    s = dict(T=T, K=K, N=N, type=type, act=act, up=(None, None), bias=None, bias_up=None, residual=None)
    s["x"], s["w"] = operand(T, 1.0), operand(N, K ** -0.5)
    if act in GATED:
        s["up"] = operand(N, K ** -0.5)
    if bias is not None:
        s["bias"] = values(N).to(bias)
        s["bias_up"] = values(N).to(bias) if act in GATED else None
    if residual is not None:
        s["residual"] = values(T, N, std=1.0).to(residual)
    return s


def descriptor(s):
    r = s["residual"]
    return moe.make_mx_linear_desc(
        s["w"][0], s["w"][1], w_up=s["up"][0], w_up_s=s["up"][1], bias=s["bias"], bias_up=s["bias_up"],
        type=moe.F16 if s["type"] == torch.float16 else moe.BF16, act=getattr(moe, "LINEAR_" + s["act"].upper()), situ_b1=B1,
        situ_b2=B2, residual_type=None if r is None or r.dtype != torch.float32 else moe.F32)


def call(s, mode=moe.OUT_BOTH, pad=0, ws=None, stream=None):
    T, N = s["T"], s["N"]
    d = descriptor(s)
    h = torch.full((T + 2, N + pad), 99.0, device="cuda").to(s["type"])
    f = torch.full((T + 2, N + pad), 99.0, device="cuda")
    ws = moe.mx_linear_workspace(d, T) if ws is None else ws
    moe.mx_linear(d, s["x"][0], s["x"][1], T, h[:, :N], f[:, :N], mode, ws, residual=s["residual"], stream=stream)
    torch.cuda.synchronize()
    for o, written in ((h, mode != moe.OUT_F32), (f, mode != moe.OUT_HALF)):
        assert (o[T:] == 99.0).all() and (o[:, N:] == 99.0).all()
        if not written:
            assert (o == 99.0).all()
    return h[:T, :N], f[:T, :N]


def finish(act, a, ea, u, eu, residual):
    """(act(a, u) + residual, bound on fp32's error of it) for sums off by up to ea, eu (test_gpu_linear.py's bounds)."""
    v, own = act64(act, a, u), 2.0 ** -23
    if act in ("none", "relu"):
        e = ea
    elif act in PLAIN:
        e = 1.13 * ea + (2 * a.abs() ** 3 * 0.1 + 2 * a.abs() + 16) * own * torch.maximum(v.abs(), a.abs() * torch.sigmoid(-a.abs()))
        if act == "gelu":
            e = e + (16 + a * a) * own * v.abs()
    else:
        silu = a * torch.sigmoid(a)
        if act == "swiglu":
            e = 1.13 * ea * (u.abs() + eu) + silu.abs() * eu + (2 * a.abs() + 16) * own * v.abs()
        else:
            e = 1.13 * ea * (u.abs() + eu) + silu.abs() * eu + (2 * a.abs() + 2 * u.abs() + 64) * own * v.abs()
    if residual is not None:
        v = v + residual.double()
        e = e + own * v.abs()
    return v, e


def product(x, w, b):
    v, m = x @ w.t(), x.abs() @ w.abs().t()
    if b is not None:
        v, m = v + b.double(), m + b.double().abs()
    return v, (x.shape[1] + 2) * 2.0 ** -23 * m


def reference(s):
    x = unpack(*s["x"])
    a, ea = product(x, unpack(*s["w"]), s["bias"])
    u, eu = product(x, unpack(*s["up"]), s["bias_up"]) if s["act"] in GATED else (None, None)
    return finish(s["act"], a, ea, u, eu, s["residual"])


def close(out, v, e):
    t = out.dtype
    half = HALF[t]
    bound = e + half * (v.abs() + e) + (2.0 ** -25 if t == torch.float16 else 1e-37)
    d = (out.double() - v).abs()
    assert torch.isfinite(out).all()
    assert (d <= bound).all(), f"{(d / bound).max().item():.2f} of the bound"


SIZES = [(1, 32, 1), (1, 64, 17), (1, 7168, 333), (2, 160, 40), (7, 256, 100), (13, 3584, 515), (24, 1024, 260), (33, 1120, 129),
         (200, 1120, 2049), (129, 2048, 640), (300, 96, 1000), (515, 3616, 770), (1100, 512, 3000), (2304, 384, 4096)]


@pytest.mark.parametrize("T,K,N", SIZES)
@pytest.mark.parametrize("gated", [0, 1])
def test_sizes(T, K, N, gated):
    print(f"case: {T}x{K}x{N} gated {gated}", flush=True)
    t = torch.float16 if (T + N) % 2 else torch.bfloat16
    s = make(T, K, N, t, act="swiglu" if gated else "none", bias=torch.float32, residual=t, seed=T + K)
    h, f = call(s, pad=3)
    v, e = reference(s)
    close(f, v, e)
    close(h, v, e)


@pytest.mark.parametrize("T,K,N", SIZES)
def test_whole_numbers_are_exact(T, K, N):
    print(f"case: {T}x{K}x{N}", flush=True)
    s = make(T, K, N, bias=torch.bfloat16, residual=torch.float32, whole=True, seed=N)
    h, f = call(s)
    v = reference(s)[0]
    assert v.abs().max() < 2 ** 24
    assert torch.equal(f.double(), v)
    assert torch.equal(h, v.float().to(s["type"]))


@pytest.mark.parametrize("act", PLAIN + GATED)
@pytest.mark.parametrize("T", [1, 20, 150, 600])
@pytest.mark.parametrize("residual", [None, torch.float32, torch.float16])
def test_activations(act, T, residual):
    s = make(T, 416, 300, torch.float16, act=act, bias=torch.float16, residual=residual, seed=T)
    v, e = reference(s)
    for mode in (moe.OUT_HALF, moe.OUT_F32):
        h, f = call(s, mode)
        close(f if mode == moe.OUT_F32 else h, v, e)


@pytest.mark.parametrize("T,K,N", [(1, 256, 64), (9, 1024, 200), (70, 640, 300), (300, 1152, 1000), (2304, 256, 4096)])
@pytest.mark.parametrize("shift", [0, 1])
def test_rows_apart(T, K, N, shift):
    """Codes at multiples of 16 bytes, scales anywhere: rows apart, 255 between them."""
    s = make(T, K, N, act="situ_glu", seed=N)
    for n in ("x", "w", "up"):
        c, sc = s[n]
        s[n] = rows_apart(c, 48), rows_apart(sc, 4 + 3 * shift, shift)
    h, f = call(s)
    v, e = reference(s)
    close(f, v, e)
    close(h, v, e)


def test_scales_of_nan_and_far_ones():
    """Byte 255 is NaN, in its row's outputs alone; scales far apart keep what fp32 holds."""
    s = make(40, 512, 96, seed=2)
    s["x"][1][3, 7] = 255
    s["w"][1][5, 2] = 255
    _, f = call(s)
    nan = torch.zeros(40, 96, dtype=torch.bool, device="cuda")
    nan[3], nan[:, 5] = True, True
    assert torch.isnan(f[nan]).all() and torch.isfinite(f[~nan]).all()
    for bx, bw in ((0, 254), (10, 240), (254, 1), (60, 100)):
        s = make(40, 512, 96, seed=3)
        s["x"][1].fill_(bx)
        s["w"][1].fill_(bw)
        _, f = call(s, moe.OUT_F32)
        v, e = reference(s)
        close(f, v, e)


def test_in_place_residual_and_fewer_rows():
    s = make(100, 512, 256, residual=torch.bfloat16, seed=8)
    v, e = reference(s)
    d = descriptor(s)
    out = s["residual"].clone()
    ws = moe.mx_linear_workspace(d, 100)
    moe.mx_linear(d, s["x"][0], s["x"][1], 100, out, None, moe.OUT_HALF, ws, residual=out)
    close(out, v, e)
    out = torch.full((100, 256), 5.0, dtype=torch.bfloat16, device="cuda")
    moe.mx_linear(d, s["x"][0], s["x"][1], 37, out, None, moe.OUT_HALF, ws, residual=s["residual"])
    close(out[:37], v[:37], e[:37])
    assert (out[37:] == 5.0).all()
    moe.mx_linear(d, s["x"][0], s["x"][1], 0, out, None, moe.OUT_HALF, ws)
    # the same row for every token
    one = s["residual"][:1].expand(100, 256)
    s["residual"] = one
    v, e = reference(s)
    moe.mx_linear(d, s["x"][0], s["x"][1], 100, out, None, moe.OUT_HALF, ws, residual=one)
    close(out, v, e)


def test_captured_and_on_another_stream():
    s = make(300, 1120, 500, act="silu", bias=torch.bfloat16, seed=4)   # (with the launch that copies scales)
    d = descriptor(s)
    want = call(s)[0].clone()
    out = torch.zeros(300, 500, dtype=torch.bfloat16, device="cuda")
    ws = moe.mx_linear_workspace(d, 300)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    moe.mx_linear(d, s["x"][0], s["x"][1], 300, out, None, moe.OUT_HALF, ws, stream=side)
    side.synchronize()
    assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.mx_linear(d, s["x"][0], s["x"][1], 300, out, None, moe.OUT_HALF, ws)
    for _ in range(3):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
        ws.fill_(255)
        torch.cuda.synchronize()


def test_quantised_on_the_way():
    """moe_mx_quantize and the product, as they are used: equal to the product of the definition's rows."""
    g = torch.Generator(device="cuda").manual_seed(9)
    x = torch.randn(50, 1000, device="cuda", generator=g).bfloat16()
    s = make(50, 1024, 320, seed=9)
    c = torch.empty(50, 512, dtype=torch.uint8, device="cuda")
    b = torch.empty(50, 32, dtype=torch.uint8, device="cuda")
    moe.mx_quantize(x, 50, c, b)
    s["x"] = pack(x)
    assert torch.equal(c, s["x"][0]) and torch.equal(b, s["x"][1])
    want = call(s, moe.OUT_F32)[1]
    s["x"] = c, b
    assert torch.equal(call(s, moe.OUT_F32)[1], want)
    v, e = reference(s)
    close(want, v, e)
    assert math.isfinite(v.abs().max().item())
