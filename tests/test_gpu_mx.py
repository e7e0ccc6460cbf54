"""moe_mx_quantize and moe_mx_dequantize on the GPU: every code, scale and value equal to the format's definition in 64
bits (nothing but the codes is rounded, so there is no tolerance)."""
import pytest

import quantized_expert_gemv_sigmoid_amd as moe
from mx_support import pack, power, unpack

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

TYPES = (torch.bfloat16, torch.float16, torch.float32)
RULES = {"floor": moe.MX_FLOOR, "fit": moe.MX_FIT}


def spread(T, n, dtype, seed):
    """Values over many powers of two, some zero blocks, values next to halfway points."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(T, n, device="cuda", generator=g, dtype=torch.float64)
    lim = 14 if dtype == torch.float16 else 100
    x = x * power(torch.randint(-lim, lim - 1, (T, 1), device="cuda", generator=g))
    ties = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.0, 7.5, 0.0], dtype=torch.float64, device="cuda")
    pick = ties[torch.randint(0, len(ties), (T, n), device="cuda", generator=g)]
    sign = torch.randint(0, 2, (T, n), device="cuda", generator=g) * 2.0 - 1
    x = torch.where(torch.rand(T, 1, device="cuda", generator=g) < 0.5, pick * sign, x)
    x = torch.where(torch.rand(T, n, device="cuda", generator=g) < 0.1, 0.0, x)
    return x.to(dtype)


def quantize(x, rule, codes_pad=0, scales_pad=0):
    """Codes and scales with sentinels between and behind the rows checked."""
    T, n = x.shape
    b = (n + 31) // 32
    codes = torch.full((T + 2, 16 * b + codes_pad), 0xA5, dtype=torch.uint8, device="cuda")
    scales = torch.full((T + 2, b + scales_pad), 0xA5, dtype=torch.uint8, device="cuda")
    moe.mx_quantize(x, T, codes[:, :16 * b], scales[:, :b], rule=RULES[rule])
    torch.cuda.synchronize()
    for o, w in ((codes, 16 * b), (scales, b)):
        assert (o[T:] == 0xA5).all() and (o[:, w:] == 0xA5).all()
    return codes[:T, :16 * b], scales[:T, :b]


SHAPES = [(1, 1), (1, 31), (1, 32), (1, 33), (3, 7), (5, 64), (1, 7168), (64, 100), (777, 1117), (2, 40000), (70000, 9),
          (301, 512), (33, 3584)]


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("rule", RULES)
@pytest.mark.parametrize("T,n", SHAPES)
def test_codes_and_scales(T, n, rule, dtype):
    print(f"case: {T}x{n} {rule} {dtype}", flush=True)
    x = spread(T, n, dtype, T + n)
    want_c, want_s = pack(x, rule)
    c, s = quantize(x, rule)
    assert torch.equal(s, want_s)
    assert torch.equal(c, want_c)
    # and back, in each type: exact but for fp16's own rounding
    v = unpack(c, s)[:, :n]
    for t in TYPES:
        out = torch.full((T + 1, n), 7.0, dtype=t, device="cuda")
        moe.mx_dequantize(c, s, T, out)
        torch.cuda.synchronize()
        assert torch.equal(out[:T], v.to(t)) and (out[T] == 7.0).all()


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("pads", [(1, 1, 1), (3, 5, 7), (8, 16, 4)])
def test_rows_apart_at_any_address(dtype, pads):
    T, n = 37, 1000
    x = spread(T, n, dtype, 3)
    wide = torch.full((T * (n + pads[0]) + 1,), float("nan"), dtype=dtype, device="cuda")
    rows = wide[1:].view(T, n + pads[0])[:, :n]
    rows.copy_(x)
    want = pack(x, "fit")
    c, s = quantize(rows, "fit", pads[1], pads[2])
    assert torch.equal(c, want[0]) and torch.equal(s, want[1])
    out = torch.full((T * (n + pads[0]) + 1,), 7.0, dtype=dtype, device="cuda")
    o = out[1:].view(T, n + pads[0])
    moe.mx_dequantize(c, s, T, o[:, :n])
    torch.cuda.synchronize()
    assert torch.equal(o[:, :n], unpack(c, s)[:, :n].to(dtype)) and (o[:, n:] == 7.0).all()


def test_every_16_bit_value():
    """Each 16-bit pattern as the largest of a block, with its neighbours and halves beside it."""
    for dtype in (torch.bfloat16, torch.float16):
        bits = torch.arange(65536, device="cuda", dtype=torch.int32)
        x = torch.zeros(65536, 32, dtype=torch.int32, device="cuda")
        x[:, 0] = bits
        for j in range(1, 32):
            x[:, j] = (bits & 0x7fff) - j * 13 * (j % 5 + 1)
        x[:, 1:] = x[:, 1:].clamp_min(0) | (torch.arange(1, 32, device="cuda") % 2 * 0x8000).int()
        x = torch.where(x > 32767, x - 65536, x).to(torch.int16).view(dtype)
        for rule in RULES:
            c, s = quantize(x, rule)
            want_c, want_s = pack(x, rule)
            assert torch.equal(s, want_s) and torch.equal(c, want_c)


def test_extremes_of_fp32():
    big, tiny = torch.finfo(torch.float32).max, 2.0 ** -149
    rows = [[big], [-big, 1.0], [tiny], [2.0 ** -126, tiny * 3], [2.0 ** -128, -2.0 ** -129, 2.0 ** -130], [0.0, -0.0],
            [2.0 ** -125 * 1.75], [2.0 ** 127, 2.0 ** 125 * 1.25]]
    x = torch.zeros(len(rows), 32, device="cuda")
    for i, r in enumerate(rows):
        x[i, :len(r)] = torch.tensor(r, dtype=torch.float64).float()
    for rule in RULES:
        c, s = quantize(x, rule)
        want = pack(x, rule)
        assert torch.equal(s, want[1]) and torch.equal(c, want[0])
        out = torch.empty_like(x)
        moe.mx_dequantize(c, s, len(rows), out)
        assert torch.equal(out, unpack(c, s).float())


@pytest.mark.parametrize("dtype", TYPES, ids=str)
def test_infinities_and_nan(dtype):
    """They mark their own block, and no other."""
    x = torch.randn(6, 128, device="cuda").to(dtype)
    x[1, 5], x[2, 40], x[3, 127], x[4, 0] = float("nan"), float("inf"), -float("inf"), -float("nan")
    c, s = quantize(x, "floor")
    want = pack(x)
    assert torch.equal(c, want[0]) and torch.equal(s, want[1])
    assert (s == 255).sum() == 4 and (c[1, :16] == 0).all()
    out = torch.empty_like(x)
    moe.mx_dequantize(c, s, 6, out)
    bad = (s == 255).repeat_interleave(32, 1)
    assert torch.isnan(out[bad]).all() and torch.isfinite(out[~bad]).all()


def test_no_rows_and_a_few_of_them():
    x = torch.ones(4, 64, device="cuda")
    c = torch.full((4, 32), 9, dtype=torch.uint8, device="cuda")
    s = torch.full((4, 2), 9, dtype=torch.uint8, device="cuda")
    moe.mx_quantize(x, 0, c, s)
    moe.mx_dequantize(c, s, 0, x)
    torch.cuda.synchronize()
    assert (c == 9).all() and (s == 9).all() and (x == 1).all()
    moe.mx_quantize(x, 3, c, s)
    torch.cuda.synchronize()
    assert (s[:3] == 125).all() and (c[:3] == 0x66).all() and (c[3] == 9).all() and (s[3] == 9).all()


def test_a_million_rows_of_one_value():
    T = (1 << 20)
    x = power(torch.arange(T, device="cuda") % 40 - 20)[:, None].bfloat16()
    c, s = quantize(x, "floor")
    assert torch.equal(s, pack(x)[1]) and torch.equal(c, pack(x)[0])


def test_weights_made_here_are_the_layers():
    """The layer on experts that moe_mx_quantize made: equal to the layer on the definition's."""
    g = torch.Generator(device="cuda").manual_seed(5)
    E, k, d, F, T = 8, 2, 256, 512, 4
    t = {"router_w": torch.randn(E, d, device="cuda", generator=g)}
    u = dict(t)
    for name, shape in (("w1", (E, F, d)), ("w3", (E, F, d)), ("w2", (E, d, F))):
        w = (torch.randn(*shape, device="cuda", generator=g) * shape[2] ** -0.5).bfloat16()
        q = torch.empty(E, shape[1], shape[2] // 2, dtype=torch.uint8, device="cuda")
        s = torch.empty(E, shape[1], shape[2] // 32, dtype=torch.uint8, device="cuda")
        moe.mx_quantize(w.view(-1, shape[2]), E * shape[1], q.view(-1, shape[2] // 2), s.view(-1, shape[2] // 32), rule=moe.MX_FIT)
        t[name + "_q"], t[name + "_s"] = q, s
        u[name + "_q"], u[name + "_s"] = pack(w, "fit")
    x = torch.randn(T, d, device="cuda", generator=g).bfloat16()
    outs = []
    for tensors in (t, u):
        desc = moe.make_desc(E, k, d, F, 0, tensors)
        out = torch.empty(T, d, device="cuda")
        moe.layer(desc, x, T, None, out, moe.OUT_F32, moe.workspace(desc, T))
        outs.append(out)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], outs[1]) and torch.isfinite(outs[0]).all()
