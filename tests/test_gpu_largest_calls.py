"""The largest tokens, choices, rows, groups, inputs and outputs that the MXFP4 product, the products of groups, moe_group and
moe_combine take, on whole numbers: every sum is exact in fp32, so outputs have to be equal."""
import pytest

import quantized_expert_gemv_sigmoid_amd as moe
from mx_support import pack, unpack

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def whole(*shape, seed=0, most=3):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(-most, most + 1, shape, device="cuda", generator=g).float()


def test_group():
    T, k, E = 1 << 20, 64, 1024
    g = torch.Generator(device="cuda").manual_seed(1)
    ids = torch.randint(-30, E, (T, k), device="cuda", generator=g, dtype=torch.int32)
    offsets, tokens = torch.empty(E + 1, dtype=torch.int32, device="cuda"), torch.full((T * k,), 77, dtype=torch.int32, device="cuda")
    places = torch.empty(T, k, dtype=torch.int32, device="cuda")
    moe.group(ids, T, E, offsets, tokens, places, moe.group_workspace(T, k, E))
    torch.cuda.synchronize()
    flat = torch.where(ids < 0, E, ids).view(-1)
    order = torch.sort(flat, stable=True)[1]
    n = int((flat < E).sum())
    assert torch.equal(offsets[1:].long(), torch.bincount(flat, minlength=E + 1)[:E].cumsum(0)) and offsets[0] == 0
    assert torch.equal(tokens[:n].long(), order[:n] // k) and (tokens[n:] == 77).all()
    want = torch.full_like(flat, -1)
    want[order[:n]] = torch.arange(n, device="cuda", dtype=torch.int32)
    assert torch.equal(places.view(-1), want)


def test_combine():
    T, k, n, R = 1 << 20, 64, 8, 5000
    g = torch.Generator(device="cuda").manual_seed(2)
    y, w, res = whole(R, n), whole(T, k, seed=3), whole(T, n, seed=4)
    places = torch.randint(-100, R + 100, (T, k), device="cuda", generator=g, dtype=torch.int32)
    out = torch.full((T + 1, n), 99.0, device="cuda")
    moe.combine(y, R, places, w, T, out, residual=res)
    torch.cuda.synchronize()
    v = res.clone()
    for j in range(k):
        on = (places[:, j] >= 0) & (places[:, j] < R)
        v += torch.where(on, w[:, j], 0.0)[:, None] * y[places[:, j].long().clamp(0, R - 1)]
    assert torch.equal(out[:T], v) and (out[T] == 99.0).all()


def grouped(E, R, X, K, N, mx, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x, w = whole(X, K, seed=seed), whole(E, N, K, seed=seed + 1)
    bias = whole(E, N, seed=seed + 2)
    cuts = torch.randint(0, R - R // 50, (E - 1,), device="cuda", generator=g)
    offsets = torch.cat([torch.zeros(1, device="cuda", dtype=torch.long), torch.sort(cuts)[0],
                         torch.full((1,), R - R // 50, device="cuda")]).int()
    rows = torch.randint(0, X, (R,), device="cuda", generator=g, dtype=torch.int32)
    rows[::1001] = -1
    s = dict(x=x.bfloat16(), w=w.bfloat16(), x_s=None, w_s=None)
    if mx:
        (s["x"], s["x_s"]), (s["w"], s["w_s"]) = pack(x, "fit"), pack(w, "fit")
        assert torch.equal(unpack(s["x"], s["x_s"]).float(), x) and torch.equal(unpack(s["w"], s["w_s"]).float(), w)
    out = torch.full((R + 1, N), 99.0, device="cuda")
    moe.grouped_linear(moe.make_grouped_desc(s["w"], w_s=s["w_s"], bias=bias), s["x"], offsets, R, None, out, moe.OUT_F32, rows=rows,
                       x_s=s["x_s"])
    torch.cuda.synchronize()
    # the sums of every row of x with every group's weights, and of a row of zeros behind them
    sums = torch.stack([torch.cat([x.double() @ w[e].double().t(), torch.zeros(1, N, device="cuda", dtype=torch.float64)]) + bias[e].double()
                        for e in range(E)]).float()
    end = int(offsets[-1])
    group = torch.bucketize(torch.arange(end, device="cuda", dtype=torch.int32), offsets[1:].contiguous(), right=True)
    assert torch.equal(out[:end], sums[group, torch.where(rows < 0, X, rows)[:end].long()])
    assert (out[end:] == 99.0).all()


@pytest.mark.parametrize("mx", [False, True])
def test_rows_and_groups(mx):
    grouped(1024, 1 << 24, 1000, 128 if mx else 8, 8, mx, 5)


@pytest.mark.parametrize("mx", [False, True])
def test_inputs_of_groups(mx):
    grouped(2, 60, 7, 1 << 20, 3, mx, 6)


@pytest.mark.parametrize("mx", [False, True])
def test_outputs_of_groups(mx):
    grouped(2, 60, 7, 128 if mx else 8, 1 << 20, mx, 7)


@pytest.mark.parametrize("T,K,N", [(1 << 20, 32, 8), (1 << 20, 160, 40), (2, 1 << 20, 3), (40, 1 << 20, 70), (2, 32, 1 << 20), (60, 256, 1 << 20)])
def test_mx_product(T, K, N):
    print(f"case: {T}x{K}x{N}", flush=True)
    x, w, bias = whole(T, K, seed=8), whole(N, K, seed=9), whole(N, seed=10)
    (xq, xs), (wq, ws) = pack(x, "fit"), pack(w, "fit")
    d = moe.make_mx_linear_desc(wq, ws, bias=bias)
    out = torch.full((T + 1, N), 99.0, device="cuda")
    moe.mx_linear(d, xq, xs, T, None, out, moe.OUT_F32, moe.mx_linear_workspace(d, T))
    torch.cuda.synchronize()
    assert torch.equal(out[:T], (x.double() @ w.double().t() + bias.double()).float()) and (out[T] == 99.0).all()


def test_rows_made_and_read_back():
    x = torch.randn(3, 1 << 20, device="cuda").bfloat16()
    c, s = torch.empty(3, 1 << 19, dtype=torch.uint8, device="cuda"), torch.empty(3, 1 << 15, dtype=torch.uint8, device="cuda")
    moe.mx_quantize(x, 3, c, s)
    out = torch.empty_like(x)
    moe.mx_dequantize(c, s, 3, out)
    torch.cuda.synchronize()
    want = pack(x)
    assert torch.equal(c, want[0]) and torch.equal(s, want[1]) and torch.equal(out, unpack(*want).bfloat16())
