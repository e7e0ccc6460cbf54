"""Rows and matrices whose offsets pass 32 bits, at the largest row distances that the calls take, against the formulas in 64 bits
(bounds as in test_gpu_grouped.py and test_gpu_mx_linear.py)."""
import pytest

import quantized_expert_gemv_sigmoid_amd as moe
from mx_support import pack, unpack
from test_gpu_grouped import make as make_grouped, descriptor as grouped_descriptor, reference as grouped_reference
from test_gpu_linear import HALF
from test_gpu_mx_linear import close, descriptor, make, reference

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

LD = 1 << 22   # elements between rows, the most


@pytest.fixture(scope="module")
def space():
    """Views of rows `ld` apart with another tensor's values, each in memory of its own."""
    if torch.cuda.mem_get_info()[0] < 96 << 30:
        pytest.skip("needs 96 GiB of device memory")

    def far(t, *strides):
        size = sum((n - 1) * s for n, s in zip(t.shape, (*strides, 1))) + 1
        v = torch.empty(size, dtype=t.dtype, device="cuda").as_strided(t.shape, (*strides, 1))
        v.copy_(t)
        return v

    yield far
    torch.cuda.empty_cache()


def sentinels(far, R, N, dtype):
    return far(torch.full((R, N), 99.0, device="cuda").to(dtype), LD)


@pytest.mark.parametrize("K,N,mx", [(128, 64, False), (129, 65, False), (512, 4096, False), (128, 64, True), (512, 4096, True)])
@pytest.mark.parametrize("gather", [0, 256])
def test_groups(space, K, N, mx, gather):
    E, R = 3, 600
    s = make_grouped(E, R, K, N, gather=gather, kind="even", mx=mx, seed=K + gather)
    cols = s["w"].shape[2]
    apart = (1 << 31) + 64   # between matrices: elements
    s["w"] = space(s["w"], apart, cols + 16 if mx else cols + 8 if K % 8 == 0 else cols)
    s["x"] = space(s["x"], 2 * LD if mx else LD)
    if mx:
        s["w_s"] = space(s["w_s"], apart, s["w_s"].shape[2] + 4)
        s["x_s"] = space(s["x_s"], LD)
    if gather:
        s["rows"][::7] = -1
        s["rows"][1::7] = gather - 1
    d = grouped_descriptor(s)
    h, f = sentinels(space, R, N, s["type"]), sentinels(space, R, N, torch.float32)
    moe.grouped_linear(d, s["x"], s["offsets"], R - 3, h, f, moe.OUT_BOTH, rows=None if s["rows"] is None else s["rows"][:R - 3], x_s=s["x_s"])
    torch.cuda.synchronize()
    v, e = grouped_reference(s)
    close(f[:R - 3], v[:R - 3], e[:R - 3])
    close(h[:R - 3], v[:R - 3], e[:R - 3])
    assert (h[R - 3:] == 99.0).all() and (f[R - 3:] == 99.0).all()


@pytest.mark.parametrize("T,K,N", [(600, 256, 520), (600, 160, 520), (1100, 512, 4096), (9, 1024, 600)])
def test_mx_product(space, T, K, N):
    s = make(T, K, N, residual=torch.float32, seed=T + K)
    s["residual"] = space(s["residual"], LD)
    for n in ("x", "w"):
        codes, scales = s[n]
        s[n] = space(codes, 2 * LD), space(scales, LD)
    d = descriptor(s)
    f = sentinels(space, T, N, torch.float32)
    moe.mx_linear(d, *s["x"], T, None, f, moe.OUT_F32, moe.mx_linear_workspace(d, T), residual=s["residual"])
    torch.cuda.synchronize()
    v, e = reference(s)
    close(f, v, e)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_rows_made_and_read_back(space, dtype):
    x = torch.randn(700, 1000, device="cuda").to(dtype)
    c, s = pack(x)
    codes, scales = space(torch.zeros_like(c), 2 * LD), space(torch.zeros_like(s), 2 * LD)
    moe.mx_quantize(space(x, 2 * LD), 700, codes, scales)
    torch.cuda.synchronize()
    assert torch.equal(codes, c) and torch.equal(scales, s)
    out = space(torch.zeros_like(x), 2 * LD)
    moe.mx_dequantize(codes, scales, 700, out)
    torch.cuda.synchronize()
    assert torch.equal(out, unpack(c, s)[:, :1000].to(dtype))


def test_rows_of_several_launches():
    """2^30 quarters of blocks, four a row of one value, are one launch's."""
    T = (1 << 28) + 1000
    x = torch.randint(-6, 7, (T, 1), device="cuda", dtype=torch.int8).bfloat16()
    codes, scales = torch.empty(T, 16, dtype=torch.uint8, device="cuda"), torch.empty(T, 1, dtype=torch.uint8, device="cuda")
    out = torch.empty_like(x)
    moe.mx_quantize(x, T, codes, scales)
    moe.mx_dequantize(codes, scales, T, out)
    torch.cuda.synchronize()
    for a in (0, (1 << 26) - 50, (1 << 28) - 500, T - 500):
        c, s = pack(x[a:a + 500])
        assert torch.equal(codes[a:a + 500], c) and torch.equal(scales[a:a + 500], s)
    assert torch.equal(out, torch.where(x.abs() == 5, x.sign() * 4, x))   # (5 lies between 4 and 6: the even code's)


@pytest.mark.parametrize("yt", [torch.bfloat16, torch.float32])
def test_combine(space, yt):
    R, T, k, n = 1500, 300, 4, 72
    y = space(torch.randn(R, n, device="cuda").to(yt), LD)
    places = torch.randint(R - 600, R, (T, k), device="cuda", dtype=torch.int32)
    w = torch.randn(T, k, device="cuda")
    res = space(torch.randn(T, n, device="cuda"), LD)
    out = sentinels(space, T + 1, n, torch.float32)
    moe.combine(y, R, places, w, T, out, residual=res)
    torch.cuda.synchronize()
    terms = w.double()[..., None] * y[places.long()].double()
    v = terms.sum(1) + res.double()
    e = (k + 1) * 2.0 ** -23 * terms.abs().sum(1) + 2.0 ** -23 * v.abs()
    bound = e + HALF[torch.float32] * (v.abs() + e) + 1e-37
    assert ((out[:T].double() - v).abs() <= bound).all() and (out[T:] == 99.0).all()
