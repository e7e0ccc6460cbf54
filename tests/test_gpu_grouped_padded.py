"""Products of groups of MXFP4 rows whose width is no multiple of 128: moe_mx_quantize writes them into wider zeroed rows (row distances),
and the blocks of zeros behind them, codes 0 and scale byte 0, add nothing: within the bounds of the formula at the rows' own width."""
import pytest

import quantized_expert_gemv_sigmoid_amd as moe
from mx_support import pack, unpack
from test_gpu_mx_linear import close, finish, product

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def quantized(x, wide):
    """(codes, scales) of rows [.., n] in zeroed rows of `wide` values."""
    rows, n = x.view(-1, x.shape[-1]), x.shape[-1]
    b = (n + 31) // 32
    c = torch.zeros(rows.shape[0], wide // 2, dtype=torch.uint8, device="cuda")
    s = torch.zeros(rows.shape[0], wide // 32, dtype=torch.uint8, device="cuda")
    moe.mx_quantize(rows, rows.shape[0], c[:, :16 * b], s[:, :b], rule=moe.MX_FIT)
    return c.view(*x.shape[:-1], -1), s.view(*x.shape[:-1], -1)


@pytest.mark.parametrize("K", [32, 100, 160, 2880])
@pytest.mark.parametrize("R", [5, 300, 2000])
@pytest.mark.parametrize("gated", [0, 1])
def test_padded_rows(K, R, gated):
    print(f"case: {R}x{K} gated {gated}", flush=True)
    g = torch.Generator(device="cuda").manual_seed(K + R)
    E, N, wide = 3, 200, (K + 127) // 128 * 128
    x = torch.randn(R, K, device="cuda", generator=g).bfloat16()
    ws = [(torch.randn(E, N, K, device="cuda", generator=g) * K ** -0.5).bfloat16() for _ in range(1 + gated)]
    xq, xs = quantized(x, wide)
    q = [quantized(w, wide) for w in ws]
    up = dict(w_up=q[1][0], w_up_s=q[1][1], act=moe.LINEAR_SWIGLU) if gated else {}
    offsets = torch.tensor([0, R // 3, R // 3, R], dtype=torch.int32, device="cuda")
    out = torch.empty(R, N, device="cuda")
    moe.grouped_linear(moe.make_grouped_desc(q[0][0], w_s=q[0][1], **up), xq, offsets, R, None, out, moe.OUT_F32, x_s=xs)
    torch.cuda.synchronize()
    xv, wv = unpack(*pack(x, "fit"))[:, :K], [unpack(*pack(w, "fit"))[..., :K] for w in ws]
    for e in range(E):
        a, b = offsets[e].item(), offsets[e + 1].item()
        if a == b:
            continue
        v, ev = product(xv[a:b], wv[0][e], None)
        u, eu = product(xv[a:b], wv[1][e], None) if gated else (None, None)
        close(out[a:b], *finish("swiglu" if gated else "none", v, ev, u, eu, None))
