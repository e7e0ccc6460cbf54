"""moe_linear's SiTU-GLU with betas far from the layer's: a beta so large that its tanh is the identity, products of both past
fp32's range, and a small one.  The bound is the product's (test_gpu_linear.reference), which holds for any betas."""
import pytest

import quantized_expert_gemv_sigmoid_amd as moe
import test_gpu_linear as plain
from test_gpu_linear import check, make

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.mark.parametrize("T,K,N", [(1, 256, 192), (24, 256, 192), (150, 264, 200), (90, 257, 131), (40, 4104, 1000), (2304, 136, 2048)])
@pytest.mark.parametrize("b1,b2", [(1e20, 1e20), (1e19, 3e38), (3e38, 3e38), (1e30, 1e-3), (1e-3, 1e30), (2.5, 1e38)])
def test_betas(monkeypatch, T, K, N, b1, b2):
    print(f"case: T={T} K={K} N={N} betas {b1} {b2}", flush=True)
    monkeypatch.setattr(plain, "B1", b1)
    monkeypatch.setattr(plain, "B2", b2)
    s = make(T, K, N, torch.bfloat16, act="situ_glu", bias=torch.float32, residual=torch.float32, seed=T)
    d = moe.make_linear_desc(s["w"], w_up=s["w_up"], bias=s["bias"], bias_up=s["bias_up"], act=moe.LINEAR_SITU_GLU,
                             situ_b1=b1, situ_b2=b2, residual_type=moe.F32)
    f = torch.empty(T, N, device="cuda")
    moe.linear(d, s["x"], T, None, f, moe.OUT_F32, moe.linear_workspace(d, T), residual=s["residual"])
    torch.cuda.synchronize()
    check(s, f, torch.float32)
