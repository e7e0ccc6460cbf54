"""moe_linear on one token that lies in a wider tensor: a single row has no second one, so its distance is not looked at."""
import ctypes

import pytest

import quantized_expert_gemv_sigmoid_amd as moe
from test_abi_gate_linear import FAKE, L, call_linear, linear_desc  # noqa: F401 (L: a fixture)

torch = pytest.importorskip("torch")

FAR = (1 << 22) + 8


def test_distances_of_one_row_are_not_refused(L):  # noqa: F811
    d = linear_desc()
    need = L.moe_linear_workspace_bytes(ctypes.byref(d), 1)
    short = dict(ws=(FAKE * 16, need - 1))   # (refused for its workspace alone: nothing is launched)
    for far in (dict(ldx=FAR), dict(ldo=FAR), dict(res=FAKE, ldr=FAR), dict(ldx=1 << 40, ldo=1 << 40, res=FAKE, ldr=1 << 40)):
        assert call_linear(L, d, T=1, **far, **short) == moe.EWORKSPACE
        assert call_linear(L, d, T=2, **far, **short) == moe.EUNSUPPORTED
    for kw in (dict(ldx=639), dict(ldo=511), dict(res=FAKE, ldr=511)):
        assert call_linear(L, d, T=1, **kw) == moe.EINVAL


def test_binding_gives_one_row_no_distance():
    wide = torch.empty(1, 3, 8)
    assert moe._rows(wide[:, -1], 1, 8, "x") == 8
    assert moe._rows(torch.empty(2, 24)[:, :8], 1, 8, "x") == 8
    assert moe._rows(torch.empty(2, 24)[:, :8], 2, 8, "x") == 24


@pytest.mark.gpu
@pytest.mark.parametrize("S", [3, 700])
@pytest.mark.parametrize("K", [7168, 7165])
@pytest.mark.parametrize("mode", [moe.OUT_HALF, moe.OUT_F32])
def test_last_token_of_a_prompt(S, K, mode):
    """x, residual and output are the last rows of prompts of one sequence: [1, S, ..][:, -1]."""
    print(f"case: S={S} K={K} mode={mode}", flush=True)
    N = 6008
    g = torch.Generator(device="cuda").manual_seed(S)
    hidden = torch.randint(-3, 4, (1, S, K), device="cuda", generator=g).bfloat16()
    w = torch.randint(-3, 4, (N, K), device="cuda", generator=g).bfloat16()
    stream = torch.randint(-9, 9, (1, S, N), device="cuda", generator=g).to(torch.float32 if mode == moe.OUT_F32 else torch.bfloat16)
    x, o = hidden[:, -1], stream[:, -1]
    assert x.stride(0) == S * K and (S < 700 or x.stride(0) > 1 << 22)
    want = (x.double() @ w.double().t() + o.double()).to(stream.dtype)   # (whole numbers: exact in fp32)
    before = stream[:, :-1].clone()
    d = moe.make_linear_desc(w, residual_type=moe.F32 if mode == moe.OUT_F32 else None)
    moe.linear(d, x, 1, o if mode == moe.OUT_HALF else None, o if mode == moe.OUT_F32 else None, mode,
               moe.linear_workspace(d, 1), residual=o)
    torch.cuda.synchronize()
    assert torch.equal(o, want) and torch.equal(stream[:, :-1], before)


@pytest.mark.gpu
def test_last_logits_of_a_prompt():
    logits = torch.randn(1, 5000, 896, device="cuda")
    d = moe.make_gate_desc(896, 16)
    out = [(torch.empty(1, 16, dtype=torch.int32, device="cuda"), torch.empty(1, 16, device="cuda")) for _ in range(2)]
    for (ids, w), l in zip(out, (logits[:, -1], logits[:, -1].contiguous())):
        moe.gate(d, l, 1, ids, w)
    torch.cuda.synchronize()
    assert torch.equal(out[0][0], out[1][0]) and torch.equal(out[0][1], out[1][1])
