"""The binding refuses a call whose descriptor was made of tensors of another device than the call's: a kernel would read
their addresses on the wrong one (no GPU needed)."""
import pytest

import quantized_expert_gemv_sigmoid_amd as moe

torch = pytest.importorskip("torch")


def half(*shape, device="cpu"):
    return torch.empty(*shape, dtype=torch.bfloat16, device=device)


def test_gate_bias_of_another_device():
    d = moe.make_gate_desc(8, 2, bias=torch.empty(8))
    ids, w = torch.empty(3, 2, dtype=torch.int32, device="meta"), torch.empty(3, 2, device="meta")
    with pytest.raises(moe.MoeError, match="tensors on cpu and meta"):
        moe.gate(d, torch.empty(3, 8, device="meta"), 3, ids, w)
    layer = moe.LayerDesc()
    layer.n_experts, layer.top_k, layer.d_model = 8, 2, 256
    with pytest.raises(moe.MoeError, match="tensors on cpu and meta"):
        moe.route_gated(layer, d, half(3, 256, device="meta"), 3, ids, w, None, (256, 1 << 30))


def test_product_weights_of_another_device():
    d = moe.make_linear_desc(half(5, 8))
    with pytest.raises(moe.MoeError, match="tensors on cpu and meta"):
        moe.linear(d, half(3, 8, device="meta"), 3, half(3, 5, device="meta"), None, moe.OUT_HALF, (256, 1 << 30))
    d = moe.make_linear_desc(half(5, 8, device="meta"))
    with pytest.raises(moe.MoeError, match="tensors on meta and cpu"):
        moe.linear(d, half(3, 8), 3, half(3, 5), None, moe.OUT_HALF, (256, 1 << 30))


def test_descriptors_filled_by_hand_are_taken_as_they_are():
    d = moe.GateDesc()
    d.n_experts, d.top_k, d.bias = 8, 2, 0x10000
    assert d.device is None
    with pytest.raises(moe.MoeError, match="tensors on cpu: "):   # (the device of the call's own tensors)
        moe.gate(d, torch.empty(3, 8), 3, torch.empty(3, 2, dtype=torch.int32), torch.empty(3, 2))
