"""Tables of choices, [tokens][choices], of another width than the call's are refused: read or written as rows of its width they would
be other tokens' (no GPU needed: the tensors are the host's, which is refused last)."""
import pytest

import quantized_expert_gemv_sigmoid_amd as moe

torch = pytest.importorskip("torch")


def i32(*shape):
    return torch.zeros(*shape, dtype=torch.int32)


def refused(match, f, *a, **kw):
    with pytest.raises(moe.MoeError, match=match):
        f(*a, **kw)


@pytest.mark.parametrize("width", [1, 3, 8])
def test_weights_of_another_width(width):
    y, places, out = torch.zeros(20, 16), i32(5, 2), torch.zeros(5, 16)
    refused("weights", moe.combine, y, 20, places, torch.zeros(12, width), 5, out)


@pytest.mark.parametrize("shape", [(5, 2), (9, 2), (10,), (12,)])
def test_weights_of_the_width(shape):
    refused("tensors on cpu", moe.combine, torch.zeros(20, 16), 20, i32(5, 2), torch.zeros(*shape), 5, torch.zeros(5, 16))


@pytest.mark.parametrize("width", [1, 3, 8])
def test_places_of_another_width(width):
    refused("places", moe.group, i32(5, 2), 5, 4, i32(5), i32(10), i32(12, width), (256, 1 << 20))


@pytest.mark.parametrize("shape", [(5, 2), (9, 2), (10,), (12,)])
def test_places_of_the_width(shape):
    refused("tensors on cpu", moe.group, i32(5, 2), 5, 4, i32(5), i32(10), i32(*shape), (256, 1 << 20))


def test_one_token():
    """One row of a wider table is its first choices."""
    refused("tensors on cpu", moe.combine, torch.zeros(20, 16), 20, i32(1, 2), torch.zeros(1, 8), 1, torch.zeros(1, 16))
    refused("tensors on cpu", moe.group, i32(1, 2), 1, 4, i32(5), i32(2), i32(1, 8), (256, 1 << 20))
