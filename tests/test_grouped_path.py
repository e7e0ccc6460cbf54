"""moe_grouped_path_for names the kernel of the call it is asked about where that call has one row: a gathered row comes from among
others, and their distance decides whether it is 16-byte aligned (no GPU needed: nothing is launched)."""
import ctypes

import pytest

import quantized_expert_gemv_sigmoid_amd as moe
from test_abi import FAKE
from test_abi_gate_linear import L  # noqa: F401 (a fixture)
from test_abi_mx_grouped import GROUPED, GROUPED_MX, filled

torch = pytest.importorskip("torch")
ANY = (moe.LINEAR_ANY64X32, moe.LINEAR_ANY64X64, moe.LINEAR_ANY128X128)


@pytest.mark.parametrize("R", [1, 2, 50])
def test_the_distance_of_rows_counts(L, R):  # noqa: F811
    d = filled(moe.GroupedDesc, GROUPED, {})

    def path(ldx, x=FAKE, desc=d):
        r = L.moe_grouped_path_for(ctypes.byref(desc), x, ldx, R)
        return r % 256 if r >= 0 else r

    assert path(640) not in ANY and path(648) not in ANY
    assert path(645) in ANY and path(640, FAKE + 2) in ANY
    m = filled(moe.GroupedDesc, GROUPED_MX, {})
    assert path(320, desc=m) == path(336, desc=m) not in ANY


def test_one_row_of_one(L):  # noqa: F811
    """One row has no distance: none that the call takes is refused."""
    d, m = filled(moe.GroupedDesc, GROUPED, {}), filled(moe.GroupedDesc, GROUPED_MX, {})
    for desc in (d, m):
        for ldx in (0, -7, 1):
            r = L.moe_grouped_path_for(ctypes.byref(desc), FAKE, ldx, 1)
            assert r >= 256 and r % 256 not in ANY


def test_binding():
    d = moe.make_grouped_desc(torch.empty(3, 8, 16, dtype=torch.bfloat16))
    wide = torch.empty(5, 21, dtype=torch.bfloat16)
    x, rows = wide[:, :16], torch.zeros(9, dtype=torch.int32)
    assert x.data_ptr() % 16 == 0
    # the row distance is x's where rows are gathered, or where there are several
    assert moe.grouped_path_for(d, x, 1, rows=rows) in ANY
    assert moe.grouped_path_for(d, x, 9, rows=rows) in ANY
    assert moe.grouped_path_for(d, x, 2) in ANY
    # the first row alone, and rows gathered from one, have none
    assert moe.grouped_path_for(d, x, 1) not in ANY
    assert moe.grouped_path_for(d, x[:1], 9, rows=rows) not in ANY
    assert moe.grouped_path_for(d, x[:1], 1, rows=rows) not in ANY


@pytest.mark.gpu
@pytest.mark.parametrize("row", [0, 3, 4, -1, 5])
def test_a_gathered_row_of_several(row):
    import test_gpu_grouped as t
    s = t.make(3, 1, 640, 40, gather=5, padx=5, whole=True, bias=torch.float32, seed=3)
    s["rows"][0] = row
    assert moe.grouped_path_for(t.descriptor(s), s["x"], 1, rows=s["rows"]) in ANY
    f = t.call(s)[1]
    a, b = t.covered(s)
    assert b - a == 1 and torch.equal(f[a:b].double(), t.reference(s)[0][a:b])
