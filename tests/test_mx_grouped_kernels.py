"""Every kernel of moe_mx_linear (with every split of n_in) and of moe_grouped_linear, plain and gated, against the formula.

The lists name the kernel of each size; the rules are asked that they still take them, and over drawn sizes that they take
no other.  Plain products are of whole numbers, so that outputs have to be equal bit for bit.
"""
import ctypes
import math
import random

import pytest

import quantized_expert_gemv_sigmoid_amd as moe
from test_abi import FAKE
from test_abi_gate_linear import L  # noqa: F401 (a fixture)
from test_abi_mx_grouped import GROUPED as GROUPED_DESC, GROUPED_MX as GROUPED_MX_DESC, MX as MX_DESC, filled

torch = pytest.importorskip("torch")

# (kernel, parts of n_in, gated, T, n_in, n_out)
MX = [
    (0, 1, 0, 2, 32, 5), (0, 1, 1, 2, 32, 5), (1, 1, 0, 2170, 32, 5), (1, 1, 1, 9, 32, 1080), (2, 1, 0, 5702, 32, 5),
    (2, 1, 1, 17, 32, 1416), (3, 1, 0, 2, 256, 8806), (3, 1, 1, 2, 256, 4481), (3, 2, 0, 35, 28704, 4431),
    (3, 2, 1, 51, 32256, 2229), (3, 4, 0, 38, 44096, 2274), (3, 4, 1, 34, 38112, 1240), (3, 8, 0, 2, 42848, 6),
    (3, 8, 1, 2, 47584, 5), (4, 1, 0, 5281, 32, 66), (4, 1, 1, 34, 32, 5343), (4, 2, 0, 39, 44128, 5859),
    (4, 2, 1, 4239, 26784, 33), (4, 4, 0, 5392, 18944, 34), (4, 4, 1, 36, 36480, 1473), (4, 8, 0, 2029, 30656, 35),
    (4, 8, 1, 2682, 38432, 9), (5, 1, 0, 67, 32, 12870), (5, 1, 1, 33, 128, 12880), (5, 2, 0, 70, 34880, 7019),
    (5, 2, 1, 81, 44224, 3482), (5, 4, 0, 67, 18080, 3263), (5, 4, 1, 137, 19808, 1047), (5, 8, 0, 73, 29856, 1975),
    (5, 8, 1, 67, 25280, 970), (6, 1, 0, 193, 32, 9555), (6, 1, 1, 67, 192, 9654), (6, 2, 0, 373, 29728, 4273),
    (6, 2, 1, 2605, 30112, 294), (6, 4, 0, 5427, 20384, 72), (6, 4, 1, 4976, 25024, 36), (6, 8, 0, 2975, 28128, 69),
    (6, 8, 1, 3276, 20256, 34), (10, 1, 0, 1160, 64, 10277), (10, 1, 1, 403, 224, 12985),
    (10, 2, 0, 4282, 31648, 1310), (10, 2, 1, 776, 34624, 3773), (10, 4, 0, 139, 27936, 13616),
    (10, 4, 1, 144, 38624, 7368), (10, 8, 0, 163, 43136, 6997), (10, 8, 1, 3518, 45696, 165),
    (11, 1, 0, 259, 32, 13306), (11, 1, 1, 130, 32, 11157), (11, 2, 0, 2323, 10560, 1767),
    (11, 2, 1, 146, 18144, 9400), (11, 4, 0, 131, 34752, 8307), (11, 4, 1, 135, 29152, 3951),
    (11, 8, 0, 3325, 44128, 130), (11, 8, 1, 134, 38848, 1950),
]
# (MXFP4, kernel, gated, groups, rows, n_in, n_out)
GROUPED = [
    (0, 3, 0, 2, 4, 40, 9), (0, 3, 1, 2, 4, 40, 9), (0, 4, 0, 9, 518, 64, 11), (0, 4, 1, 5, 482, 48, 9),
    (0, 5, 0, 173, 1461, 56, 75), (0, 5, 1, 261, 636, 64, 37), (0, 6, 0, 13, 2581, 48, 81), (0, 6, 1, 4, 4417, 40, 40),
    (0, 7, 0, 2, 6, 103, 18), (0, 7, 1, 2, 6, 68, 15), (0, 8, 0, 4, 4008, 55, 9), (0, 8, 1, 34, 6608, 45, 10),
    (0, 9, 0, 24, 4046, 54, 80), (0, 9, 1, 7, 3335, 41, 51), (0, 11, 0, 23, 48, 40, 642), (0, 11, 1, 37, 74, 56, 230),
    (1, 3, 0, 2, 6, 256, 9), (1, 3, 1, 2, 4, 256, 25), (1, 4, 0, 3, 452, 256, 10), (1, 4, 1, 3, 498, 256, 15),
    (1, 5, 0, 276, 786, 256, 65), (1, 5, 1, 265, 615, 384, 44), (1, 6, 0, 2, 3189, 256, 70),
    (1, 6, 1, 3, 2287, 256, 34), (1, 11, 0, 17, 35, 256, 1166), (1, 11, 1, 6, 12, 256, 1252),
]
ANY = (moe.LINEAR_ANY64X32, moe.LINEAR_ANY64X64, moe.LINEAR_ANY128X128)


def mx_taken(lib, T, K, N, gated):
    more = dict(act=moe.LINEAR_SWIGLU, w_up=FAKE, w_up_s=FAKE) if gated else {}
    d = filled(moe.MxLinearDesc, MX_DESC, dict(n_in=K, n_out=N, ldw=K // 2, ldw_s=K // 32, **more))
    r = lib.moe_mx_linear_path_for(ctypes.byref(d), T)
    assert r > 0
    return r % 256, r // 256


def grouped_taken(lib, mx, E, R, K, N, gated, unaligned):
    more = dict(act=moe.LINEAR_SWIGLU, w_up=FAKE, w_up_s=FAKE if mx else None) if gated else {}
    ld = K // 2 if mx else K
    scales = dict(ldw_s=K // 32, group_w_s=K // 32 * N) if mx else {}
    d = filled(moe.GroupedDesc, GROUPED_MX_DESC if mx else GROUPED_DESC,
               dict(n_groups=E, n_in=K, n_out=N, ldw=ld, group_w=ld * N, **scales, **more))
    r = lib.moe_grouped_path_for(ctypes.byref(d), FAKE + 2 * unaligned, ld, R)
    assert r // 256 == 1
    return r % 256


def test_cases_take_their_kernels(L):  # noqa: F811
    for kind, parts, gated, T, K, N in MX:
        assert mx_taken(L, T, K, N, gated) == (kind, parts), (T, K, N, gated)
    for mx, kind, gated, E, R, K, N in GROUPED:
        assert grouped_taken(L, mx, E, R, K, N, gated, 0) == kind, (mx, E, R, K, N, gated)


def test_the_rules_take_no_other(L):  # noqa: F811
    rng, found, grouped = random.Random(7), set(), set()
    for _ in range(20000):
        T, K, N = (int(round(math.exp(rng.uniform(0.0, math.log(m))))) for m in (6000, 50000, 14000))
        gated = rng.random() < 0.5
        found.add(mx_taken(L, T, max(32, K // 32 * 32), N, gated) + (int(gated),))
        E, R, K, N = (int(round(math.exp(rng.uniform(0.0, math.log(m))))) for m in (1024, 100000, 8000, 8000))
        mx, unaligned = rng.random() < 0.5, rng.random() < 0.4
        K = max(128, K // 128 * 128) if mx else K if unaligned else max(8, K // 8 * 8)
        grouped.add((int(mx), grouped_taken(L, mx, E, R, K, N, gated, 0), int(gated)))
    assert found <= {c[:3] for c in MX}
    assert grouped <= {c[:3] for c in GROUPED}
    # every kernel that each has, both ways
    tiles = {moe.LINEAR_TILE64X32, moe.LINEAR_TILE64X64, moe.LINEAR_TILE128X64, moe.LINEAR_TILE128X128, moe.LINEAR_TILE256X128}
    few = {moe.LINEAR_ROWS16X8, moe.LINEAR_ROWS16X16, moe.LINEAR_ROWS16X32, moe.LINEAR_TILE256X256}
    assert {(c[0], c[2]) for c in MX} == {(k, g) for k in tiles | few for g in (0, 1)}
    assert {c[:3] for c in GROUPED} == ({(m, k, g) for k in tiles for m in (0, 1) for g in (0, 1)} |
                                        {(0, k, g) for k in ANY for g in (0, 1)})


def test_path_for_refused(L):  # noqa: F811
    d = filled(moe.MxLinearDesc, MX_DESC, {})
    assert L.moe_mx_linear_path_for(ctypes.byref(d), 0) == moe.EINVAL
    assert L.moe_mx_linear_path_for(ctypes.byref(d), (1 << 20) + 1) == moe.EUNSUPPORTED
    assert L.moe_mx_linear_path_for(None, 3) == moe.EINVAL
    d = filled(moe.GroupedDesc, GROUPED_DESC, {})
    for x, ldx, R, status in ((FAKE, 640, 0, moe.EINVAL), (None, 640, 3, moe.EINVAL), (FAKE, 639, 3, moe.EINVAL), (FAKE + 1, 640, 3, moe.EINVAL),
                              (FAKE, 640, (1 << 24) + 1, moe.EUNSUPPORTED), (FAKE, (1 << 22) + 1, 3, moe.EUNSUPPORTED)):
        assert L.moe_grouped_path_for(ctypes.byref(d), x, ldx, R) == status
    assert L.moe_grouped_path_for(None, FAKE, 640, 3) == moe.EINVAL


@pytest.mark.gpu
@pytest.mark.parametrize("case", MX, ids=str)
def test_each_mx_kernel(case):
    import test_gpu_mx_linear as t
    kind, parts, gated, T, K, N = case
    print(f"case: {case}", flush=True)
    s = t.make(T, K, N, torch.float16 if T % 2 else torch.bfloat16, act="swiglu" if gated else "none", bias=torch.float32,
               residual=torch.float32, whole=not gated, seed=T + N)
    assert moe.mx_linear_path_for(t.descriptor(s), T) == (kind, parts)
    h, f = t.call(s)
    v, e = t.reference(s)
    if gated:
        t.close(f, v, e)
        t.close(h, v, e)
    else:
        assert v.abs().max() < 2 ** 24
        assert torch.equal(f.double(), v) and torch.equal(h, v.float().to(s["type"]))


@pytest.mark.gpu
@pytest.mark.parametrize("case", GROUPED, ids=str)
@pytest.mark.parametrize("gather", [0, 1])
def test_each_grouped_kernel(case, gather):
    import test_gpu_grouped as t
    mx, kind, gated, E, R, K, N = case
    print(f"case: {case} gather {gather}", flush=True)
    s = t.make(E, R, K, N, torch.float16 if R % 2 else torch.bfloat16, act="situ_glu" if gated else "none", bias=torch.float32,
               mx=bool(mx), gather=R // 2 + 1 if gather else 0, whole=not gated and not mx, seed=R)
    if gather:
        s["rows"][::13] = -1
    assert moe.grouped_path_for(t.descriptor(s), s["x"], R) == kind
    h, f = t.check(s)
    if not gated and not mx:
        a, b = t.covered(s)
        assert torch.equal(f[a:b].double(), t.reference(s)[0][a:b])
