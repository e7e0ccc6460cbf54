"""Every kernel of moe_grouped_linear over rows long enough for its ring: more than twice the ring's stages and a last one that is not
full, so that every slot is filled anew several times while rows are gathered, and rows without a source stay zeros to the end.

The sizes are found by asking the rule: the least work among drawn ones that each kernel is taken for.  Plain products are of whole
numbers and have to be equal bit for bit.
"""
import functools
import math
import random

import pytest

import quantized_expert_gemv_sigmoid_amd as moe
from test_abi_gate_linear import L  # noqa: F401 (a fixture)
from test_mx_grouped_kernels import ANY, grouped_taken

torch = pytest.importorskip("torch")

TILES = (moe.LINEAR_TILE64X32, moe.LINEAR_TILE64X64, moe.LINEAR_TILE128X64, moe.LINEAR_TILE128X128, moe.LINEAR_TILE256X128)
# stages a ring holds at most: of 64 values, or 256 MXFP4 codes
RING = 6
N_IN = {"16": 840, "odd": 871, "mx": 3200}
CASES = [(form, kind, gated) for form, kinds in (("16", TILES), ("odd", ANY), ("mx", TILES)) for kind in kinds for gated in (0, 1)]


@functools.lru_cache(None)
def sizes(form):
    """{(kernel, gated): (groups, rows, n_out)}"""
    lib, rng, K, best = moe.lib(), random.Random(11), N_IN[form], {}
    for _ in range(6000):
        E, R, N = (int(round(math.exp(rng.uniform(math.log(a), math.log(b))))) for a, b in ((3, 60), (40, 6000), (30, 1500)))
        gated = rng.randrange(2)
        cost = E * N * (1 + gated) * K + R * K + 8 * R * N
        kind = grouped_taken(lib, form == "mx", E, R, K, N, gated, form == "odd")
        if cost < best.get((kind, gated), (1e30,))[0]:
            best[kind, gated] = cost, (E, R, N)
    return {k: v[1] for k, v in best.items()}


def test_sizes_reach_every_kernel(L):  # noqa: F811
    for form, kind, gated in CASES:
        E, R, N = sizes(form)[kind, gated]
        assert E * N * (1 + gated) * N_IN[form] < 2 ** 27, (form, kind, gated, E, R, N)
    for form, K in N_IN.items():
        stage = 256 if form == "mx" else 64
        assert K > 2 * RING * stage and K % stage != 0


@pytest.mark.gpu
@pytest.mark.parametrize("gather", [0, 1])
@pytest.mark.parametrize("form,kind,gated", CASES)
def test_each_kernel(form, kind, gated, gather):
    import test_gpu_grouped as t
    E, R, N = sizes(form)[kind, gated]
    K, X = N_IN[form], R // 2 + 3
    print(f"case: {form} kernel {kind} gated {gated} gather {gather}: {E} groups, {R}x{K}x{N}", flush=True)
    s = t.make(E, R, K, N, torch.float16 if R % 2 else torch.bfloat16, act="situ_glu" if gated else "none", bias=torch.float32,
               mx=form == "mx", gather=X if gather else 0, whole=not gated, seed=R + gather)
    if gather:
        s["rows"][::13] = -1
        s["rows"][1::17] = X
        s["rows"][2::19] = X - 1
    assert moe.grouped_path_for(t.descriptor(s), s["x"], R, rows=s["rows"]) == kind
    h, f = t.check(s)
    if not gated:
        a, b = t.covered(s)
        v = t.reference(s)[0][a:b]
        assert v.abs().max() < 2 ** 24
        assert torch.equal(f[a:b].double(), v) and torch.equal(h[a:b], f[a:b].to(s["type"]))
