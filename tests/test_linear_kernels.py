"""Every kernel of moe_linear, whole and with every split of K that the rule gives it, plain and gated, against the formula.

`CASES` names the kernel and split of each size; the rule is asked (moe_linear_path_for) that it still takes them, and over
drawn sizes that it takes no other.  Inputs are whole numbers, so that outputs have to be equal bit for bit.  The large
tiles' whole-tile epilogue is run with every activation, residual and output.
"""
import ctypes
import math
import random

import pytest

import quantized_expert_gemv_sigmoid_amd as moe
from test_abi_gate_linear import FAKE, L, linear_desc  # noqa: F401 (L: a fixture)
from test_gpu_linear import B1, B2, GATED, PLAIN, check, make, reference

torch = pytest.importorskip("torch")

# (kernel, parts of K, gated, T, K, N)
CASES = [
    (0, 1, 0, 1, 8, 1), (0, 1, 1, 1, 8, 1), (1, 1, 0, 2173, 8, 1), (1, 1, 1, 211, 8, 73), (2, 1, 0, 5731, 8, 1),
    (2, 1, 1, 18, 8, 1585), (3, 1, 0, 1, 8, 13199), (3, 1, 1, 1, 8, 6629), (3, 2, 0, 35, 5600, 4557),
    (3, 2, 1, 43, 5920, 2008), (3, 4, 0, 39, 12784, 1882), (3, 4, 1, 53, 11536, 958), (3, 8, 0, 1, 10624, 1),
    (3, 8, 1, 1, 11472, 1), (4, 1, 0, 5574, 8, 65), (4, 1, 1, 33, 8, 5496), (4, 2, 0, 585, 7176, 796),
    (4, 2, 1, 586, 6576, 385), (4, 4, 0, 336, 4040, 765), (4, 4, 1, 299, 4192, 403), (4, 8, 0, 419, 8624, 180),
    (4, 8, 1, 147, 7968, 306), (5, 1, 0, 66, 8, 13232), (5, 1, 1, 69, 8, 6343), (5, 2, 0, 654, 10512, 1404),
    (5, 2, 1, 519, 9464, 825), (5, 4, 0, 792, 5256, 498), (5, 4, 1, 276, 4856, 628), (5, 8, 0, 500, 6304, 387),
    (5, 8, 1, 459, 5888, 209), (6, 1, 0, 136, 8, 12825), (6, 1, 1, 69, 8, 9536), (6, 2, 0, 796, 7896, 1799),
    (6, 2, 1, 1069, 7304, 755), (6, 4, 0, 657, 6048, 949), (6, 4, 1, 474, 5832, 704), (6, 8, 0, 544, 6192, 661),
    (6, 8, 1, 198, 5928, 710), (7, 1, 0, 1, 8, 1), (7, 1, 1, 1, 9, 1), (7, 2, 1, 3, 4515, 8305), (7, 4, 0, 1, 973, 1),
    (7, 4, 1, 1, 994, 1), (7, 8, 0, 1, 2899, 1), (7, 8, 1, 1, 2018, 1), (8, 1, 0, 5524, 8, 70), (8, 1, 1, 5169, 8, 34),
    (8, 2, 0, 257, 3176, 2815), (8, 2, 1, 179, 3195, 2319), (8, 4, 0, 432, 1221, 345), (8, 4, 1, 353, 1090, 201),
    (8, 8, 0, 248, 1986, 296), (8, 8, 1, 133, 2158, 238), (9, 1, 0, 67, 17, 14210), (9, 1, 1, 72, 11, 7503),
    (9, 2, 0, 1000, 1753, 1421), (9, 2, 1, 783, 1625, 948), (9, 4, 0, 859, 1969, 459), (9, 4, 1, 202, 1738, 890),
    (9, 8, 0, 368, 1989, 582), (9, 8, 1, 194, 2522, 421), (10, 1, 0, 514, 24, 13517), (10, 1, 1, 257, 8, 11712),
    (10, 2, 0, 2329, 3768, 2106), (10, 2, 1, 1319, 3944, 1784), (10, 4, 0, 3080, 6904, 706), (10, 4, 1, 1233, 7368, 987),
    (10, 8, 0, 1312, 10592, 979), (10, 8, 1, 1287, 9136, 525),
]
ANY = (moe.LINEAR_ANY64X32, moe.LINEAR_ANY64X64, moe.LINEAR_ANY128X128)


def taken(lib, T, K, N, gated, unaligned):
    d = linear_desc(n_in=K, n_out=N, ldw=K, act=moe.LINEAR_SWIGLU if gated else moe.LINEAR_NONE, w_up=FAKE if gated else None)
    r = lib.moe_linear_path_for(ctypes.byref(d), FAKE + 2 * unaligned, K, T)
    assert r > 0
    return r % 256, r // 256


def test_cases_take_their_kernels(L):  # noqa: F811
    for kind, parts, gated, T, K, N in CASES:
        assert taken(L, T, K, N, gated, kind in ANY) == (kind, parts), (T, K, N, gated)


def test_the_rule_takes_no_other(L):  # noqa: F811
    rng, found = random.Random(5), set()
    for _ in range(40000):
        T, K, N = (int(round(math.exp(rng.uniform(0.0, math.log(m))))) for m in (8192, 16384, 16384))
        gated, unaligned = rng.random() < 0.5, rng.random() < 0.4
        if not unaligned:
            K = max(8, K // 8 * 8)
        found.add(taken(L, T, K, N, gated, unaligned) + (int(gated),))
    assert found <= {c[:3] for c in CASES}
    assert {c[:1] + c[2:3] for c in CASES} == {(k, g) for k in range(11) for g in (0, 1)}   # every kernel, both ways


def test_path_for_refused(L):  # noqa: F811
    d = linear_desc()
    for x, ldx, T, status in ((FAKE, 640, 0, moe.EINVAL), (FAKE, 639, 2, moe.EINVAL), (None, 640, 2, moe.EINVAL),
                              (FAKE + 1, 640, 2, moe.EINVAL), (FAKE, 640, (1 << 20) + 1, moe.EUNSUPPORTED),
                              (FAKE, (1 << 22) + 1, 2, moe.EUNSUPPORTED)):
        assert L.moe_linear_path_for(ctypes.byref(d), x, ldx, T) == status
    assert L.moe_linear_path_for(ctypes.byref(linear_desc(n_in=0)), FAKE, 640, 2) == moe.EINVAL
    assert L.moe_linear_path_for(None, FAKE, 640, 2) == moe.EINVAL
    assert L.moe_linear_path_for(ctypes.byref(d), FAKE, 1 << 30, 1) > 0   # (one row: whatever its distance)


def call(s, mode, path, in_place=False):
    """(16-bit output, fp32 output) of the kernel and split `path`."""
    T, N, r = s["T"], s["N"], s["residual"]
    d = moe.make_linear_desc(s["w"], w_up=s["w_up"], bias=s["bias"], bias_up=s["bias_up"],
                             act=getattr(moe, "LINEAR_" + s["act"].upper()), situ_b1=B1, situ_b2=B2,
                             residual_type=None if r is None or r.dtype != torch.float32 else moe.F32)
    assert moe.linear_path_for(d, s["x"], T) == path
    h = torch.full((T, N), 99.0, device="cuda", dtype=s["dtype"])
    f = torch.full((T, N), 99.0, device="cuda")
    if in_place:
        r = r.clone()
        h, f = (h, r) if r.dtype == torch.float32 else (r, f)
    moe.linear(d, s["x"], T, h, f, mode, moe.linear_workspace(d, T), residual=r)
    torch.cuda.synchronize()
    return h, f


@pytest.mark.gpu
@pytest.mark.parametrize("case", CASES, ids=str)
def test_each_kernel_is_exact(case):
    kind, parts, gated, T, K, N = case
    dtype = torch.float16 if (T + N) % 2 else torch.bfloat16
    print(f"case: {case} {dtype}", flush=True)
    s = make(T, K, N, dtype, act="swiglu" if gated else "none", bias=torch.float32, residual=torch.float32, whole=True, seed=T + K + N)
    if kind in ANY and K % 8 == 0:
        for n in ("x", "w"):
            t = s[n]
            s[n] = torch.empty(t.numel() + 8, dtype=dtype, device="cuda")[1:1 + t.numel()].view(t.shape)
            s[n].copy_(t)
    if not gated:
        v, _ = reference(s)
        h, f = call(s, moe.OUT_BOTH, (kind, parts))
        assert torch.equal(f.double(), v)
        assert torch.equal(h, v.float().to(dtype))
        return
    # sums of 32 and more have a sigmoid of 1 in fp32: out = a u
    x, r = s["x"].double(), s["residual"].double()
    w, up = s["w"].clone(), s["w_up"].clone()
    for which in (0, 1):
        s["w"].copy_(w if which == 0 else w.zero_())
        s["w_up"].copy_(up if which == 1 else torch.zeros_like(up))
        if which == 0:     # a = 2^17 + x w, u = 1
            s["bias"].fill_(2.0 ** 17)
            s["bias_up"].fill_(1.0)
            v = x @ s["w"].double().t() + 2.0 ** 17 + r
        else:              # a = 32, u = x w_up
            s["bias"].fill_(32.0)
            s["bias_up"].zero_()
            v = 32.0 * (x @ up.double().t()) + r
        h, f = call(s, moe.OUT_BOTH, (kind, parts))
        assert torch.equal(f.double(), v)
        assert torch.equal(h, f.to(dtype))


@pytest.mark.gpu
@pytest.mark.parametrize("act", PLAIN + GATED)
@pytest.mark.parametrize("residual", ["none", "half", "f32", "broadcast half", "broadcast f32", "in place half", "in place f32"])
@pytest.mark.parametrize("ragged", [0, 1])
def test_large_tiles_epilogue(act, residual, ragged):
    """256 x 256 tiles in one part: whole tiles, and some that end inside a tile in both directions."""
    T, K, N = (2304, 136, 4096) if not ragged else (2205, 136, 4300)
    if act in GATED:
        N //= 2
    dtype = torch.bfloat16 if len(act) % 2 else torch.float16
    print(f"case: {act} {residual} {T}x{K}x{N} {dtype}", flush=True)
    rt = None if residual == "none" else torch.float32 if "f32" in residual else dtype
    s = make(T, K, N, dtype, act=act, bias=dtype, residual=rt, seed=T + len(act))
    if "broadcast" in residual:
        s["residual"] = s["residual"][:1].expand(T, N)
    modes = (moe.OUT_HALF, moe.OUT_F32, moe.OUT_BOTH)
    if "in place" in residual:
        modes = (moe.OUT_F32 if rt == torch.float32 else moe.OUT_HALF, moe.OUT_BOTH)
    for mode in modes:
        h, f = call(s, mode, (moe.LINEAR_TILE256X256, 1), "in place" in residual)
        if mode != moe.OUT_F32:
            check(s, h, dtype)
        if mode != moe.OUT_HALF:
            check(s, f, torch.float32)


@pytest.mark.gpu
@pytest.mark.parametrize("gated", [0, 1])
def test_large_tiles_with_the_largest_row_distances(gated):
    """Rows 2^22 elements apart for the 256 x 256 tiles: offsets of more than 2^31 bytes inside a tile."""
    T, K, N, ld = 2304, 136, 4096 // (1 + gated), 1 << 22
    s = make(T, K, N, torch.bfloat16, act="swiglu" if gated else "none", whole=not gated, residual=torch.float32, seed=7)
    for n in ("x", "residual"):
        far = torch.empty(T * ld, dtype=s[n].dtype, device="cuda").view(T, ld)[:, :s[n].shape[1]]
        s[n] = far.copy_(s[n])
    d = moe.make_linear_desc(s["w"], w_up=s["w_up"], act=getattr(moe, "LINEAR_" + s["act"].upper()), residual_type=moe.F32)
    assert moe.linear_path_for(d, s["x"], T) == (moe.LINEAR_TILE256X256, 1)
    h, f = (torch.empty(T * ld, dtype=t, device="cuda").view(T, ld)[:, :N + 8].fill_(99.0) for t in (torch.bfloat16, torch.float32))
    moe.linear(d, s["x"], T, h[:, :N], f[:, :N], moe.OUT_BOTH, moe.linear_workspace(d, T), residual=s["residual"])
    torch.cuda.synchronize()
    check(s, f[:, :N], torch.float32)
    if not gated:
        assert torch.equal(f[:, :N].double(), reference(s)[0])
    assert torch.equal(h[:, :N], f[:, :N].bfloat16())
    assert (h[:, N:] == 99.0).all() and (f[:, N:] == 99.0).all()
    del s, h, f
    torch.cuda.empty_cache()
