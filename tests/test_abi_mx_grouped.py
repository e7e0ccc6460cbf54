"""Host-side checks of the MXFP4 rows and product, the products of groups, moe_group and moe_combine: descriptor layouts,
and arguments refused before any launch (no GPU needed)."""
import ctypes

import pytest

import quantized_expert_gemv_sigmoid_amd as moe
from mx_support import pack, unpack
from test_abi import FAKE
from test_abi_gate_linear import L, test_layout_matches_c as layout_matches_c  # noqa: F401 (L: a fixture)

torch = pytest.importorskip("torch")
WS = FAKE * 16


@pytest.mark.parametrize("mirror,name", [(moe.MxLinearDesc, "moe_mx_linear_desc"), (moe.GroupedDesc, "moe_grouped_desc")])
def test_layout_matches_c(tmp_path, mirror, name):
    layout_matches_c(tmp_path, mirror, name)


def filled(cls, base, kw):
    d = cls()
    for k, v in {**base, **kw}.items():
        setattr(d, k, v)
    return d


MX = dict(n_in=640, n_out=512, type=moe.BF16, act=moe.LINEAR_NONE, situ_b1=4.0, situ_b2=25.0, bias_type=moe.F32,
          residual_type=moe.BF16, ldw=320, ldw_s=20, w=FAKE, w_s=FAKE)


def call_mx(L, d, x=FAKE, ldx=320, xs=FAKE, ldxs=20, T=3, res=None, ldr=0, oh=FAKE, of=None, ldo=512, mode=moe.OUT_HALF,
            ws=(WS, 1 << 40)):
    return L.moe_mx_linear(ctypes.byref(d) if d is not None else None, x, ldx, xs, ldxs, T, res, ldr, oh, of, ldo, mode, ws[0], ws[1],
                           None)


@pytest.mark.parametrize("kw,status", [
    (dict(n_in=0), moe.EINVAL), (dict(n_in=656), moe.EINVAL), (dict(n_out=0), moe.EINVAL), (dict(ldw=319), moe.EINVAL),
    (dict(ldw=328), moe.EINVAL), (dict(ldw_s=19), moe.EINVAL), (dict(type=moe.F32), moe.EINVAL), (dict(type=moe.MXFP4), moe.EINVAL),
    (dict(act=7), moe.EINVAL), (dict(bias_type=moe.F16), moe.EINVAL), (dict(residual_type=moe.F16), moe.EINVAL),
    (dict(w=None), moe.EINVAL), (dict(w_s=None), moe.EINVAL), (dict(w=FAKE + 8), moe.EINVAL),
    (dict(w_up=FAKE, w_up_s=FAKE), moe.EINVAL), (dict(bias_up=FAKE), moe.EINVAL), (dict(act=moe.LINEAR_SWIGLU), moe.EINVAL),
    (dict(act=moe.LINEAR_SWIGLU, w_up=FAKE), moe.EINVAL), (dict(act=moe.LINEAR_SWIGLU, w_up=FAKE + 8, w_up_s=FAKE), moe.EINVAL),
    (dict(act=moe.LINEAR_SITU_GLU, w_up=FAKE, w_up_s=FAKE, situ_b1=-1.0), moe.EINVAL), (dict(bias=FAKE + 2), moe.EINVAL),
    (dict(n_out=(1 << 20) + 1), moe.EUNSUPPORTED), (dict(ldw=(1 << 23) + 16), moe.EUNSUPPORTED),
    (dict(ldw_s=(1 << 22) + 1), moe.EUNSUPPORTED),
])
def test_mx_descriptor_refused(L, kw, status):  # noqa: F811
    d = filled(moe.MxLinearDesc, MX, kw)
    assert call_mx(L, d, ldx=1 << 20, ldxs=1 << 20, ldo=1 << 21) == status
    assert L.moe_mx_linear_workspace_bytes(ctypes.byref(d), 4) == 0
    assert L.moe_mx_linear_path_for(ctypes.byref(d), 4) == status


def test_mx_call_refused(L):  # noqa: F811
    d = filled(moe.MxLinearDesc, MX, {})
    assert call_mx(L, None) == moe.EINVAL
    assert call_mx(L, d, T=0, x=None, xs=None, ws=(None, 0)) == moe.OK
    need = L.moe_mx_linear_workspace_bytes(ctypes.byref(d), 3)
    for kw in (dict(T=-1), dict(ldx=319), dict(ldx=336 - 8), dict(ldxs=19), dict(ldo=511), dict(x=None), dict(x=FAKE + 8), dict(xs=None),
               dict(oh=None), dict(oh=FAKE + 1), dict(mode=3), dict(res=FAKE, ldr=511), dict(res=FAKE + 1, ldr=512), dict(mode=moe.OUT_F32),
               dict(mode=moe.OUT_BOTH), dict(mode=moe.OUT_F32, of=FAKE + 2), dict(ws=(None, need)), dict(ws=(WS + 16, need))):
        assert call_mx(L, d, **kw) == moe.EINVAL, kw
    assert call_mx(L, d, ws=(WS, need - 1)) == moe.EWORKSPACE
    for kw in (dict(T=(1 << 20) + 1), dict(ldx=(1 << 23) + 16), dict(ldxs=(1 << 22) + 1), dict(ldo=(1 << 22) + 1),
               dict(res=FAKE, ldr=(1 << 22) + 1)):
        assert call_mx(L, d, **kw) == moe.EUNSUPPORTED, kw
    # scales that start anywhere need room for a copy; x's may in any call
    assert L.moe_mx_linear_workspace_bytes(ctypes.byref(filled(moe.MxLinearDesc, MX, dict(w_s=FAKE + 1))), 3) >= need + 512 * 24


GROUPED = dict(n_groups=8, n_in=640, n_out=512, type=moe.F16, operands=moe.F16, act=moe.LINEAR_NONE, situ_b1=4.0, situ_b2=25.0,
               bias_type=moe.F32, ldw=640, group_w=640 * 512, w=FAKE)
GROUPED_MX = dict(GROUPED, operands=moe.MXFP4, ldw=320, group_w=320 * 512, ldw_s=20, group_w_s=20 * 512, w_s=FAKE)


def call_grouped(L, d, x=FAKE, ldx=None, xs=0, ldxs=20, x_rows=3, rows=None, offsets=FAKE, R=3, oh=FAKE, of=None, ldo=512,
                 mode=moe.OUT_HALF):
    mx = d is not None and d.operands == moe.MXFP4
    ldx = (320 if mx else 640) if ldx is None else ldx
    xs = (FAKE if mx else None) if xs == 0 else xs
    return L.moe_grouped_linear(ctypes.byref(d) if d is not None else None, x, ldx, xs, ldxs, x_rows, rows, offsets, R, oh, of, ldo,
                                mode, None)


@pytest.mark.parametrize("kw,status", [
    (dict(n_groups=0), moe.EINVAL), (dict(n_in=0), moe.EINVAL), (dict(n_out=0), moe.EINVAL), (dict(ldw=639), moe.EINVAL),
    (dict(group_w=-1), moe.EINVAL), (dict(type=moe.F32, operands=moe.F32), moe.EINVAL), (dict(operands=moe.BF16), moe.EINVAL),
    (dict(operands=7), moe.EINVAL), (dict(act=9), moe.EINVAL), (dict(bias_type=moe.BF16), moe.EINVAL), (dict(w=None), moe.EINVAL),
    (dict(w=FAKE + 1), moe.EINVAL), (dict(w_up=FAKE), moe.EINVAL), (dict(act=moe.LINEAR_SWIGLU), moe.EINVAL), (dict(bias_up=FAKE), moe.EINVAL),
    (dict(act=moe.LINEAR_SITU_GLU, w_up=FAKE, situ_b2=float("nan")), moe.EINVAL), (dict(bias=FAKE + 2), moe.EINVAL),
    (dict(n_groups=1025), moe.EUNSUPPORTED), (dict(n_out=(1 << 20) + 1), moe.EUNSUPPORTED), (dict(ldw=(1 << 22) + 1), moe.EUNSUPPORTED),
])
def test_grouped_descriptor_refused(L, kw, status):  # noqa: F811
    d = filled(moe.GroupedDesc, GROUPED, kw)
    assert call_grouped(L, d, ldx=1 << 20, ldo=1 << 21) == status
    assert L.moe_grouped_path_for(ctypes.byref(d), FAKE, 1 << 20, 3) == status


@pytest.mark.parametrize("kw,status", [
    (dict(n_in=624), moe.EINVAL), (dict(ldw=312), moe.EINVAL), (dict(ldw=328), moe.EINVAL), (dict(ldw_s=19), moe.EINVAL),
    (dict(w_s=None), moe.EINVAL), (dict(w=FAKE + 8), moe.EINVAL), (dict(group_w=320 * 512 + 8), moe.EINVAL), (dict(group_w_s=-4), moe.EINVAL),
    (dict(act=moe.LINEAR_SWIGLU, w_up=FAKE), moe.EINVAL), (dict(type=moe.F32), moe.EINVAL), (dict(n_in=608), moe.EUNSUPPORTED),
    (dict(ldw_s=22), moe.EUNSUPPORTED), (dict(w_s=FAKE + 2), moe.EUNSUPPORTED), (dict(group_w_s=20 * 512 + 2), moe.EUNSUPPORTED),
    (dict(ldw=(1 << 23) + 16), moe.EUNSUPPORTED), (dict(ldw_s=(1 << 22) + 4), moe.EUNSUPPORTED),
])
def test_grouped_mx_descriptor_refused(L, kw, status):  # noqa: F811
    assert call_grouped(L, filled(moe.GroupedDesc, GROUPED_MX, kw), ldx=1 << 20, ldxs=1 << 16, ldo=1 << 21) == status


def test_grouped_call_refused(L):  # noqa: F811
    d, m = filled(moe.GroupedDesc, GROUPED, {}), filled(moe.GroupedDesc, GROUPED_MX, {})
    assert call_grouped(L, None) == moe.EINVAL
    assert call_grouped(L, d, R=0, x=None, offsets=None, oh=FAKE) == moe.OK
    for kw in (dict(R=-1), dict(ldx=639), dict(ldo=511), dict(x=None), dict(x=FAKE + 1), dict(xs=FAKE), dict(x_rows=2), dict(x_rows=0, rows=FAKE),
               dict(rows=FAKE + 2), dict(offsets=None), dict(offsets=FAKE + 2), dict(oh=None), dict(oh=FAKE + 1), dict(mode=3),
               dict(mode=moe.OUT_F32), dict(mode=moe.OUT_BOTH), dict(mode=moe.OUT_F32, of=FAKE + 2)):
        assert call_grouped(L, d, **kw) == moe.EINVAL, kw
    for kw in (dict(ldx=312), dict(ldx=328), dict(ldxs=19), dict(x=FAKE + 8), dict(xs=None)):
        assert call_grouped(L, m, **kw) == moe.EINVAL, kw
    for kw in (dict(R=(1 << 24) + 1, x_rows=1 << 25), dict(ldx=(1 << 22) + 1), dict(ldo=(1 << 22) + 1),
               dict(rows=FAKE, x_rows=1 << 21)):   # gathered rows over more than 2 GiB
        assert call_grouped(L, d, **kw) == moe.EUNSUPPORTED, kw
    for kw in (dict(ldxs=22), dict(xs=FAKE + 2), dict(ldx=(1 << 23) + 16), dict(ldxs=(1 << 22) + 4), dict(rows=FAKE, x_rows=1 << 23),
               dict(rows=FAKE, x_rows=1 << 10, ldxs=1 << 22)):
        assert call_grouped(L, m, **kw) == moe.EUNSUPPORTED, kw



@pytest.mark.parametrize("base", [GROUPED, GROUPED_MX])
@pytest.mark.parametrize("gated", [0, 1])
def test_groups_of_more_threads_than_a_launch_holds_are_refused(L, base, gated):  # noqa: F811
    up = dict(act=moe.LINEAR_SWIGLU, w_up=FAKE, w_up_s=FAKE if base is GROUPED_MX else None) if gated else {}
    ld = 320 if base is GROUPED_MX else 640

    d = filled(moe.GroupedDesc, base, {**up, "n_out": 1 << 20, "n_groups": 1024, "group_w": 0, "group_w_s": 0})
    assert L.moe_grouped_path_for(ctypes.byref(d), FAKE, ld, 1 << 24) == moe.EUNSUPPORTED
    assert call_grouped(L, d, R=1 << 24, x_rows=1 << 24, ldo=1 << 20) == moe.EUNSUPPORTED
    # (64 x 32 tiles, with the least idle rows, would be 2^25.6 blocks of 256)
    assert L.moe_grouped_path_for(ctypes.byref(d), FAKE, ld, 65536) == moe.LINEAR_TILE256X128 + 256
    if base is GROUPED:
        d.n_out = 1 << 17
        r = L.moe_grouped_path_for(ctypes.byref(d), FAKE + 2, ld, 1 << 17)
        assert r >= 0 and r % 256 in (moe.LINEAR_ANY64X32, moe.LINEAR_ANY64X64, moe.LINEAR_ANY128X128)
        d.n_out = 1 << 20
        assert L.moe_grouped_path_for(ctypes.byref(d), FAKE + 2, ld, 1 << 17) == moe.EUNSUPPORTED


def test_mx_rows_refused(L):  # noqa: F811
    def quantize(x=FAKE, type=moe.BF16, ldx=70, T=3, n=70, rule=0, c=FAKE, ldc=48, s=FAKE, lds=3):
        return L.moe_mx_quantize(x, type, ldx, T, n, rule, c, ldc, s, lds, None)

    def dequantize(o=FAKE, type=moe.BF16, ldo=70, T=3, n=70, c=FAKE, ldc=48, s=FAKE, lds=3):
        return L.moe_mx_dequantize(c, ldc, s, lds, T, n, o, type, ldo, None)

    assert quantize(T=0, x=None, c=None, s=None) == moe.OK and dequantize(T=0, o=None, c=None, s=None) == moe.OK
    for kw in (dict(type=3), dict(T=-1), dict(n=0), dict(ldc=47), dict(lds=2), dict(c=None), dict(s=None)):
        assert quantize(**kw) == moe.EINVAL and dequantize(**kw) == moe.EINVAL, kw
    for kw in (dict(x=None), dict(x=FAKE + 1), dict(x=FAKE + 2, type=moe.F32), dict(ldx=69), dict(rule=2), dict(rule=-1)):
        assert quantize(**kw) == moe.EINVAL, kw
    for kw in (dict(o=None), dict(o=FAKE + 1), dict(ldo=69)):
        assert dequantize(**kw) == moe.EINVAL, kw
    assert quantize(n=(1 << 20) + 1, ldx=1 << 21, ldc=1 << 21, lds=1 << 21) == moe.EUNSUPPORTED


def test_group_and_combine_refused(L):  # noqa: F811
    def group(ids=FAKE, T=3, k=4, E=8, o=FAKE, t=FAKE, p=FAKE, ws=(WS, 1 << 30)):
        return L.moe_group(ids, T, k, E, o, t, p, ws[0], ws[1], None)

    for kw in (dict(T=-1), dict(k=0), dict(E=0), dict(o=None), dict(ids=None), dict(t=None), dict(p=None), dict(ids=FAKE + 2),
               dict(o=FAKE + 1), dict(t=FAKE + 2), dict(p=FAKE + 2), dict(ws=(None, 1 << 30)), dict(ws=(WS + 8, 1 << 30))):
        assert group(**kw) == moe.EINVAL, kw
    for kw in (dict(T=(1 << 20) + 1), dict(k=65), dict(E=1025)):
        assert group(**kw) == moe.EUNSUPPORTED, kw
    need = L.moe_group_workspace_bytes(1 << 20, 64, 1024)
    assert group(T=1 << 20, k=64, E=1024, ws=(WS, need - 1)) == moe.EWORKSPACE
    assert L.moe_group_workspace_bytes(4, 65, 8) == 0 and L.moe_group_workspace_bytes(-1, 4, 8) == 0

    def combine(y=FAKE, yt=moe.F32, ldy=64, R=9, p=FAKE, w=FAKE, T=3, k=4, n=64, r=None, rt=moe.F32, ldr=64, o=FAKE, ot=moe.BF16, ldo=64):
        return L.moe_combine(y, yt, ldy, R, p, w, T, k, n, r, rt, ldr, o, ot, ldo, None)

    assert combine(T=0, y=None, p=None, o=None) == moe.OK
    for kw in (dict(yt=3), dict(ot=-1), dict(r=FAKE, rt=5), dict(T=-1), dict(R=-1), dict(k=0), dict(n=0), dict(ldy=63), dict(ldo=63),
               dict(r=FAKE, ldr=63), dict(y=None), dict(p=None), dict(o=None), dict(y=FAKE + 2), dict(p=FAKE + 2), dict(w=FAKE + 2),
               dict(o=FAKE + 1), dict(r=FAKE + 2)):
        assert combine(**kw) == moe.EINVAL, kw
    for kw in (dict(T=(1 << 20) + 1), dict(k=65), dict(n=(1 << 20) + 1, ldy=1 << 21, ldo=1 << 21)):
        assert combine(**kw) == moe.EUNSUPPORTED, kw


@pytest.mark.parametrize("E", [1, 31, 64, 1024])
def test_a_group_workspace_serves_fewer_tokens(L, E):  # noqa: F811
    need = [L.moe_group_workspace_bytes(T, 4, E) for T in (0, 1, 255, 256, 257, 300, 1000, 16384, 16385, 16500, 30000, 1 << 20)]
    assert need == sorted(need) and need[0] >= 256


# ------------------------------------------------------------------ the binding

def u8(*shape, device="cpu"):
    return torch.empty(*shape, dtype=torch.uint8, device=device)


def half(*shape, device="cpu", dtype=torch.bfloat16):
    return torch.empty(*shape, dtype=dtype, device=device)


def i32(*shape, device="cpu"):
    return torch.empty(*shape, dtype=torch.int32, device=device)


def refused(match, f, *a, **kw):
    with pytest.raises(moe.MoeError, match=match):
        f(*a, **kw)


def test_binding_refuses_mx():
    x = half(4, 70)
    refused("codes", moe.mx_quantize, x, 4, u8(4, 40), u8(4, 3))
    refused("scales", moe.mx_quantize, x, 4, u8(4, 48), u8(3, 3))
    refused("x: 5 rows", moe.mx_quantize, x, 5, u8(5, 48), u8(5, 3))
    refused("dtype", moe.mx_quantize, x.double(), 4, u8(4, 48), u8(4, 3))
    refused("codes", moe.mx_quantize, x, 4, half(4, 48), u8(4, 3))
    refused("tensors on", moe.mx_quantize, x, 4, u8(4, 48, device="meta"), u8(4, 3))
    refused("tensors on cpu", moe.mx_quantize, x, 4, u8(4, 48), u8(4, 3))
    refused("tensors on cpu", moe.mx_dequantize, u8(4, 48), u8(4, 3), 4, x)
    refused("out", moe.mx_dequantize, u8(4, 48), u8(4, 3), 4, half(4))
    refused("w_s", moe.make_mx_linear_desc, u8(8, 32), u8(8, 3))
    refused("together", moe.make_mx_linear_desc, u8(8, 32), u8(8, 2), w_up=u8(8, 32))
    refused("not laid out", moe.make_mx_linear_desc, u8(8, 32), u8(8, 2), w_up=u8(8, 64)[:, :32], w_up_s=u8(8, 2))
    refused("tensors on", moe.make_mx_linear_desc, u8(8, 32), u8(8, 2, device="meta"))
    d = moe.make_mx_linear_desc(u8(8, 32), u8(8, 2))
    ws = (256, 1 << 30)
    refused("x_s", moe.mx_linear, d, u8(3, 32), u8(3, 3), 3, half(3, 8), None, moe.OUT_HALF, ws)
    refused("x: ", moe.mx_linear, d, half(3, 32), u8(3, 2), 3, half(3, 8), None, moe.OUT_HALF, ws)
    refused("out_half", moe.mx_linear, d, u8(3, 32), u8(3, 2), 3, half(3, 8, dtype=torch.float16), None, moe.OUT_HALF, ws)
    refused("residual", moe.mx_linear, d, u8(3, 32), u8(3, 2), 3, half(3, 8), None, moe.OUT_HALF, ws, residual=torch.empty(3, 8))
    refused("tensors on cpu and meta", moe.mx_linear, d, u8(3, 32, device="meta"), u8(3, 2, device="meta"), 3, half(3, 8, device="meta"), None,
            moe.OUT_HALF, ws)
    refused("tensors on cpu", moe.mx_linear, d, u8(3, 32), u8(3, 2), 3, half(3, 8), None, moe.OUT_HALF, ws)


def test_binding_refuses_groups():
    w = half(3, 8, 16)
    refused("matrices", moe.make_grouped_desc, half(8, 16))
    refused("matrices", moe.make_grouped_desc, half(3, 16, 8).transpose(1, 2))
    refused("not laid out", moe.make_grouped_desc, w, w_up=half(3, 8, 32)[..., :16], act=moe.LINEAR_SWIGLU)
    refused("not laid out", moe.make_grouped_desc, w, w_up=half(3, 9, 16), act=moe.LINEAR_SWIGLU)
    refused("bias", moe.make_grouped_desc, w, bias=half(8))
    refused("type", moe.make_grouped_desc, w, type=moe.F16)
    refused("type", moe.make_grouped_desc, w.float())
    refused("together", moe.make_grouped_desc, w, w_up_s=u8(3, 8, 4))
    refused("w_s", moe.make_grouped_desc, u8(3, 8, 64), w_s=u8(3, 8, 3))
    refused("together", moe.make_grouped_desc, u8(3, 8, 64), w_s=u8(3, 8, 4), w_up=u8(3, 8, 64))
    d = moe.make_grouped_desc(w)
    assert (d.n_groups, d.n_out, d.n_in, d.ldw, d.group_w) == (3, 8, 16, 16, 128)
    o, x, out = i32(4), half(5, 16), half(5, 8)
    refused("x: ", moe.grouped_linear, d, half(5, 16, dtype=torch.float16), o, 5, out, None, moe.OUT_HALF)
    refused("x: 6 rows", moe.grouped_linear, d, x, o, 6, half(6, 8), None, moe.OUT_HALF)
    refused("offsets", moe.grouped_linear, d, x, i32(3), 5, out, None, moe.OUT_HALF)
    refused("rows", moe.grouped_linear, d, x, o, 5, out, None, moe.OUT_HALF, rows=i32(4))
    refused("rows", moe.grouped_linear, d, x, o, 5, out, None, moe.OUT_HALF, rows=torch.empty(5, dtype=torch.int64))
    refused("x_s", moe.grouped_linear, d, x, o, 5, out, None, moe.OUT_HALF, x_s=u8(5, 1))
    refused("tensors on", moe.grouped_linear, d, x, i32(4, device="meta"), 5, out, None, moe.OUT_HALF)
    refused("tensors on cpu", moe.grouped_linear, d, x, o, 5, out, None, moe.OUT_HALF)
    ids, ws = i32(5, 2), (256, 1 << 20)
    refused("ids", moe.group, ids, 6, 4, i32(5), i32(12), i32(6, 2), ws)
    refused("offsets", moe.group, ids, 5, 4, i32(4), i32(10), i32(5, 2), ws)
    refused("tokens", moe.group, ids, 5, 4, i32(5), i32(9), i32(5, 2), ws)
    refused("places", moe.group, ids, 5, 4, i32(5), i32(10), i32(5, 1), ws)
    refused("ids", moe.group, ids.long(), 5, 4, i32(5), i32(10), i32(5, 2), ws)
    refused("tensors on cpu", moe.group, ids, 5, 4, i32(5), i32(10), i32(5, 2), ws)
    p = i32(5, 2)
    refused("weights", moe.combine, x, 5, p, torch.empty(9), 5, half(5, 16))
    refused("out", moe.combine, x, 5, p, None, 5, half(5, 8))
    refused("residual", moe.combine, x, 5, p, None, 5, half(5, 16), residual=half(4, 16))
    refused("tensors on cpu", moe.combine, x, 5, p, None, 5, half(5, 16))


def test_the_definition_of_the_tests():
    """pack and unpack of mx_support on cases worked by hand."""
    x = torch.zeros(5, 32)
    x[0, :4] = torch.tensor([6.0, 2.5, -0.25, 0.75])      # scale 1: ties to even
    x[1, :2] = torch.tensor([7.5, 1.0])                   # floor: 7.5 becomes 6; fit: scale 2, 3.75 -> 4
    x[2, 0] = float("inf")
    x[4, :2] = torch.tensor([2.0 ** -149, -2.0 ** -140])
    c, s = pack(x)
    assert s[:, 0].tolist() == [127, 127, 255, 0, 0]
    assert unpack(c, s)[0, :4].tolist() == [6.0, 2.0, 0.0, 1.0] and unpack(c, s)[1, :2].tolist() == [6.0, 1.0]
    assert c[0, 0] == 0x47 and c[0, 1] == 0x28 and (c[2:] == 0).all(1).tolist()[:2] == [True, True]
    c, s = pack(x, "fit")
    assert s[1, 0] == 128 and unpack(c, s)[1, :2].tolist() == [8.0, 1.0]
