"""MXFP4 rows in plain torch, for the tests: made and read back as the format says, in 64 bits."""
import torch

def power(e):
    """2^e in float64 from its bits, -1022 <= e <= 1023 (pow and exp2 may be off by a bit)."""
    return ((e.long() + 1023) << 52).view(torch.float64)


E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def scale_bytes(blocks, rule):
    """Scale bytes of blocks [.., 32] of finite float64 values (as a list of integers' arithmetic: exact)."""
    top = blocks.abs().amax(-1)
    m, e = torch.frexp(top)           # top = m 2^e, 0.5 <= m < 1
    e = e.int() - 3                   # floor(log2 top) - 2
    if rule == "fit":
        e = e + (top > 6.0 * power(e)).int()
    e = torch.where(top > 0, e, -127).clamp_min(-127)
    return (e + 127).to(torch.uint8)


def pack(x, rule="floor"):
    """(codes [.., 16 blocks], scales [.., blocks]) of rows x, any float type; the last block filled with zeros."""
    x = x.double()
    n = x.shape[-1]
    b = (n + 31) // 32
    v = torch.zeros(*x.shape[:-1], b * 32, dtype=torch.float64, device=x.device)
    v[..., :n] = x
    v = v.view(*x.shape[:-1], b, 32)
    bad = ~torch.isfinite(v).all(-1)
    v = torch.where(bad[..., None], 0.0, v)
    s = scale_bytes(v, rule)
    q = v * power(127 - s[..., None].int())
    a = q.abs()
    # between neighbours the even code's is the tie's
    c = torch.zeros_like(a, dtype=torch.uint8)
    for code in range(1, 8):
        mid = (E2M1[code - 1] + E2M1[code]) / 2
        c = torch.where(a >= mid if code % 2 == 0 else a > mid, code, c).to(torch.uint8)
    c = c | (torch.signbit(q).to(torch.uint8) << 3)
    c = torch.where(bad[..., None], 0, c).to(torch.uint8)
    c = c.view(*x.shape[:-1], b * 32)
    s = torch.where(bad, 255, s).to(torch.uint8)
    return (c[..., 0::2] | (c[..., 1::2] << 4)).contiguous(), s.contiguous()


def unpack(codes, scales):
    """float64 values of such rows (NaN for scale byte 255)."""
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), dtype=torch.float64, device=codes.device)
    v = table[torch.stack([codes & 15, codes >> 4], -1).long()].view(*codes.shape[:-1], -1, 32)
    v = v * power(scales[..., None].int() - 127)
    v = torch.where(scales[..., None] == 255, float("nan"), v)
    return v.reshape(*codes.shape[:-1], -1)
