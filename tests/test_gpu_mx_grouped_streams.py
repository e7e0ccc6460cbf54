"""A whole FFN of experts (rows sorted, products of groups, sums; with 4-bit experts the rows made in between) on two streams at once,
and captured: graphs that share workspaces and buffers, replayed in turn with new inputs and eager calls between them, equal to the eager
result bit for bit."""
import pytest

import quantized_expert_gemv_sigmoid_amd as moe
from mx_support import pack

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


class Ffn:
    def __init__(self, T, E, k, d, F, mx, seed, share=None):
        g = torch.Generator(device="cuda").manual_seed(seed)
        u8, i32, half = torch.uint8, torch.int32, torch.bfloat16

        def e(*shape, dtype=half):
            return torch.empty(*shape, dtype=dtype, device="cuda")

        self.T, self.E, self.R, self.mx, self.g = T, E, T * k, mx, g
        self.x, self.ids, self.weights = e(T, d), e(T, k, dtype=i32), e(T, k, dtype=torch.float32)
        w1, w3, w2 = (torch.randn(E, *n, device="cuda", generator=g) * n[1] ** -0.5 for n in ((F, d), (F, d), (d, F)))
        if mx:
            self.q = [pack(w, "fit") for w in (w1, w3, w2)]
            self.up = moe.make_grouped_desc(self.q[0][0], w_s=self.q[0][1], w_up=self.q[1][0], w_up_s=self.q[1][1], act=moe.LINEAR_SITU_GLU)
            self.down = moe.make_grouped_desc(self.q[2][0], w_s=self.q[2][1])
        else:
            self.q = [w.to(half) for w in (w1, w3, w2)]
            self.up = moe.make_grouped_desc(self.q[0], w_up=self.q[1], act=moe.LINEAR_SWIGLU)
            self.down = moe.make_grouped_desc(self.q[2])
        self.buffers = share.buffers if share else dict(
            offsets=e(E + 1, dtype=i32), tokens=e(self.R, dtype=i32), places=e(T, k, dtype=i32), ws=moe.group_workspace(T, k, E),
            h=e(self.R, F), y=e(self.R, d, dtype=torch.float32), xq=e(T, d // 2, dtype=u8), xs=e(T, d // 32, dtype=u8),
            hq=e(self.R, F // 2, dtype=u8), hs=e(self.R, F // 32, dtype=u8))
        self.out = e(T, d)
        self.refill()

    def refill(self):
        T, k = self.ids.shape
        self.x.copy_(torch.randn(self.x.shape, device="cuda", generator=self.g))
        self.ids.copy_(torch.rand(T, self.E, device="cuda", generator=self.g).topk(k, dim=1)[1])
        self.ids[torch.rand(T, k, device="cuda", generator=self.g) < 0.1] = -1
        self.weights.copy_(torch.rand(T, k, device="cuda", generator=self.g))

    def run(self, out=None, stream=None):
        b, T, R = self.buffers, self.T, self.R
        moe.group(self.ids, T, self.E, b["offsets"], b["tokens"], b["places"], b["ws"], stream=stream)
        x, h, xs, hs = self.x, b["h"], None, None
        if self.mx:
            moe.mx_quantize(x, T, b["xq"], b["xs"], stream=stream)
            x, xs = b["xq"], b["xs"]
        moe.grouped_linear(self.up, x, b["offsets"], R, h, None, moe.OUT_HALF, rows=b["tokens"], x_s=xs, stream=stream)
        if self.mx:
            # (rows of no choice hold whatever was there: they are quantised with the rest, and no group reads them)
            moe.mx_quantize(h, R, b["hq"], b["hs"], rule=moe.MX_FIT, stream=stream)
            h, hs = b["hq"], b["hs"]
        moe.grouped_linear(self.down, h, b["offsets"], R, None, b["y"], moe.OUT_F32, x_s=hs, stream=stream)
        out = self.out if out is None else out
        moe.combine(b["y"], R, b["places"], self.weights, T, out, residual=self.x, stream=stream)
        return out


def eager(f):
    return f.run(out=torch.empty_like(f.out)).clone()


@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("T", [1, 70, 900])
def test_two_streams_at_once(mx, T):
    a, b = Ffn(T, 16, 4, 512, 384, mx, 1), Ffn(T, 24, 3, 384, 640, mx, 2)
    want = eager(a), eager(b)
    assert torch.isfinite(want[0]).all() and want[0].float().abs().max() > 0
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for f in (a, b):
        f.out.fill_(7.0)
    torch.cuda.synchronize()
    for _ in range(20):
        for f, s in zip((a, b), streams):
            f.run(stream=s)
    torch.cuda.synchronize()
    assert torch.equal(a.out, want[0]) and torch.equal(b.out, want[1])


@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("T", [1, 70, 900])
def test_graphs_that_share_workspaces(mx, T):
    a = Ffn(T, 16, 4, 512, 384, mx, 3)
    b = Ffn(T, 16, 4, 512, 384, mx, 4, share=a)
    eager(a), eager(b)
    torch.cuda.synchronize()
    graphs = []
    for f in (a, b):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            f.run()
        graphs.append(g)
    for _ in range(4):
        for f in (a, b):
            f.refill()
            f.out.fill_(7.0)
        for t in a.buffers.values():
            t.fill_(0 if t.is_floating_point() else 255 if t.dtype == torch.uint8 else -1)
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        got = a.out.clone(), b.out.clone()
        assert torch.equal(got[0], eager(a)) and torch.equal(got[1], eager(b))
        torch.cuda.synchronize()
