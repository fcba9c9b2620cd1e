"""A block's end, the loss and the weights' step run together, as a training
step would: a linear block, its output through the gated norms, the cross
entropy of the head, both backwards, the block's weight gradient by the
library's product, and the Muon step on the block's weight.

Against float64 the chain carries a few independent bf16 roundings (block
output, norm output, dz, dy: RMS 2^-9.8 each), held to the step's bar of
rel-L2 2e-2. Captured into a graph, on other streams and side by side the
operators give the same bits."""
import numpy as np
import pytest

from tests import muon_ref
from tests.common import rel_l2
from tests.gpu_util import from_dev, need_gpu

pytestmark = pytest.mark.gpu


class Step:
    """Buffers of one model and batch; run() issues every operator once on the current stream."""

    def __init__(self, torch, mt, T, V, h, seed):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        n = lambda *s, std=1.0: torch.empty(s, device="cuda").normal_(0, std, generator=g)  # noqa: E731
        e = lambda *s, dt=torch.float32: torch.full(s, 7, device="cuda").to(dt)  # noqa: E731
        bf, u8 = torch.bfloat16, torch.uint8
        self.torch, self.mt, self.dims = torch, mt, (T, V, h)
        self.x, self.a, self.gate = n(T, h), n(T, h).to(bf), n(T, h).to(bf)
        self.Wb, self.M0 = n(h, h, std=h ** -0.5).to(bf), n(h, h, std=1e-3)
        self.Wb0, self.M = self.Wb.clone(), self.M0.clone()
        self.head = n(V, h, std=h ** -0.5).to(bf)
        self.wa, self.wb = 1 + 0.1 * n(h), 1 + 0.1 * n(h)
        self.labels = torch.randint(-1, V, (T,), device="cuda", generator=g).to(torch.int32)
        self.g = torch.rand(T, device="cuda", generator=g) / T
        self.y, self.xo, self.n, self.ra, self.rb = e(T, h, dt=bf), e(T, h), e(T, h, dt=bf), e(T), e(T)
        self.loss, self.lse, self.dn, self.dhead = e(T), e(T), e(T, h), e(V, h, dt=bf)
        self.dx, self.dy, self.dgate, self.dwa, self.dwb, self.dWb = e(T, h), e(T, h, dt=bf), e(T, h, dt=bf), e(h), e(h), e(h, h)
        self.ws_ce = e(max(mt.mt_op_linear_ce_fwd_workspace(T, V, h), mt.mt_op_linear_ce_bwd_workspace(T, V, h)), dt=u8)
        self.ws_n = e(mt.mt_op_sandwich_norm_bwd_workspace(T, h))
        self.ws_m = e(mt.mt_op_orthogonalize_workspace(1, h, h), dt=u8)

    OUT = ("y", "xo", "n", "ra", "rb", "loss", "lse", "dn", "dhead", "dx", "dy", "dgate", "dwa", "dwb", "dWb", "M", "Wb")

    def reset(self):
        self.Wb.copy_(self.Wb0)
        self.M.copy_(self.M0)

    def run(self):
        mt, (T, V, h) = self.mt, self.dims
        B, F = mt.MT_BF16, mt.MT_F32
        mt.mt_op_gemm(mt.MT_GEMM_NT, mt.MT_EPI_BF16, self.a, self.Wb, self.y, None, T, h, h, h, h, h)
        mt.mt_op_sandwich_norm_fwd(self.x, self.y, self.gate, B, self.wa, self.wb, 0.9, 1e-5, self.xo, self.n, self.ra, self.rb, T, h)
        mt.mt_op_linear_ce_fwd(self.n, self.head, self.labels, 1.0, 0.05, 1e-4, self.loss, self.lse, self.ws_ce, T, V, h, h, h)
        mt.mt_op_linear_ce_bwd(self.n, self.head, self.labels, 1.0, 0.05, 1e-4, self.lse, self.g, self.dn, F, self.dhead, B, 0,
                               self.ws_ce, T, V, h, h, h)
        mt.mt_op_sandwich_norm_bwd(self.xo, self.y, self.gate, B, self.wa, self.wb, 0.9, self.ra, self.rb, self.dn, None, self.dx,
                                   self.dy, self.dgate, self.dwa, self.dwb, self.ws_n, T, h)
        mt.mt_op_gemm(mt.MT_GEMM_TN, mt.MT_EPI_F32, self.dy, self.a, self.dWb, None, h, h, T, h, h, h)
        mt.mt_op_muon_update(self.Wb, B, self.M, self.dWb, F, 0.9, 1, 0.02, 0.1, 0.2 * h ** 0.5, None, 5, 1e-9, self.ws_m, 1, h, h)

    def outputs(self):
        return {k: getattr(self, k).clone() for k in self.OUT}


def _same(torch, a, b):
    for k in a:
        assert torch.equal(a[k], b[k]), k


@pytest.mark.parametrize("T,V,h", [(300, 1000, 256), (64, 5000, 128), (1, 300, 64), (1030, 2600, 512)])
def test_step_against_float64(T, V, h):
    torch, mt = need_gpu()
    s = Step(torch, mt, T, V, h, T + V)
    if T == 1:
        s.labels[:] = 5
    s.run()
    torch.cuda.synchronize()
    d = lambda t: t.double()  # noqa: E731
    p = [d(t).requires_grad_() for t in (s.x, s.gate, s.Wb0, s.wa, s.wb, s.head)]
    x, gate, Wb, wa, wb, head = p
    eps = float(np.float32(1e-5))
    y = d(s.a) @ Wb.T
    rms = lambda t: t * (t.square().mean(1, keepdim=True) + eps).rsqrt()  # noqa: E731
    xo = float(np.float32(0.9)) * x + torch.sigmoid(gate) * wa * rms(y)
    z = (wb * rms(xo)) @ head.T
    lse = torch.logsumexp(z, 1)
    keep = s.labels >= 0
    loss = lse - 0.95 * z.gather(1, s.labels.long().clamp(min=0)[:, None])[:, 0] - 0.05 * z.mean(1) + 1e-4 * lse ** 2
    loss = torch.where(keep, loss, 0.0)
    (loss * d(s.g)).sum().backward()
    n = lambda t: t.detach().double().cpu().numpy()  # noqa: E731
    assert rel_l2(n(s.loss), n(loss)) < 2e-2
    # the residual's own path: dres is none here, so x's gradient is the kernel's
    for got, want in ((s.dx, x.grad), (s.dgate, gate.grad), (s.dwa, wa.grad), (s.dwb, wb.grad), (s.dhead, head.grad), (s.dWb, Wb.grad)):
        assert rel_l2(n(got), n(want)) < 2e-2
    # the weights' step from the gradient that the chain left, to its own accuracy
    M = float(np.float32(0.9)) * d(s.M0) + d(s.dWb)
    U = d(s.dWb) + float(np.float32(0.9)) * M
    X = muon_ref.exact(U[None], 5, eps=1e-9)[0]
    W = (1 - 0.002) * d(s.Wb0) - 0.02 * 0.2 * h ** 0.5 * X
    assert rel_l2(n(s.M), n(M)) < 1e-6 and rel_l2(n(s.Wb), n(W)) < 4e-3
    assert mt.mt_op_device_error() == 0


def test_captured_replayed_and_on_other_streams():
    torch, mt = need_gpu()
    a, b = Step(torch, mt, 300, 1500, 256, 1), Step(torch, mt, 77, 4000, 512, 2)
    a.run()
    b.run()
    torch.cuda.synchronize()
    wa, wb = a.outputs(), b.outputs()
    # side by side on two streams, several times over
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        a.reset()
        b.reset()
        torch.cuda.synchronize()
        for st, s in zip(streams, (a, b)):
            with torch.cuda.stream(st):
                s.run()
        torch.cuda.synchronize()
        _same(torch, a.outputs(), wa)
        _same(torch, b.outputs(), wb)
    # captured, replayed with other inputs in the same buffers, and with the first ones again
    g = torch.cuda.CUDAGraph()
    a.reset()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        a.run()
    labels, x = a.labels.clone(), a.x.clone()
    for other in (True, False):
        a.reset()
        a.labels.copy_(labels.flip(0) if other else labels)
        a.x.copy_(-x if other else x)
        for k in ("loss", "dx", "dhead", "dWb"):
            getattr(a, k).fill_(float("nan"))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        got = a.outputs()
        if other:
            a.reset()
            a.run()
            torch.cuda.synchronize()
            _same(torch, got, a.outputs())
            assert not torch.equal(got["loss"], wa["loss"])
        else:
            _same(torch, got, wa)
    # two graphs, each with its own buffers, at the same time
    g2 = torch.cuda.CUDAGraph()
    b.reset()
    torch.cuda.synchronize()
    with torch.cuda.graph(g2):
        b.run()
    for _ in range(3):
        a.reset()
        b.reset()
        torch.cuda.synchronize()
        with torch.cuda.stream(streams[0]):
            g.replay()
        with torch.cuda.stream(streams[1]):
            g2.replay()
        torch.cuda.synchronize()
        _same(torch, a.outputs(), wa)
        _same(torch, b.outputs(), wb)
    assert mt.mt_op_device_error() == 0


def test_behind_copies_and_other_kernels():
    """Inputs that a copy, a fill or a library kernel of the same stream has just written: the operators' blocks may
    start while those end, and have to wait for them."""
    torch, mt = need_gpu()
    s = Step(torch, mt, 500, 3000, 384, 5)
    s.run()
    torch.cuda.synchronize()
    want = s.outputs()
    keep = {k: getattr(s, k).clone() for k in ("x", "a", "gate", "head", "labels", "g", "wa", "wb")}
    big = torch.empty(1 << 27, device="cuda")
    for _ in range(5):
        s.reset()
        for k, v in keep.items():
            getattr(s, k).zero_()
        torch.cuda.synchronize()
        big.fill_(1.0)
        for k, v in keep.items():
            getattr(s, k).copy_(v)
        s.run()
        got = s.outputs()
        s.n.zero_()  # what follows does not reach back
        s.dn.zero_()
        torch.cuda.synchronize()
        _same(torch, got, want)


def test_one_workspace_for_calls_in_order():
    """Cross entropy and orthogonalising share a buffer one after the other on a stream."""
    torch, mt = need_gpu()
    T, V, h = 200, 900, 128
    s = Step(torch, mt, T, V, h, 7)
    s.run()
    torch.cuda.synchronize()
    want = s.outputs()
    shared = torch.full((max(s.ws_ce.numel(), s.ws_m.numel(), 4 * s.ws_n.numel()),), 0xff, dtype=torch.uint8, device="cuda")
    s.ws_ce = s.ws_m = shared
    s.ws_n = shared.view(torch.float32)
    s.reset()
    s.run()
    torch.cuda.synchronize()
    _same(torch, s.outputs(), want)
