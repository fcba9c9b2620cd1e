"""The gated norms around a block's end against float64, element by element.

Errors counted: a sum of h squares or products acc(h) of its magnitudes, each
further operation 2^-24, the hardware's exponential and reciprocal a few of
those (the exponential's argument |s| 2^-24 more), bf16 results 2^-8."""
import numpy as np
import pytest

from tests.bounds import U16, U32, acc, check
from tests.gpu_util import from_dev, need_gpu

pytestmark = pytest.mark.gpu


class Case:
    def __init__(self, torch, T, h, bf16, gate, seed, resid=True):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        n = lambda *s: torch.randn(s, device="cuda", generator=g)  # noqa: E731
        dt = torch.bfloat16 if bf16 else torch.float32
        self.T, self.h, self.dt, self.torch = T, h, dt, torch
        self.x, self.y = n(T, h) * torch.exp(n(T, 1)), (n(T, h) * torch.exp(n(T, 1))).to(dt)
        self.gate = (3 * n(T, h)).to(dt) if gate else None
        self.wa, self.wb = 1 + 0.2 * n(h), 1 + 0.2 * n(h)
        self.dn, self.dres = n(T, h), n(T, h) if resid else None
        self.alpha, self.eps = 0.75, 1e-5

    def run(self, mt, x_out=None, dx=None):
        torch, T, h = self.torch, self.T, self.h
        code = mt.MT_BF16 if self.dt == torch.bfloat16 else mt.MT_F32
        self.guards = []

        def out(*s, dt=torch.float32):
            n = int(np.prod(s))
            raw = torch.full((n + 64,), float("nan"), device="cuda", dtype=dt)
            self.guards.append(raw[n:])
            return raw[:n].view(s)
        r = Case.__new__(Case)
        r.x_out, r.n = out(T, h) if x_out is None else x_out, out(T, h, dt=torch.bfloat16)
        r.ra, r.rb = out(T), out(T)
        mt.mt_op_sandwich_norm_fwd(self.x if x_out is None else x_out, self.y, self.gate, code, self.wa, self.wb, self.alpha,
                                   self.eps, r.x_out, r.n, r.ra, r.rb, T, h)
        r.dx, r.dy = out(T, h) if dx is None else dx, out(T, h, dt=self.dt)
        r.ds = out(T, h, dt=self.dt) if self.gate is not None else None
        r.dwa, r.dwb = out(h), out(h)
        ws = out(mt.mt_op_sandwich_norm_bwd_workspace(T, h))
        mt.mt_op_sandwich_norm_bwd(r.x_out, self.y, self.gate, code, self.wa, self.wb, self.alpha, r.ra, r.rb, self.dn,
                                   self.dres if dx is None else dx, r.dx, r.dy, r.ds, r.dwa, r.dwb, ws, T, h)
        assert all(torch.isnan(g).all() for g in self.guards)
        return r

    def check(self, r):
        torch, h, T = self.torch, self.h, self.T
        f = lambda t: None if t is None else t.double()  # noqa: E731
        n = lambda t: t.cpu().numpy()  # noqa: E731
        x, y, wa, wb, al = f(self.x), f(self.y), f(self.wa), f(self.wb), self.alpha
        eps = float(np.float32(self.eps))
        u = U16 if self.dt == torch.bfloat16 else U32
        A = acc(h) + 8 * U32
        ra = (y.square().mean(1, keepdim=True) + eps).rsqrt()
        check(from_dev(r.ra), n(ra[:, 0]), n(A * ra[:, 0]), "rstd_post")
        yh = y * ra
        uu = yh * wa
        sg = torch.sigmoid(f(self.gate)) if self.gate is not None else torch.ones_like(y)
        # relative error of the sigmoid; from |s| = 200 on e^-|s| is below 2^-126, so that it is exactly 0 or 1
        se = (16 * U32 + 2 * U32 * f(self.gate).abs().clamp(max=200.0)) if self.gate is not None else 0.0
        xo = al * x + sg * uu
        xe = (A + se) * (sg * uu).abs() + 3 * U32 * ((al * x).abs() + xo.abs()) + 2.0 ** -126 * uu.abs()
        check(from_dev(r.x_out), n(xo), n(xe + 1e-37), "x_out")
        # what follows is computed from the x_out and the statistics that the kernel left, as it does itself
        xo, rb, ra = f(r.x_out), f(r.rb)[:, None], f(r.ra)[:, None]
        want_rb = (xo.square().mean(1, keepdim=True) + eps).rsqrt()
        check(n(rb), n(want_rb), n(A * want_rb), "rstd_pre")
        xh, yh = xo * rb, y * ra
        uu = yh * wa
        want = xh * wb
        check(from_dev(r.n), n(want), n((U16 + 4 * U32) * want.abs() + 1e-38), "n")
        g = f(self.dn) * wb
        prod = g * xh
        mb, mbe = prod.mean(1, keepdim=True), A * prod.abs().mean(1, keepdim=True)
        d = rb * (g - xh * mb)
        de = rb * (6 * U32 * (g.abs() + (xh * mb).abs()) + xh.abs() * mbe)
        if self.dres is not None:
            d = d + f(self.dres)
            de = de + 2 * U32 * (d.abs() + f(self.dres).abs())
        check(from_dev(r.dx), n(al * d), n(abs(al) * (de + U32 * d.abs()) + 1e-37), "dx")
        tiny = 2.0 ** -126
        if self.gate is not None:
            ds = d * uu * sg * (1 - sg)
            # 1 - sigmoid: its rounding where it is small is absolute
            dse = (de * uu.abs() + 8 * U32 * (d * uu).abs()) * sg * (1 - sg) + (d * uu).abs() * (sg * se * (1 - sg) + sg * (sg * se + U32) + tiny)
            check(from_dev(r.ds), n(ds), n(dse + u * (ds.abs() + dse) + 1e-37), "dgate")
        k, ke = d * sg, (de + (se + 2 * U32) * d.abs()) * sg + tiny * d.abs()
        g = k * wa
        prod = g * yh
        ma = prod.mean(1, keepdim=True)
        mae = A * prod.abs().mean(1, keepdim=True) + (ke * (wa * yh).abs()).mean(1, keepdim=True)
        dy = ra * (g - yh * ma)
        dye = ra * (ke * wa.abs() + 6 * U32 * (g.abs() + (yh * ma).abs()) + yh.abs() * mae)
        check(from_dev(r.dy), n(dy), n(dye + u * (dy.abs() + dye) + 1e-37), "dy")
        check(from_dev(r.dwa), n((k * yh).sum(0)), n((acc(T) + 4 * U32) * (k * yh).abs().sum(0) + (ke * yh.abs()).sum(0) + 1e-37), "dw_post")
        check(from_dev(r.dwb), n((f(self.dn) * xh).sum(0)), n((acc(T) + 4 * U32) * (f(self.dn) * xh).abs().sum(0) + 1e-37), "dw_pre")


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("gate", [True, False])
@pytest.mark.parametrize("T,h", [(1, 4), (1, 4096), (3, 36), (33, 64), (77, 1024), (200, 1028), (515, 260), (700, 4096), (160, 4100),
                                 (333, 5636), (310, 8192), (2500, 132), (1217, 8)])
def test_forward_and_gradients(T, h, gate, bf16):
    torch, mt = need_gpu()
    c = Case(torch, T, h, bf16, gate, T + h)
    c.check(c.run(mt))
    assert mt.mt_op_device_error() == 0


@pytest.mark.parametrize("T,h", [(40, 64), (300, 4096), (170, 8192)])
def test_without_residual_gradient_in_place_and_repeats(T, h):
    torch, mt = need_gpu()
    c = Case(torch, T, h, True, True, 5, resid=False)
    r = c.run(mt)
    c.check(r)
    c = Case(torch, T, h, True, True, 6)
    a = c.run(mt)
    b = c.run(mt, x_out=c.x.clone(), dx=c.dres.clone())
    for k in ("x_out", "n", "ra", "rb", "dx", "dy", "ds", "dwa", "dwb"):
        assert torch.equal(getattr(a, k), getattr(b, k)), k


def test_gates_at_their_ends_and_empty_rows():
    """Gates of +-inf and the types' ends open and close exactly; a row of zeros stays finite."""
    torch, mt = need_gpu()
    T, h = 6, 256
    c = Case(torch, T, h, False, True, 9)
    inf = float("inf")
    for i, v in enumerate((-inf, inf, -3e38, 3e38, -200.0, 200.0)):
        c.gate[i] = v
    c.y[3] = 0
    c.x[5] = 0
    r = c.run(mt)
    c.check(r)
    closed = torch.tensor([0, 2], device="cuda")
    assert torch.equal(r.x_out[closed], c.alpha * c.x[closed]) and not r.ds[closed].any() and not r.dy[closed].any()
    assert not r.ds[torch.tensor([1, 3], device="cuda")].any()
    # everything closed on a residual of zeros: n is zero
    c.gate[:] = -inf
    c.x[:] = 0
    r = c.run(mt)
    assert not r.x_out.any() and not r.n.float().any() and torch.isfinite(r.dx).all()


def test_rows_do_not_reach_each_other():
    torch, mt = need_gpu()
    c = Case(torch, 300, 512, True, True, 11)
    a = c.run(mt)
    c.y[17] = float("nan")
    c.x[170] = float("inf")
    b = c.run(mt)
    keep = torch.ones(300, dtype=torch.bool, device="cuda")
    keep[17] = keep[170] = False
    for k in ("x_out", "n", "ra", "rb", "dx", "dy", "ds"):
        assert torch.equal(getattr(a, k)[keep], getattr(b, k)[keep]), k
    assert torch.isnan(b.n[17].float()).all()


def test_gradient_against_differences():
    torch, mt = need_gpu()
    c = Case(torch, 20, 64, False, True, 13)
    r = c.run(mt)

    def total(x, y, s, wa, wb):
        yh = y * (y.square().mean(1, keepdim=True) + float(np.float32(c.eps))).rsqrt()
        xo = c.alpha * x + torch.sigmoid(s) * wa * yh
        nn = wb * xo * (xo.square().mean(1, keepdim=True) + float(np.float32(c.eps))).rsqrt()
        return (nn * c.dn.double() + xo * c.dres.double()).sum()
    base = [t.double() for t in (c.x, c.y, c.gate, c.wa, c.wb)]
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    for i, got in enumerate((r.dx, r.dy, r.ds, r.dwa, r.dwb)):
        d = torch.randn(base[i].shape, device="cuda", dtype=torch.float64, generator=g)
        lo, hi = list(base), list(base)
        lo[i], hi[i] = base[i] - 1e-5 * d, base[i] + 1e-5 * d
        num = float(total(*hi) - total(*lo)) / 2e-5
        mag = float((got.double() * d).abs().sum())
        assert abs(float((got.double() * d).sum()) - num) <= 1e-5 * mag


def test_offsets_past_32_bits():
    torch, mt = need_gpu()
    T, h = 540000, 4096
    one = Case(torch, 1, h, True, True, 15)
    code = mt.MT_BF16
    want = one.run(mt)
    x = torch.zeros((T, h), device="cuda")
    y = torch.zeros((T, h), device="cuda", dtype=torch.bfloat16)
    gate = torch.zeros_like(y)
    x[-1], y[-1], gate[-1] = one.x[0], one.y[0], one.gate[0]
    n, ra, rb = torch.empty_like(y), torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    mt.mt_op_sandwich_norm_fwd(x, y, gate, code, one.wa, one.wb, one.alpha, one.eps, x, n, ra, rb, T, h)
    assert torch.equal(x[-1], want.x_out[0]) and torch.equal(n[-1], want.n[0]) and not x[-2].any()
    dn, dres = torch.zeros((T, h), device="cuda"), torch.zeros((T, h), device="cuda")
    dn[-1], dres[-1] = one.dn[0], one.dres[0]
    dwa, dwb = torch.empty(h, device="cuda"), torch.empty(h, device="cuda")
    ws = torch.empty(mt.mt_op_sandwich_norm_bwd_workspace(T, h), device="cuda")
    dgate = torch.empty_like(gate)
    mt.mt_op_sandwich_norm_bwd(x, y, gate, code, one.wa, one.wb, one.alpha, ra, rb, dn, dres, dres, n, dgate, dwa, dwb, ws, T, h)
    assert torch.equal(dres[-1], want.dx[0]) and torch.equal(n[-1], want.dy[0]) and torch.equal(dgate[-1], want.ds[0])
    assert torch.equal(dwa, want.dwa) and torch.equal(dwb, want.dwb)
