"""The gate's gradient at open and closed gates relative to its own size, and
rows whose bits do not depend on how many there are."""
import pytest

from tests.bounds import U16, U32, acc, check
from tests.gpu_util import from_dev, need_gpu
from tests.test_gpu_sandwich_norm import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("T,h", [(170, 256), (40, 4096), (33, 5636), (21, 8192)])
def test_gate_gradients_keep_their_own_size(T, h, bf16):
    """dgate = d u s (1 - s) for gates from -80 to 80: s and 1 - s are each e^-|gate| where they are small, whose relative
    error is the exponential's (2^-22, and its argument's rounding, |gate| 2^-23) and the reciprocal's."""
    torch, mt = need_gpu()
    c = Case(torch, T, h, bf16, True, T + h)
    c.gate = torch.linspace(-80, 80, T * h, device="cuda")[torch.randperm(T * h, device="cuda")].view(T, h).to(c.dt)
    r = c.run(mt)
    f = lambda t: t.double()  # noqa: E731
    xo, ra, rb, y, s = f(r.x_out), f(r.ra)[:, None], f(r.rb)[:, None], f(c.y), f(c.gate)
    u = y * ra * f(c.wa)
    xh = xo * rb
    g = f(c.dn) * f(c.wb)
    prod = g * xh
    mb = prod.mean(1, keepdim=True)
    d = rb * (g - xh * mb) + f(c.dres)
    de = rb * (6 * U32 * (g.abs() + (xh * mb).abs()) + xh.abs() * (acc(h) + 8 * U32) * prod.abs().mean(1, keepdim=True)) \
        + 2 * U32 * (d.abs() + f(c.dres).abs())
    ss = torch.sigmoid(s) * torch.sigmoid(-s)
    want = d * u * ss
    rel = 16 * U32 + 4 * U32 * s.abs()
    e = (de * u.abs() + (rel + 8 * U32) * (d * u).abs()) * ss
    n = lambda t: t.cpu().numpy()  # noqa: E731
    check(from_dev(r.ds), n(want), n(e + (U16 if bf16 else U32) * (want.abs() + e) + 1e-37), "dgate")


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("gate", [True, False])
@pytest.mark.parametrize("h", [4, 36, 260, 1024, 1028, 2052, 4092, 4096, 5636, 8192])
def test_a_rows_bits_do_not_depend_on_the_others(h, gate, bf16):
    torch, mt = need_gpu()
    T = 700
    c = Case(torch, T, h, bf16, gate, h)
    code = mt.MT_BF16 if bf16 else mt.MT_F32

    def fwd(t):
        xo, n, ra, rb = torch.empty_like(c.x[:t]), torch.empty((t, h), device="cuda", dtype=torch.bfloat16), *torch.empty((2, t), device="cuda")
        mt.mt_op_sandwich_norm_fwd(c.x, c.y, c.gate, code, c.wa, c.wb, c.alpha, c.eps, xo, n, ra, rb, t, h)
        return xo, n, ra, rb

    full = fwd(T)
    for t in (1, 33, 304, 305):
        for a, b in zip(fwd(t), full):
            assert torch.equal(a, b[:t]), t
