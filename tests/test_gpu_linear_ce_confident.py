"""Cross entropy from a head's inputs where the label holds nearly all of the
probability, and logits far past ordinary ones.

The gradients of the logits are read off dX: beside random columns W has an
identity, X zeros there, so dX's columns there are dz itself (one term a sum)."""
import pytest

from tests.bounds import U16, U32, check
from tests.gpu_util import need_gpu
from tests.test_gpu_linear_ce import _case, _check, _reference, _run

pytestmark = pytest.mark.gpu


def _confident(torch, T, V, h, seed, shift):
    """Rows whose label's probability is 1 - q, q from 1e-2 to 1e-6; all logits moved by `shift`, exactly."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    n = lambda *s: torch.randn(s, device="cuda", generator=g)  # noqa: E731
    wide = h - V - 8
    X = torch.zeros((T, h), device="cuda", dtype=torch.bfloat16)
    W = torch.zeros((V, h), device="cuda", dtype=torch.bfloat16)
    W[:, :wide] = n(V, wide) / wide ** 0.5
    W[:, wide] = 1.0
    W[:, wide + 8:] = torch.eye(V, device="cuda")
    labels = torch.randint(0, V, (T,), device="cuda", generator=g).to(torch.int32)
    q = 10.0 ** torch.linspace(-2, -6, T, device="cuda")
    X[:, :wide] = n(T, wide) + torch.log(1.65 * V / q)[:, None] * W[labels.long(), :wide].float()
    X[:, wide] = shift
    return X, W, labels, torch.rand(T, device="cuda", generator=g) + 0.5


CONFIDENT = [(300, 256, 4096 + 264), (100, 128, 1024 + 136), (1200, 4096, 8192), (700, 5000, 16384)]


def _definition(torch, X, W, labels):
    """In float64: logits, the label's, log-sum-exp, probabilities, q = 1 - p of the label without a difference of near ones."""
    z = X.double() @ W.double().T
    at = labels.long()[:, None]
    lse = torch.logsumexp(z, 1)
    p = torch.exp(z - lse[:, None])
    q = p.scatter(1, at, 0.0).sum(1)
    assert float(q.max()) > 5e-3 and float(q.min()) < 2e-6
    return z, at, z.gather(1, at)[:, 0], lse, p, q


def _logit_error(h):
    """A logit of the products is off by at most a step of the largest partial sum (below 32) lost at each of the h / 16
    additions; that moves q by up to twice as much of itself."""
    return (h / 16 + 16) * 2.0 ** -23 * 32


@pytest.mark.parametrize("e,c", [(0.0, 0.0), (0.1, 1e-3)])
@pytest.mark.parametrize("T,V,h", CONFIDENT)
@pytest.mark.parametrize("shift", [0.0, -14.0, -30.0])
def test_losses_of_confident_tokens(T, V, h, shift, e, c):
    """A loss of 1e-6 is as good, relative to itself, as one of 1: it is not a difference of two logits."""
    torch, mt = need_gpu()
    X, W, labels, gl = _confident(torch, T, V, h, T + V, shift)
    r = _run(torch, mt, X, W, labels, gl, 1.0, e, c)
    z, at, zy, lse, p, q = _definition(torch, X, W, labels)
    loss = -torch.log1p(-q) + e * (zy - z.mean(1)) + c * lse ** 2
    n = lambda t: t.double().cpu().numpy()  # noqa: E731
    E = _logit_error(h)
    mag = e * z.abs().mean(1) + (e > 0) * (zy.abs() + c * lse ** 2)
    check(n(r.loss), n(loss), n(2 * E * (-torch.log1p(-q) + e + 2 * c * lse.abs()) + 2.0 ** -17 * mag + 2.0 ** -40), "loss")
    check(n(r.lse), n(lse), n(2 * E + 8 * U32 * lse.abs()), "lse")


@pytest.mark.parametrize("e,c", [(0.0, 0.0), (0.1, 1e-3)])
@pytest.mark.parametrize("T,V,h", CONFIDENT)
@pytest.mark.parametrize("shift", [0.0, -14.0, -30.0])
def test_gradients_of_confident_tokens(T, V, h, shift, e, c):
    """dz of the label keeps its own size's accuracy. q moves with the products' errors, 2 E of itself; beside that the
    label's dz knows lse to a rounding (2^-24 of |lse|) and the hardware's exponential to 2^-22: nothing that grows with
    h is left of p. dz is rounded to bf16."""
    torch, mt = need_gpu()
    X, W, labels, gl = _confident(torch, T, V, h, T + V, shift)
    r = _run(torch, mt, X, W, labels, gl, 1.0, e, c, torch.float32, torch.float32)
    z, at, zy, lse, p, q = _definition(torch, X, W, labels)
    n = lambda t: t.double().cpu().numpy()  # noqa: E731
    E = _logit_error(h)
    k = 1 + 2 * c * lse
    dz = p * k[:, None] - e / V
    by_label = k - 1 + e - k * q - e / V  # k p - (1 - e) - e / V
    dz = gl.double()[:, None] * dz.scatter(1, at, by_label[:, None])
    pe = p * (2 * E + 8 * U32 * (lse.abs()[:, None] + z.abs()) + 2.0 ** -21)
    pe = pe.scatter(1, at, (2 * E * q + 1.01 * U32 * lse.abs() + 2.0 ** -21)[:, None])
    mag = p * k[:, None] + e / V + torch.zeros_like(p).scatter(1, at, 1 - e)
    de = gl.double().abs()[:, None] * (k[:, None] * pe + (e > 0) * (8 * U32 + 4 * c * E) * mag)
    check(n(r.dX[:, h - V:]), n(dz), n(U16 * dz.abs() + (1 + U16) * de + 1e-37), "dz")
    assert mt.mt_op_device_error() == 0


@pytest.mark.parametrize("T,V,h", CONFIDENT)
def test_log_sum_exp_of_confident_tokens_leans_to_no_side(T, V, h):
    """It is the label's logit there, a tree of fp32 sums whose roundings have no sign of their own (the products' have:
    1e-6 of it and more). A mean over the rows is off by less than 2^-22 of it, eight single roundings' mean size."""
    torch, mt = need_gpu()
    X, W, labels, gl = _confident(torch, T, V, h, T + V, 0.0)
    r = _run(torch, mt, X, W, labels, gl, 1.0, 0.0, 0.0)
    lse = _definition(torch, X, W, labels)[3]
    assert abs(float((r.lse.double() - lse).mean())) <= 2.0 ** -22 * float(lse.abs().mean())


def _far(torch, V, sign, size, scale):
    """Logits of `size`: the label's is the largest by far, with sign -1 in every other row the lowest."""
    X, W, labels, gl = _case(torch, 400, V, 64, 77, spread=1.0)
    w = W[labels.long()].float()
    X[:, :] = sign * (w / w.square().sum(1, keepdim=True) + 1e-3 * X.float()) * (size / scale) * (0.5 + torch.rand(400, 1, device="cuda"))
    X[::2] = -X[::2] if sign < 0 and V > 1 else X[::2]
    return X, W, labels, gl


@pytest.mark.parametrize("scale", [0.7, 1.0, 30.0, 1e6])
@pytest.mark.parametrize("size", [1e5, 1e6, 1e7, 1e8, 3e9, 1e13])
@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("V", [1, 2, 300])
def test_losses_of_logits_of_any_size(V, sign, size, scale):
    """Finite logits give finite losses of at least 0, whatever the sums' rounding."""
    torch, mt = need_gpu()
    X, W, labels, gl = _far(torch, V, sign, size, scale)
    r = _run(torch, mt, X, W, labels, gl, scale, 0.0, 0.0)
    assert torch.isfinite(r.loss).all() and torch.isfinite(r.lse).all()
    assert bool((r.loss >= 0).all())
    _check(torch, r, _reference(torch, X, W, labels, gl, scale, 0.0, 0.0, 64))
    assert V > 1 or not r.loss.any()


@pytest.mark.parametrize("scale", [0.7, 1.0, 30.0, 1e6])
@pytest.mark.parametrize("size", [1e5, 1e6, 1e7, 1e8, 3e9, 1e13])
@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("V", [1, 2, 300])
def test_gradients_of_logits_of_any_size(V, sign, size, scale):
    """Probabilities of at most 1, whatever the sums' rounding."""
    torch, mt = need_gpu()
    X, W, labels, gl = _far(torch, V, sign, size, scale)
    r = _run(torch, mt, X, W, labels, gl, scale, 0.0, 0.0, torch.float32, torch.float32)
    most = 1.02 * scale * (V + 1) * gl.abs()[:, None] * W.float().abs().amax(0)[None]  # |dz_j| <= |g| (p_j + [label])
    assert bool((r.dX.abs() <= most).all()) and torch.isfinite(r.dW).all()
    assert V > 1 or not (r.dX.any() or r.dW.any())
    assert mt.mt_op_device_error() == 0


def test_one_infinite_logit():
    """Rows with an infinite logit have no finite loss, the others keep theirs."""
    torch, mt = need_gpu()
    inf = float("inf")
    X, W, labels, gl = _case(torch, 6, 40, 64, 3)
    labels[:] = 7
    X[:, 0] = 0
    W[:, 0] = 0
    W[7, 0] = 1.0
    X[1, 0], X[2, 0] = inf, -inf
    r = _run(torch, mt, X, W, labels, gl, 1.0, 0.0, 0.0)
    assert torch.isnan(r.loss[1:3]).all() and torch.isfinite(r.loss[[0, 3, 4, 5]]).all()
    # one class: its logit alone
    X, W, labels, gl = _case(torch, 6, 1, 64, 3)
    W[:] = 1.0
    X[1, 0], X[2, 0] = inf, -inf
    r = _run(torch, mt, X, W, labels, gl, 1.0, 0.0, 0.0)
    assert torch.isnan(r.loss[1:3]).all() and not r.loss[[0, 3, 4, 5]].any()
    # two classes of which the label's is -inf
    X, W, labels, gl = _case(torch, 6, 2, 64, 3)
    labels[:] = 0
    W[0], W[1] = -1.0, 1.0
    X[2] = 1.0
    X[2, 0] = 3e38
    X[2, 1] = 3e38
    r = _run(torch, mt, X, W, labels, gl, 1.0, 0.0, 0.0)
    assert not torch.isfinite(r.loss[2]) and torch.isfinite(r.loss[[0, 1, 3, 4, 5]]).all()


@pytest.mark.parametrize("bf16", [True, False])
def test_several_pieces_added_and_one_gradient_alone(bf16):
    torch, mt = need_gpu()
    T, V, h = 70000, 5000, 16
    X, W, labels, gl = _case(torch, T, V, h, 33)
    labels[::7] = -1
    X[::7] = float("nan")
    dt = torch.bfloat16 if bf16 else torch.float32
    start = torch.randn((V, h), device="cuda").to(dt)
    both = _run(torch, mt, X, W, labels, gl, 1.0, 0.1, 1e-3, dt, dt, start=start)
    Xc = torch.where((labels >= 0)[:, None], X, torch.zeros_like(X))
    _check(torch, both, _reference(torch, Xc, W, labels, gl, 1.0, 0.1, 1e-3, h), start)
    assert torch.equal(_run(torch, mt, X, W, labels, gl, 1.0, 0.1, 1e-3, dt, None).dX, both.dX)
    assert torch.equal(_run(torch, mt, X, W, labels, gl, 1.0, 0.1, 1e-3, None, dt, start=start).dW, both.dW)


def test_gradient_against_differences_of_the_definition():
    """As close as dz's rounding allows: an error of at most U16 dz in each, in no particular direction, so that six of
    their joint standard deviations (U16 / sqrt(3) each) hold."""
    torch, mt = need_gpu()
    T, V, h, e, c = 50, 333, 64, 0.1, 1e-2
    X, W, labels, gl = _case(torch, T, V, h, 43)
    r = _run(torch, mt, X, W, labels, gl, 1.0, e, c, torch.float32, torch.float32)
    x, w, g = X.double(), W.double(), gl.double()
    at = labels.long()[:, None]

    def total(x, w):
        z = x @ w.T
        lse = torch.logsumexp(z, 1)
        return (g * (lse - (1 - e) * z.gather(1, at)[:, 0] - e * z.mean(1) + c * lse ** 2)).sum()

    z = x @ w.T
    lse = torch.logsumexp(z, 1)
    dz = torch.exp(z - lse[:, None]) * (1 + 2 * c * lse)[:, None] - e / V
    dz = g[:, None] * (dz - torch.zeros_like(z).scatter_(1, at, 1 - e))
    gen = torch.Generator(device="cuda")
    gen.manual_seed(5)
    for k in range(4):
        for which, base in (("dX", x), ("dW", w)):
            d = torch.randn(base.shape, device="cuda", dtype=torch.float64, generator=gen)
            s = 1e-5
            num = (total(x + s * d, w) - total(x - s * d, w)) if which == "dX" else (total(x, w + s * d) - total(x, w - s * d))
            num = float(num) / (2 * s)
            along = (d @ w.T) if which == "dX" else (x @ d.T)
            sd = float((dz * along).norm()) * U16 / 3 ** 0.5
            got = float((getattr(r, which).double() * d).sum())
            # differences: s^2 times the third derivative, and 1e-16 of the sums over s
            assert abs(got - num) <= 6 * sd + 4e-6 * float((dz * along).abs().sum()), (which, got, num, sd)
