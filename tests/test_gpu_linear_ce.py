"""Cross entropy from a head's inputs and weights against float64, element by
element. Inputs are the bf16 values themselves, so the products' terms are
exact and only their fp32 sums round: a logit is off by acc(h) sum |x w|, its
exponential by that much relative (plus a few 2^-24 of |z| for the arguments
and of the hardware's exponential), the gradients by one bf16 rounding of dz,
their own sums and their type's rounding."""
import numpy as np
import pytest

from tests.bounds import U16, U32, acc, check
from tests.gpu_util import from_dev, need_gpu

pytestmark = pytest.mark.gpu


def _case(torch, T, V, h, seed, ldx=None, ldw=None, spread=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    ldx, ldw = ldx or h, ldw or h
    X = torch.full((T, ldx), float("nan"), device="cuda", dtype=torch.bfloat16)
    W = torch.full((V, ldw), float("nan"), device="cuda", dtype=torch.bfloat16)
    X[:, :h] = torch.randn((T, h), device="cuda", generator=g) * spread
    W[:, :h] = torch.randn((V, h), device="cuda", generator=g) / h ** 0.5
    labels = torch.randint(0, V, (T,), device="cuda", generator=g).to(torch.int32)
    gl = torch.randn((T,), device="cuda", generator=g)
    return X, W, labels, gl


def _guarded(torch, shape, dtype, fill=float("nan")):
    """A tensor of NaN with 64 guard values behind it."""
    n = int(np.prod(shape))
    raw = torch.full((n + 64,), fill, device="cuda", dtype=dtype)
    return raw[:n].view(shape), raw[n:]


class Result:
    pass


def _run(torch, mt, X, W, labels, gl, scale, e, c, dxt=None, dwt=None, start=None):
    T, V, h = X.shape[0], W.shape[0], min(X.shape[1], W.shape[1])
    r = Result()
    ws = torch.full((mt.mt_op_linear_ce_fwd_workspace(T, V, h),), 0xff, dtype=torch.uint8, device="cuda")
    r.loss, g1 = _guarded(torch, (T,), torch.float32)
    r.lse, g2 = _guarded(torch, (T,), torch.float32)
    mt.mt_op_linear_ce_fwd(X, W, labels, scale, e, c, r.loss, r.lse, ws, T, V, h, X.stride(0), W.stride(0))
    assert torch.isnan(g1).all() and torch.isnan(g2).all()
    if dxt is not None or dwt is not None:
        code = {torch.float32: mt.MT_F32, torch.bfloat16: mt.MT_BF16, None: mt.MT_F32}
        wsb = torch.full((mt.mt_op_linear_ce_bwd_workspace(T, V, h),), 0xff, dtype=torch.uint8, device="cuda")
        r.dX = r.dW = None
        guards = []
        if dxt is not None:
            r.dX, g = _guarded(torch, (T, h), dxt)
            guards.append(g)
        if dwt is not None:
            r.dW, g = _guarded(torch, (V, h), dwt)
            guards.append(g)
            if start is not None:
                r.dW.copy_(start)
        mt.mt_op_linear_ce_bwd(X, W, labels, scale, e, c, r.lse, gl, r.dX, code[dxt], r.dW, code[dwt], start is not None,
                               wsb, T, V, h, X.stride(0), W.stride(0))
        assert all(torch.isnan(g).all() for g in guards)
    return r


def _reference(torch, X, W, labels, gl, scale, e, c, h):
    """The definition in float64 and the magnitudes that the bounds are made of."""
    f = Result()
    x, w = X[:, :h].double(), W[:, :h].double()
    V = W.shape[0]
    keep = (labels >= 0) & (labels < V)
    x = torch.where(keep[:, None], x, 0.0)
    lab = labels.long().clamp(0, V - 1)
    z = scale * x @ w.T
    zm = scale * (x.abs() @ w.abs().T)
    lse = torch.logsumexp(z, 1)
    p = torch.exp(z - lse[:, None])
    zy = z.gather(1, lab[:, None])[:, 0]
    f.lse = torch.where(keep, lse, 0.0)
    f.loss = torch.where(keep, lse - (1 - e) * zy - e * z.mean(1) + c * lse ** 2, 0.0)
    # logit error: the sum's, and two roundings of its scaling
    f.dz_logit = (acc(h) + 2 * U32) * zm + 1e-30
    top = f.dz_logit.max(1).values
    f.lse_err = top + 8 * U32 * (1 + lse.abs()) + acc(V)
    f.loss_err = f.lse_err * (1 + 2 * c * lse.abs()) + top + acc(V) * e * zm.mean(1) + 4 * U32 * (lse.abs() + zy.abs() + c * lse ** 2)
    g = torch.where(keep, gl.double(), 0.0)[:, None]
    k = (1 + 2 * c * lse)[:, None]
    oh = torch.zeros_like(p).scatter_(1, lab[:, None], 1.0)
    dz = g * (k * p - (1 - e) * oh - e / V)
    mag = g.abs() * (k.abs() * p + (1 - e) * oh + e / V)
    pe = g.abs() * k.abs() * p * (f.dz_logit + f.lse_err[:, None] + 4 * U32 * (z.abs() + lse.abs()[:, None]))
    # fp32 subnormals count as 0: a p below 2^-126 does, so |g k| 2^-126 is lost at most, and as much again where dz
    # itself ends below 2^-126
    tiny = 2.0 ** -126 * (g.abs() * k.abs() + 1)
    de = U16 * dz.abs() + (1 + U16) * (pe + 8 * U32 * mag) + tiny
    f.dX, f.dW = scale * dz @ w, scale * dz.T @ x
    f.dX_err = scale * (de @ w.abs() + (acc(V) + 2 * U32) * (mag @ w.abs()))
    f.dW_err = scale * (de.T @ x.abs() + (acc(X.shape[0]) + 2 * U32) * (mag.T @ x.abs()))
    return f


def _check(torch, r, f, start=None):
    n = lambda t: t.detach().double().cpu().numpy()  # noqa: E731
    check(n(r.lse), n(f.lse), n(f.lse_err), "lse")
    check(n(r.loss), n(f.loss), n(f.loss_err), "loss")
    if getattr(r, "dX", None) is not None:
        u = U16 if r.dX.dtype == torch.bfloat16 else U32
        check(from_dev(r.dX), n(f.dX), n(f.dX_err + u * (f.dX.abs() + f.dX_err)) + 1e-37, "dX")
    if getattr(r, "dW", None) is not None:
        u = U16 if r.dW.dtype == torch.bfloat16 else U32
        want = f.dW if start is None else f.dW + start.double()
        check(from_dev(r.dW), n(want), n(f.dW_err + u * (want.abs() + f.dW_err) + 2 * U32 * (want.abs() + f.dW.abs())) + 1e-37,
              "dW")


SHAPES = [(1, 1, 8), (1, 129, 64), (3, 5, 8), (127, 300, 72), (128, 256, 128), (129, 257, 40), (300, 1000, 200),
          (257, 4097, 64), (1000, 777, 136), (64, 33000, 64), (2049, 2500, 256)]


@pytest.mark.parametrize("T,V,h", SHAPES)
@pytest.mark.parametrize("e,c,scale", [(0.0, 0.0, 1.0), (0.1, 1e-2, 0.7)])
def test_loss_and_gradients(T, V, h, e, c, scale):
    torch, mt = need_gpu()
    X, W, labels, gl = _case(torch, T, V, h, T + V + h, spread=2.0)
    f = _reference(torch, X, W, labels, gl, scale, e, c, h)
    bf, f4 = torch.bfloat16, torch.float32
    for dxt, dwt in ((bf, f4), (f4, bf)):
        _check(torch, _run(torch, mt, X, W, labels, gl, scale, e, c, dxt, dwt), f)
    assert mt.mt_op_device_error() == 0


@pytest.mark.parametrize("bf16", [True, False])
def test_rows_that_are_not_scored_and_strides(bf16):
    torch, mt = need_gpu()
    T, V, h = 200, 515, 72
    X, W, labels, gl = _case(torch, T, V, h, 5, ldx=88, ldw=80)
    labels[::3] = -1
    labels[1] = -(1 << 31)
    X[::3] = float("nan")  # padding holds anything
    X[3] = float("inf")
    gl[::3] = float("nan")
    dt = torch.bfloat16 if bf16 else torch.float32
    start = torch.randn((V, h), device="cuda").to(dt)
    T_, V_ = X.shape[0], W.shape[0]
    r = Result()
    ws = torch.empty(mt.mt_op_linear_ce_fwd_workspace(T_, V_, h), dtype=torch.uint8, device="cuda")
    r.loss, r.lse = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    mt.mt_op_linear_ce_fwd(X, W, labels, 1.0, 0.1, 1e-3, r.loss, r.lse, ws, T, V, h, 88, 80)
    wsb = torch.full((mt.mt_op_linear_ce_bwd_workspace(T_, V_, h),), 0xff, dtype=torch.uint8, device="cuda")
    r.dX, r.dW = torch.empty((T, h), device="cuda", dtype=dt), start.clone()
    code = mt.MT_BF16 if bf16 else mt.MT_F32
    mt.mt_op_linear_ce_bwd(X, W, labels, 1.0, 0.1, 1e-3, r.lse, gl, r.dX, code, r.dW, code, 1, wsb, T, V, h, 88, 80)
    Xc = torch.where((labels >= 0)[:, None], X, torch.zeros_like(X))
    f = _reference(torch, Xc, W, labels, gl, 1.0, 0.1, 1e-3, h)
    _check(torch, r, f, start)
    assert (r.loss[labels < 0] == 0).all() and (r.lse[labels < 0] == 0).all() and (r.dX[labels < 0] == 0).all()
    # all rows masked: nothing but zeros, nothing added
    labels[:] = -1
    X[:] = float("nan")
    mt.mt_op_linear_ce_fwd(X, W, labels, 1.0, 0.1, 1e-3, r.loss, r.lse, ws, T, V, h, 88, 80)
    before = r.dW.clone()
    mt.mt_op_linear_ce_bwd(X, W, labels, 1.0, 0.1, 1e-3, r.lse, gl, r.dX, code, r.dW, code, 1, wsb, T, V, h, 88, 80)
    assert not r.loss.any() and not r.dX.any() and torch.equal(before, r.dW)
    assert mt.mt_op_device_error() == 0


def test_label_past_the_vocabulary():
    torch, mt = need_gpu()
    X, W, labels, gl = _case(torch, 40, 100, 64, 9)
    labels[7] = 100
    labels[8] = (1 << 31) - 1
    r = _run(torch, mt, X, W, labels, gl, 1.0, 0.0, 0.0, torch.float32, torch.float32)
    assert mt.mt_op_device_error() != 0
    bad = torch.zeros(40, dtype=torch.bool, device="cuda")
    bad[7:9] = True
    assert torch.isnan(r.loss[bad]).all() and torch.isnan(r.lse[bad]).all() and not r.dX[bad].any()
    labels[bad] = -1
    f = _reference(torch, X, W, labels, gl, 1.0, 0.0, 0.0, 64)
    r.loss[bad] = 0
    r.lse[bad] = 0
    _check(torch, r, f)


def test_a_bad_label_does_not_reach_the_calls_after_it():
    """Its bit waits in the device error word; later calls, with waits of many microseconds, run as ever."""
    torch, mt = need_gpu()
    X, W, labels, gl = _case(torch, 300, 9000, 8192, 61)
    bf = torch.bfloat16
    clean = _run(torch, mt, X, W, labels, gl, 1.0, 0.1, 1e-3, bf, bf)
    assert mt.mt_op_device_error() == 0
    bad = labels.clone()
    bad[0] = 9000
    _run(torch, mt, X, W, bad, gl, 1.0, 0.1, 1e-3)
    after = _run(torch, mt, X, W, labels, gl, 1.0, 0.1, 1e-3, bf, bf)
    for k in ("loss", "lse", "dX", "dW"):
        assert torch.equal(getattr(clean, k), getattr(after, k)), k
    assert mt.mt_op_device_error() != 0 and mt.mt_op_device_error() == 0


@pytest.mark.parametrize("which", ["dX", "dW"])
def test_one_gradient_alone_is_the_same(which):
    torch, mt = need_gpu()
    X, W, labels, gl = _case(torch, 300, 700, 64, 11)
    both = _run(torch, mt, X, W, labels, gl, 1.0, 0.0, 0.0, torch.bfloat16, torch.bfloat16)
    one = _run(torch, mt, X, W, labels, gl, 1.0, 0.0, 0.0, torch.bfloat16 if which == "dX" else None,
               torch.bfloat16 if which == "dW" else None)
    assert torch.equal(getattr(one, which), getattr(both, which))
    again = _run(torch, mt, X, W, labels, gl, 1.0, 0.0, 0.0, torch.bfloat16, torch.bfloat16)
    assert torch.equal(both.dX, again.dX) and torch.equal(both.dW, again.dW) and torch.equal(both.loss, again.loss)


@pytest.mark.parametrize("size", [60.0, 3000.0])
def test_large_logits(size):
    """Logits of hundreds and thousands: the sums stay finite, one column takes all."""
    torch, mt = need_gpu()
    X, W, labels, gl = _case(torch, 130, 600, 64, 21, spread=size)
    r = _run(torch, mt, X, W, labels, gl, 1.0, 0.0, 0.0, torch.float32, torch.float32)
    f = _reference(torch, X, W, labels, gl, 1.0, 0.0, 0.0, 64)
    _check(torch, r, f)


def test_infinite_logits_make_their_rows_nan():
    torch, mt = need_gpu()
    X, W, labels, gl = _case(torch, 130, 600, 64, 23)
    X[5, 3] = float("inf")
    X[9, 0] = float("nan")
    r = _run(torch, mt, X, W, labels, gl, 1.0, 0.0, 0.0)
    bad = torch.zeros(130, dtype=torch.bool, device="cuda")
    bad[5] = bad[9] = True
    assert torch.isnan(r.loss[bad]).all() and torch.isfinite(r.loss[~bad]).all()


def test_several_pieces_of_the_vocabulary():
    """2^28 / T columns a piece: 70000 tokens take 5000 columns in two."""
    torch, mt = need_gpu()
    T, V, h = 70000, 5000, 16
    X, W, labels, gl = _case(torch, T, V, h, 31)
    labels[::7] = -1
    assert mt.mt_op_linear_ce_bwd_workspace(T, V, h) < T * V * 2
    for dt in (torch.bfloat16, torch.float32):
        r = _run(torch, mt, X, W, labels, gl, 1.0, 0.1, 1e-3, dt, dt)
        f = _reference(torch, X, W, labels, gl, 1.0, 0.1, 1e-3, h)
        _check(torch, r, f)


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("T,V,h", [(3000, 300, 64), (130, 20000, 128), (5000, 200, 320)])
def test_sums_cut_into_ranges_and_added(T, V, h, bf16):
    """Few tiles and deep sums: partial sums, joined and added to what is there."""
    torch, mt = need_gpu()
    X, W, labels, gl = _case(torch, T, V, h, 71)
    labels[::5] = -1
    dt = torch.bfloat16 if bf16 else torch.float32
    start = torch.randn((V, h), device="cuda").to(dt)
    r = _run(torch, mt, X, W, labels, gl, 1.0, 0.0, 1e-3, dt, dt, start=start)
    f = _reference(torch, X, W, labels, gl, 1.0, 0.0, 1e-3, h)
    _check(torch, r, f, start)


@pytest.mark.parametrize("T,V,h", [(1 << 24, 200, 8), (3, 1 << 24, 8), (5, 70, 1 << 16)])
def test_largest_sizes(T, V, h):
    """The most rows, columns and depth that are taken, at rows picked from all over."""
    torch, mt = need_gpu()
    X, W, labels, gl = _case(torch, T, V, h, 81)
    ws = torch.empty(max(mt.mt_op_linear_ce_fwd_workspace(T, V, h), mt.mt_op_linear_ce_bwd_workspace(T, V, h)),
                     dtype=torch.uint8, device="cuda")
    loss, lse = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    dX, dW = torch.empty((T, h), device="cuda"), torch.empty((V, h), device="cuda")
    mt.mt_op_linear_ce_fwd(X, W, labels, 1.0, 0.0, 0.0, loss, lse, ws, T, V, h, h, h)
    mt.mt_op_linear_ce_bwd(X, W, labels, 1.0, 0.0, 0.0, lse, gl, dX, mt.MT_F32, dW, mt.MT_F32, 0, ws, T, V, h, h, h)
    at = torch.unique(torch.linspace(0, T - 1, 37, device="cuda").long())
    f = _reference(torch, X[at], W, labels[at], gl[at], 1.0, 0.0, 0.0, h)
    r = Result()
    r.loss, r.lse, r.dX = loss[at], lse[at], dX[at]
    _check(torch, r, f)
    # over the vocabulary a row's dz adds up to g (sum p - 1) = 0, so dW's rows do: up to dz's rounding, at most 2^-8 of
    # the magnitudes |g| (p + 1) |x|, and the fp32 sums
    total = dW.double().sum(0)
    mag = sum((2 * gl[i:i + (1 << 20)].double().abs()[:, None] * X[i:i + (1 << 20)].double().abs()).sum(0) for i in range(0, T, 1 << 20))
    assert bool((total.abs() <= (U16 * 1.1 + acc(T)) * mag).all())
    assert mt.mt_op_device_error() == 0


def test_gradient_against_differences():
    """Central differences of the float64 sum of the kernel's own losses' definition, by the direction of dX and dW."""
    torch, mt = need_gpu()
    T, V, h, e, c = 50, 333, 64, 0.1, 1e-2
    X, W, labels, gl = _case(torch, T, V, h, 41)
    r = _run(torch, mt, X, W, labels, gl, 1.0, e, c, torch.float32, torch.float32)

    def total(x, w):
        z = x @ w.T
        lse = torch.logsumexp(z, 1)
        return (gl.double() * (lse - (1 - e) * z.gather(1, labels.long()[:, None])[:, 0] - e * z.mean(1) + c * lse ** 2)).sum()

    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    for which, base in (("dX", X.double()), ("dW", W.double())):
        d = torch.randn(base.shape, device="cuda", dtype=torch.float64, generator=gen)
        s = 1e-4
        up, dn = base + s * d, base - s * d
        num = (total(up, W.double()) - total(dn, W.double())) if which == "dX" else (total(X.double(), up) - total(X.double(), dn))
        num = float(num) / (2 * s)
        got = getattr(r, which).double()
        # the kernel's rounding of dz: 2^-8 of its terms, of random sign over the elements
        assert abs(float((got * d).sum()) - num) <= 2.0 ** -7 * float((got.norm() * d.norm())) / d.numel() ** 0.5 * 8 + 1e-6


def test_offsets_past_32_bits():
    """dW of more than 2^31 values, rows at its end looked at."""
    torch, mt = need_gpu()
    T, V, h = 130, 160000, 16384
    X, W, labels, gl = _case(torch, T, V, h, 51)
    labels[3], labels[4] = V - 1, V - 2
    ws = torch.empty(max(mt.mt_op_linear_ce_fwd_workspace(T, V, h), mt.mt_op_linear_ce_bwd_workspace(T, V, h)),
                     dtype=torch.uint8, device="cuda")
    loss, lse, dW = torch.empty(T, device="cuda"), torch.empty(T, device="cuda"), torch.empty((V, h), device="cuda", dtype=torch.bfloat16)
    mt.mt_op_linear_ce_fwd(X, W, labels, 1.0, 0.0, 0.0, loss, lse, ws, T, V, h, h, h)
    mt.mt_op_linear_ce_bwd(X, W, labels, 1.0, 0.0, 0.0, lse, gl, None, mt.MT_F32, dW, mt.MT_BF16, 0, ws, T, V, h, h, h)
    x = X.double()
    rows = [0, V // 2, 131072, V - 2, V - 1]
    z = torch.cat([x.float() @ W[i:i + 20000].float().T for i in range(0, V, 20000)], 1).double()
    want_lse = torch.logsumexp(z, 1)
    assert torch.allclose(lse.double(), want_lse, rtol=2e-5)
    for v in rows:
        dz = gl.double() * (torch.exp(z[:, v] - want_lse) - (labels == v).double())
        want = dz @ x
        mag = (dz.abs()[:, None] * x.abs()).sum(0)
        check(from_dev(dW[v]), want.cpu().numpy(), ((U16 + 2e-4) * mag + U16 * 1.01 * want.abs() + 1e-30).cpu().numpy(), f"dW[{v}]")
