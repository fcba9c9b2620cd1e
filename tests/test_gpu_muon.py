"""Orthogonalised matrices and the Muon step against float64.

Rounding operands to fp16 moves a result by an amount that depends on the
matrix: tests/muon_ref.py makes the same roundings in float64 and says how
much, before the kernel runs. The kernel may be off by twice that in norm (its
fp32 sums make some roundings fall the other way, each an error of the same
size and of its own sign), by three times the model's largest in any element,
plus the output's own rounding and 2^-20 for the sums."""
import numpy as np
import pytest

from tests import muon_ref as ref
from tests.bounds import U16, U32, check
from tests.gpu_util import from_dev, need_gpu

pytestmark = pytest.mark.gpu


def _matrix(torch, kind, b, rows, cols, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    n = lambda *s: torch.randn(s, device="cuda", generator=g)  # noqa: E731
    if kind == "flat":
        return n(b, rows, cols)
    if kind == "spikes":
        G = n(b, rows, cols)
        for i in range(6):
            G = G + 30.0 * 2.0 ** -i * n(b, rows, 1) * n(b, 1, cols)
        return G
    if kind == "low":  # of rank 4
        return n(b, rows, 4) @ n(b, 4, cols)
    e = n(b, 64, rows) * torch.exp(1.5 * n(b, 64, 1))
    return (e.mT @ (n(b, 64, cols) + n(b, 1, cols))) * 1e-6 + 1e-6 * n(b, rows, cols)


def _ortho(torch, mt, G, steps=5, coef=None, eps=0.0, out=None, o=None):
    b, rows, cols = G.shape
    out = out or torch.float32
    n = G.numel()
    raw = torch.full((n + 64,), float("nan"), device="cuda", dtype=out)
    O = raw[:n].view(G.shape) if o is None else o
    ws = torch.full((mt.mt_op_orthogonalize_workspace(b, rows, cols),), 0xff, dtype=torch.uint8, device="cuda")
    code = lambda t: mt.MT_F32 if t.dtype == torch.float32 else mt.MT_BF16  # noqa: E731
    mt.mt_op_orthogonalize(G, code(G), O, code(O), coef, steps, eps, ws, b, rows, cols)
    assert torch.isnan(raw[n:]).all()
    return O


def _check(torch, got, G, steps=5, coef=None, eps=0.0):
    want, model = ref.exact(G, steps, coef, eps), ref.rounded(G, steps, coef, eps)
    off = model - want
    u = U16 if got.dtype == torch.bfloat16 else U32
    for i in range(G.shape[0]):
        w, o, r = want[i], off[i], got[i].double()
        norm = float(w.norm())
        assert float((r - w).norm()) <= 2 * float(o.norm()) + u * norm + 2.0 ** -20 * norm, (float((r - w).norm()) / norm, float(o.norm()) / norm)
        big = 3 * float(o.abs().max()) + 2.0 ** -20 * float(w.abs().max())
        check(r.cpu().numpy(), w.cpu().numpy(), (u * (w.abs() + big) + big).cpu().numpy(), "O")


SHAPES = [(1, 1, 1), (1, 1, 9), (1, 7, 1), (2, 2, 3), (1, 33, 40), (3, 64, 64), (1, 100, 37), (2, 129, 257),
          (1, 300, 1000), (1, 777, 130), (5, 65, 520), (1, 1024, 1024), (2, 513, 2049), (1, 2600, 700), (1, 128, 2048),
          (1, 128, 2049), (2, 1500, 90), (40, 64, 256), (3, 20, 1100), (1, 2048, 127), (170, 30, 300), (1, 600, 128), (1, 100, 4096), (2, 3001, 64), (1, 2300, 128), (30, 16, 2500), (1, 60, 4097)]


@pytest.mark.parametrize("kind", ["flat", "spikes", "low", "gradient"])
@pytest.mark.parametrize("b,rows,cols", SHAPES)
def test_orthogonalize(b, rows, cols, kind):
    torch, mt = need_gpu()
    G = _matrix(torch, kind, b, rows, cols, rows + cols)
    _check(torch, _ortho(torch, mt, G), G)
    Gb = G.bfloat16()
    _check(torch, _ortho(torch, mt, Gb, out=torch.bfloat16), Gb)
    assert mt.mt_op_device_error() == 0


@pytest.mark.parametrize("b,rows,cols", [(1, 4096, 5000), (1, 5003, 4100), (12, 1536, 2048)])
def test_large_tiles(b, rows, cols):
    """Sizes whose products run on SM pairs, with ragged last tiles."""
    torch, mt = need_gpu()
    G = _matrix(torch, "gradient", b, rows, cols, 3)
    _check(torch, _ortho(torch, mt, G, out=torch.bfloat16), G)


@pytest.mark.parametrize("steps", [1, 2, 6, 12])
def test_steps_and_coefficients(steps):
    torch, mt = need_gpu()
    G = _matrix(torch, "spikes", 2, 96, 200, 7)
    cubic = [(1.5, -0.5, 0.0)] * steps
    _check(torch, _ortho(torch, mt, G, steps, cubic), G, steps, cubic)
    mixed = [(3.4445, -4.7750, 2.0315)] * (steps - 1) + [(1.875, -1.25, 0.375)]
    _check(torch, _ortho(torch, mt, G, steps, mixed), G, steps, mixed)


def test_known_results():
    """A row keeps its direction, and a scaled orthogonal matrix its vectors: all singular values are one number,
    which the scalar polynomial takes where it goes. fp16 rounding of the operands: a few 2^-12 a step."""
    torch, mt = need_gpu()

    def poly(s):
        for _ in range(5):
            s = 3.4445 * s - 4.7750 * s ** 3 + 2.0315 * s ** 5
        return s
    v = torch.randn((1, 1, 500), device="cuda")
    O = _ortho(torch, mt, v)
    assert torch.allclose(O.double(), poly(1.0) * v.double() / v.double().norm(), rtol=5 * 3.5 * 2.0 ** -12, atol=1e-6)
    Q = torch.linalg.qr(torch.randn((256, 256), device="cuda", dtype=torch.float64)).Q
    O = _ortho(torch, mt, (1e-3 * Q).float()[None].contiguous())[0].double()  # (QR gives columns first)
    assert float((O - poly(1 / 16) * Q).norm() / O.norm()) < 4e-3


@pytest.mark.parametrize("rows,cols", [(70, 90), (140, 200), (333, 150)])
def test_scale_eps_and_odd_matrices_of_a_batch(rows, cols):
    torch, mt = need_gpu()
    G = _matrix(torch, "gradient", 6, rows, cols, 9)
    plain = _ortho(torch, mt, G)
    for k in (2.0 ** -40, 2.0 ** 30):  # powers of two change nothing but the norm's own range
        assert torch.equal(_ortho(torch, mt, G * k), plain)
    _check(torch, _ortho(torch, mt, G, eps=float(G[0].norm())), G, eps=float(np.float32(float(G[0].norm()))))
    G[1] = 0
    G[2, 3, 4] = float("inf")
    G[3, -1, -1] = float("nan")
    G[4] *= 1e30
    got = _ortho(torch, mt, G)
    assert torch.equal(got[0], plain[0]) and torch.equal(got[5], plain[5])
    assert not got[1].any() and torch.isnan(got[2:5]).all()


@pytest.mark.parametrize("b,rows,cols", [(1, 1, 1 << 16), (1, 1 << 16, 3), (4096, 3, 2), (1, 130, 1 << 16), (1, 1 << 16, 200)])
def test_longest_sides_and_largest_batches(b, rows, cols):
    torch, mt = need_gpu()
    G = _matrix(torch, "gradient", b, rows, cols, 29)
    got = _ortho(torch, mt, G)
    if b > 8:
        at = torch.tensor([0, 1, b // 2, b - 1], device="cuda")
        G, got = G[at].contiguous(), got[at]
    _check(torch, got, G)


def test_in_place_and_repeats():
    torch, mt = need_gpu()
    for shape in ((2, 100, 300), (2, 300, 101), (2, 200, 300), (1, 700, 260)):
        G = _matrix(torch, "spikes", *shape, 11)
        want = _ortho(torch, mt, G)
        assert torch.equal(want, _ortho(torch, mt, G))
        o = G.clone()
        assert torch.equal(want, _ortho(torch, mt, o, o=o))


def test_values_off_any_boundary():
    torch, mt = need_gpu()
    for dt in (torch.float32, torch.bfloat16):
        G = _matrix(torch, "spikes", 1, 64, 72, 13).to(dt)
        raw = torch.empty(G.numel() + 1, device="cuda", dtype=dt)
        shifted = raw[1:].view(G.shape)
        shifted.copy_(G)
        out = torch.empty(G.numel() + 1, device="cuda", dtype=dt)[1:].view(G.shape)
        assert torch.equal(_ortho(torch, mt, shifted, o=out), _ortho(torch, mt, G, out=dt))
        # rows whose ends lie between two words, guards on both sides
        for rows, cols in ((130, 201), (700, 513), (150, 264)):
            G = _matrix(torch, "spikes", 1, rows, cols, 13).to(dt)
            raw = torch.full((G.numel() + 2,), 7.0, device="cuda", dtype=dt)
            out = raw[1:-1].view(G.shape)
            _ortho(torch, mt, G, o=out)
            assert torch.equal(out, _ortho(torch, mt, G, out=dt)) and raw[0] == 7 and raw[-1] == 7


@pytest.mark.parametrize("nesterov", [0, 1])
@pytest.mark.parametrize("wb,gb", [(False, False), (True, False), (True, True), (False, True)])
@pytest.mark.parametrize("b,rows,cols", [(1, 1, 5), (2, 129, 130), (1, 520, 264), (3, 40, 333), (2, 700, 100), (3, 64, 1536), (2, 131, 259),
                                         (1, 401, 6001), (1, 5003, 301), (3, 260, 140), (1, 2001, 1999)])
def test_update(b, rows, cols, wb, gb, nesterov):
    torch, mt = need_gpu()
    bf, f4 = torch.bfloat16, torch.float32
    G = _matrix(torch, "gradient", b, rows, cols, 17).to(bf if gb else f4)
    M = 3 * _matrix(torch, "gradient", b, rows, cols, 18)
    W = (0.02 * _matrix(torch, "flat", b, rows, cols, 19)).to(bf if wb else f4)
    M0, W0 = M.clone(), W.clone()
    mu, lr, wd, scale = 0.95, 0.01, 0.1, 0.2 * max(rows, cols) ** 0.5
    ws = torch.full((mt.mt_op_orthogonalize_workspace(b, rows, cols),), 0xff, dtype=torch.uint8, device="cuda")
    mt.mt_op_muon_update(W, mt.MT_BF16 if wb else mt.MT_F32, M, G, mt.MT_BF16 if gb else mt.MT_F32, mu, nesterov, lr, wd,
                         scale, None, 5, 1e-7, ws, b, rows, cols)
    mu32, eps32 = float(np.float32(mu)), float(np.float32(1e-7))
    want_M = mu32 * M0.double() + G.double()
    check(from_dev(M), want_M.cpu().numpy(), (U32 * want_M.abs() + 1e-45).cpu().numpy(), "M")
    U = G.double() + mu32 * want_M if nesterov else want_M
    X, off = ref.exact(U, 5, eps=eps32), None
    off = 3 * (ref.rounded(U, 5, eps=eps32) - X).abs().amax() + 2.0 ** -18 * X.abs().amax()
    keep, step = 1 - float(np.float32(lr)) * float(np.float32(wd)), float(np.float32(lr)) * float(np.float32(scale))
    want = keep * W0.double() - step * X
    u = U16 if wb else U32
    check(from_dev(W), want.cpu().numpy(), (step * off * (1 + u) + u * want.abs() + 4 * U32 * (W0.double().abs() + step * X.abs())).cpu().numpy(), "W")


def test_offsets_past_32_bits():
    """A batch of more than 2^31 values: its last matrix as it comes out alone."""
    torch, mt = need_gpu()
    b, rows, cols = 2200, 1000, 1000
    G = torch.randn((1, rows, cols), device="cuda").bfloat16().expand(b, rows, cols).contiguous()
    last = _matrix(torch, "gradient", 1, rows, cols, 23).bfloat16()
    G[-1] = last[0]
    O = _ortho(torch, mt, G, steps=2, o=G)
    _check(torch, O[-1:].clone(), last, 2)
    assert torch.equal(O[0], O[1500]) and torch.equal(O[0], O[-2])


@pytest.mark.parametrize("b,rows,cols", [(1, 128, 256), (2, 128, 260), (3, 97, 512), (1, 128, 1028), (1, 5, 2052), (2, 128, 4096)])
def test_one_launch_from_any_boundary(b, rows, cols):
    """Tensors that begin one value off take the way by rows: the same sums in the same order, so equal bits."""
    torch, mt = need_gpu()
    bf, f4 = torch.bfloat16, torch.float32

    def off(t):
        raw = torch.full((t.numel() + 2,), 7.0, device="cuda", dtype=t.dtype)
        raw[1:-1] = t.flatten()
        return raw, raw[1:-1].view(t.shape)

    for dt in (f4, bf):
        G = _matrix(torch, "gradient", b, rows, cols, 37).to(dt)
        M = 3 * _matrix(torch, "gradient", b, rows, cols, 38)
        W = (0.02 * _matrix(torch, "flat", b, rows, cols, 39)).to(dt)
        (_, g), (rm, m), (rw, w) = off(G), off(M), off(W)
        code = mt.MT_F32 if dt == f4 else mt.MT_BF16
        ws = torch.empty(mt.mt_op_orthogonalize_workspace(b, rows, cols), device="cuda", dtype=torch.uint8)
        mt.mt_op_muon_update(W, code, M, G, code, 0.9, 1, 0.01, 0.1, 1.0, None, 5, 1e-7, ws, b, rows, cols)
        mt.mt_op_muon_update(w, code, m, g, code, 0.9, 1, 0.01, 0.1, 1.0, None, 5, 1e-7, ws, b, rows, cols)
        assert torch.equal(m, M) and torch.equal(w, W)
        assert rm[0] == 7 and rm[-1] == 7 and rw[0] == 7 and rw[-1] == 7


@pytest.mark.parametrize("b,rows,cols", [(2, 128, 255), (1, 128, 257), (1, 127, 1027), (2, 128, 4095)])
def test_one_launch_of_odd_rows_in_place(b, rows, cols):
    torch, mt = need_gpu()
    G = _matrix(torch, "gradient", b, rows, cols, 41)
    want = _ortho(torch, mt, G)
    _check(torch, want, G)
    o = G.clone()
    assert torch.equal(want, _ortho(torch, mt, o, o=o))
    assert mt.mt_op_device_error() == 0
