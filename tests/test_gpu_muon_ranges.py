"""Orthogonalised matrices at the ends of their ranges: singular values that
grow from step to step, updates far below fp32's squares, the accuracy that
the header states."""
import numpy as np
import pytest

from tests import muon_ref as ref
from tests.bounds import U32, check
from tests.gpu_util import need_gpu
from tests.test_gpu_muon import _check, _matrix, _ortho

pytestmark = pytest.mark.gpu

QUINTIC = ref.QUINTIC


def _eleven_bits(torch, x):
    """Rounded to fp16's 11 bits, without its range."""
    m, e = torch.frexp(x)
    return torch.ldexp(torch.round(m * 2048) / 2048, e)


def _wide_range(torch, G, steps, coef):
    """tests/muon_ref.py's `rounded` with the square matrices' fp16 taken as 11 bits of any exponent."""
    X, flip = (G.double(), False) if G.shape[-2] <= G.shape[-1] else (G.double().mT, True)
    X = X / X.flatten(-2).norm(dim=-1)[..., None, None]
    r = lambda x: _eleven_bits(torch, x)  # noqa: E731
    off = 1 - torch.eye(X.shape[-2], dtype=torch.float64, device=X.device)
    hi = r(X)
    lo = r(X - hi)
    for a, b, c in [[float(np.float32(v)) for v in row] for row in coef]:
        A = hi @ hi.mT
        d = A.diagonal(dim1=-2, dim2=-1)
        O = r(A * off)
        B = b * O + c * (O @ O + (d[..., :, None] + d[..., None, :]) * O)
        db = b * d + c * (d * d + (O @ O).diagonal(dim1=-2, dim2=-1))
        X = (a + db)[..., None] * hi + (a + db / 2)[..., None] * lo + r(B * off) @ hi
        hi = r(X)
        lo = r(X - hi)
    return X.mT if flip else X


SIZES = [(2, 4, 6), (1, 100, 300), (2, 300, 90), (3, 60, 2000), (1, 300, 400), (2, 700, 260), (1, 2048, 2600), (1, 5003, 4100)]
GROW = {"5": [(5.0, 0.0, 0.0), QUINTIC], "8": [(8.0, 0.0, 0.0), QUINTIC], "12": [(12.0, 0.0, 0.0), QUINTIC],
        "steep": [(2.0, 0.0, 0.0), (3.0, -50.0, 100.0)], "back": [(12.0, 0.0, 0.0), (4.0, -0.07, 0.0003), (0.1, 0.0, 0.0)],
        "most": [(14.5, 0.0, 0.0), (100.0, 100.0, 100.0)]}


@pytest.mark.parametrize("name", GROW)
@pytest.mark.parametrize("b,rows,cols", SIZES)
@pytest.mark.parametrize("rank", [1, 3])
def test_singular_values_up_to_the_limit(b, rows, cols, name, rank):
    """Singular values below 15 before a step whose b A + c A A is far larger. fp16 of a power-of-two scale is 11 bits
    down to 2^-24 of the largest value that it has to hold, which is of no account beside these."""
    torch, mt = need_gpu()
    g = torch.Generator(device="cuda")
    g.manual_seed(rows + cols + rank)
    n = lambda *s: torch.randn(s, device="cuda", generator=g)  # noqa: E731
    G = n(b, rows, rank) @ n(b, rank, cols)
    coef = GROW[name]
    want = ref.exact(G, len(coef), coef)
    off = _wide_range(torch, G, len(coef), coef) - want
    got = _ortho(torch, mt, G, len(coef), coef).double()
    for i in range(b):
        w, o, r = want[i], off[i], got[i]
        norm = float(w.norm())
        # Twice the model's error in norm, three times its largest in an element, and the sums': the tensor core cuts its
        # sums, a running sum loses up to a unit, 2^-23 of itself, at each of K / 16 instructions and their products as much
        # again. A step goes through A twice (the long side), A A and B X (the short one). The terms a s, b s^3, c s^5
        # partly cancel.
        terms, s = norm, 1.0
        for ca, cb, cc in coef[:2]:
            terms = max(terms, rank ** 0.5 * (abs(ca) * s + abs(cb) * s ** 3 + abs(cc) * s ** 5))
            s = max(s, abs(ca * s))
        terms *= (2 * max(rows, cols) + 2 * min(rows, cols) + 64) / 16 * 2.0 ** -22
        assert float((r - w).norm()) <= 2 * float(o.norm()) + U32 * norm + terms, (float((r - w).norm()) / norm, float(o.norm()) / norm)
        big = 3 * float(o.abs().max()) + terms
        check(r.cpu().numpy(), w.cpu().numpy(), (U32 * w.abs() + big).cpu().numpy(), "O")
    assert mt.mt_op_device_error() == 0


@pytest.mark.parametrize("b,rows,cols", SIZES)
def test_past_the_limit_is_right_or_not_finite(b, rows, cols):
    """A singular value of 60: either the result holds, or it says so by infinities and NaN; another matrix of the batch
    is not touched."""
    torch, mt = need_gpu()
    G = _matrix(torch, "flat", b + 1, rows, cols, 5)
    low = _matrix(torch, "low", 1, rows, cols, 6)[:, :, :1] @ _matrix(torch, "flat", 1, 1, cols, 7)
    G[0] = low[0]
    coef = [(60.0, 0.0, 0.0), QUINTIC]
    got = _ortho(torch, mt, G, 2, coef)
    if bool(torch.isfinite(got[0]).all()):
        want = ref.exact(G[:1], 2, coef)
        assert float((got[:1].double() - want).norm()) <= 1e-2 * float(want.norm())
    if rows >= 60:  # flat ones have no singular value anywhere near 1
        mild = [(6.0, 0.0, 0.0), QUINTIC]
        before = _ortho(torch, mt, G, 2, mild)
        G[0, 0, 0] = float("inf")
        after = _ortho(torch, mt, G, 2, mild)
        assert torch.equal(after[1:], before[1:]) and torch.isnan(after[0]).all()


@pytest.mark.parametrize("eps", [0.0, 1e-45, 1e-40, 1e-37, 1e-30, 1e-7, 1e30])
@pytest.mark.parametrize("b,rows,cols", [(3, 20, 30), (2, 90, 1000), (3, 300, 200), (2, 140, 333)])
def test_zero_matrices_are_zero_for_any_eps(b, rows, cols, eps):
    torch, mt = need_gpu()
    G = torch.zeros((b, rows, cols), device="cuda")
    assert not _ortho(torch, mt, G, eps=eps).any()
    W, M = torch.ones_like(G), torch.zeros_like(G)
    ws = torch.empty(mt.mt_op_orthogonalize_workspace(b, rows, cols), dtype=torch.uint8, device="cuda")
    mt.mt_op_muon_update(W, mt.MT_F32, M, G, mt.MT_F32, 0.9, 1, 0.5, 0.0, 1.0, None, 5, eps, ws, b, rows, cols)
    assert bool((W == 1).all()) and not M.any()


@pytest.mark.parametrize("size", [1e-18, 1e-20, 1e-22, 1e-26, 1e-32, 1e-35])
@pytest.mark.parametrize("b,rows,cols", [(3, 20, 30), (2, 90, 1000), (2, 200, 60), (3, 300, 200), (2, 140, 333), (1, 257, 1024)])
def test_small_updates_are_scaled_to_norm_one(b, rows, cols, size):
    """Their squares lie among fp32's subnormals or below all of them."""
    torch, mt = need_gpu()
    G = _matrix(torch, "flat", b, rows, cols, 3) * size
    _check(torch, _ortho(torch, mt, G), G)
    Gb = G.bfloat16()
    _check(torch, _ortho(torch, mt, Gb), Gb)
    eps = float(np.float32(3 * size))
    _check(torch, _ortho(torch, mt, G, eps=eps), G, eps=eps)
    k = 2.0 ** 40
    assert torch.equal(_ortho(torch, mt, G * k), _ortho(torch, mt, (G * k) * 2.0 ** 20))


@pytest.mark.parametrize("steps,full,ranks", [(5, 1.6e-3, 0.7), (6, 2e-3, 1.4)])
@pytest.mark.parametrize("kind", ["flat", "spikes", "gradient", 1, 2, 4])
@pytest.mark.parametrize("b,rows,cols", [(8, 16, 64), (4, 64, 64), (1, 4096, 64), (3, 100, 1001), (2, 300, 1000), (1, 1024, 1024),
                                         (2, 700, 260), (1, 5003, 4100)])
def test_accuracy_as_stated(b, rows, cols, kind, steps, full, ranks):
    """Of full rank within `full`; of rank 1 to 4 within ranks / m as well: what the first step's rounding leaves in the
    other directions grows by 3.44 a step. Few directions also feel the sums' cutting, 2^-23 K / 16 of each product: four
    products a step, c s^5 up to 5 times what a s + b s^3 leave of it, and the next steps take a relative error up to 5
    times as far (s p'(s) / p(s) at 1.2, the top of the quintic's range) and then about as it is twice: 20 (1 + 5 + 5)."""
    torch, mt = need_gpu()
    if isinstance(kind, str):
        G = _matrix(torch, kind, b, rows, cols, 51)
    else:
        g = torch.Generator(device="cuda")
        g.manual_seed(51 + kind)
        G = torch.randn((b, rows, kind), device="cuda", generator=g) @ torch.randn((b, kind, cols), device="cuda", generator=g)
        full = max(full, ranks / min(rows, cols)) + 220 * max(rows, cols) / 16 * 2.0 ** -23
    got, want = _ortho(torch, mt, G, steps).double(), ref.exact(G, steps)
    rel = (got - want).flatten(1).norm(dim=1) / want.flatten(1).norm(dim=1)
    assert bool((rel <= full).all()), rel
