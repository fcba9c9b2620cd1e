"""Newton-Schulz steps in float64: exactly, and with the roundings that the
kernels make (fp16 operands with scales 2^10 and 2^8, X as hi + lo, diagonals
apart), which says how far those roundings take a given matrix."""
import torch

QUINTIC = (3.4445, -4.7750, 2.0315)


def _coefs(coef, steps):
    c = [QUINTIC] * steps if coef is None else coef
    return [[float(torch.tensor(v, dtype=torch.float32)) for v in row] for row in c]


def _wide(G):
    return (G, False) if G.shape[-2] <= G.shape[-1] else (G.mT, True)


def exact(G, steps, coef=None, eps=0.0):
    X, flip = _wide(G.double())
    X = X / (X.flatten(-2).norm(dim=-1)[..., None, None] + eps)
    for a, b, c in _coefs(coef, steps):
        A = X @ X.mT
        X = a * X + (b * A + c * A @ A) @ X
    return X.mT if flip else X


def _fp16(x, scale):
    return (x * scale).to(torch.float16).double() / scale


def rounded(G, steps, coef=None, eps=0.0):
    X, flip = _wide(G.double())
    X = X / (X.flatten(-2).norm(dim=-1)[..., None, None] + eps)

    def pair(x):
        hi = _fp16(x, 1024)
        return hi, _fp16(x - hi, 1024)

    off = 1 - torch.eye(X.shape[-2], dtype=torch.float64, device=X.device)
    hi, lo = pair(X)
    for i, (a, b, c) in enumerate(_coefs(coef, steps)):
        A = hi @ hi.mT
        d = A.diagonal(dim1=-2, dim2=-1)
        O = _fp16(A * off, 256)
        B = b * O + c * (O @ O + (d[..., :, None] + d[..., None, :]) * O)
        db = b * d + c * (d * d + (O @ O).diagonal(dim1=-2, dim2=-1))
        B = _fp16(B * off, 256)
        X = (a + db)[..., None] * hi + (a + db / 2)[..., None] * lo + B @ hi
        hi, lo = pair(X)
    return X.mT if flip else X
