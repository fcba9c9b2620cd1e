"""The dense decoder step in float64 with the residual checkpoints rounded to
their 8-bit form below the top block (no GPU): each of those blocks is run
again from its rounded input, and its gradients are those of that second run
under the gradient that arrives from above."""
from __future__ import annotations

import numpy as np
import torch

import oracle
from tests import ckpt8_ref as ref


def _norm(x, w, eps):
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + eps) * w


def _rope(x, theta):  # [B, S, heads, d], pairs (i, i + d/2)
    S, d = x.shape[1], x.shape[3]
    a = torch.arange(S, dtype=torch.float64)[:, None] * theta ** (-2.0 * torch.arange(d // 2, dtype=torch.float64) / d)
    c, s = torch.cos(a)[None, :, None], torch.sin(a)[None, :, None]
    lo, hi = x[..., :d // 2], x[..., d // 2:]
    return torch.cat([lo * c - hi * s, lo * s + hi * c], -1)


def _layer(cfg, p, l, x):  # x [B, S, h]
    B, S, _ = x.shape
    n = lambda k: p[f"layer{l}.{k}"]
    a = _norm(x, n("w_attn_norm"), cfg.norm_eps)
    heads = lambda w, k: (a @ w.T).view(B, S, k, cfg.head_dim)
    q = _rope(heads(n("wq"), cfg.n_heads), cfg.rope_theta)
    k = _rope(heads(n("wk"), cfg.n_kv_heads), cfg.rope_theta)
    v = heads(n("wv"), cfg.n_kv_heads)
    g = cfg.n_heads // cfg.n_kv_heads
    k, v = k.repeat_interleave(g, 2), v.repeat_interleave(g, 2)
    z = torch.einsum("bihd,bjhd->bhij", q, k) / cfg.head_dim ** 0.5
    z = z.masked_fill(torch.ones(S, S, dtype=torch.bool).triu(1), float("-inf"))
    o = torch.einsum("bhij,bjhd->bihd", torch.softmax(z, -1), v).reshape(B, S, -1)
    x = x + o @ n("wo").T
    m = _norm(x, n("w_ffn_norm"), cfg.norm_eps)
    return x + (torch.nn.functional.silu(m @ n("wg").T) * (m @ n("wu").T)) @ n("wd").T


def step(cfg: oracle.Config, packed_f32: np.ndarray, tok: np.ndarray, lab: np.ndarray, K: int, fmt: int | None,
         only: int | None = None, inputs_out: list | None = None):
    """(loss, {tensor: float64 gradient}); fmt None keeps the checkpoints, only
    rounds that of one block. inputs_out receives the blocks' inputs [T, h]."""
    p = {k: torch.from_numpy(v.astype(np.float64)).requires_grad_() for k, v in oracle.unpack(cfg, packed_f32).items()}
    tok, lab = torch.from_numpy(tok.astype(np.int64)), torch.from_numpy(lab.astype(np.int64))
    blocks = [range(b, min(b + K, cfg.n_layers)) for b in range(0, cfg.n_layers, K)]

    def run(block, x):
        for l in block:
            x = _layer(cfg, p, l, x)
        return x

    inputs = [p["embed"].detach()[tok]]
    with torch.no_grad():
        for block in blocks[:-1]:
            inputs.append(run(block, inputs[-1]))
    x = inputs[-1].clone().requires_grad_()
    z = _norm(run(blocks[-1], x), p["w_final_norm"], cfg.norm_eps) @ p["w_out"].T
    loss = torch.nn.functional.cross_entropy(z.flatten(0, 1), lab.flatten())
    loss.backward()
    if inputs_out is not None:
        inputs_out.extend(h.reshape(-1, cfg.hidden).numpy() for h in inputs)
    for b in range(len(blocks) - 2, -1, -1):
        block, h, above = blocks[b], inputs[b], x.grad
        if fmt is not None and only in (None, b):
            rows = h.reshape(-1, cfg.hidden).numpy().astype(np.float32)
            h = torch.from_numpy(ref.values_of(rows, fmt)).view_as(h)
        x = h.clone().requires_grad_()
        run(block, x).backward(above)
    dE = torch.zeros_like(p["embed"])
    dE.index_add_(0, tok.flatten(), x.grad.flatten(0, 1))
    grads = {k: (dE if k == "embed" else v.grad).numpy() for k, v in p.items()}
    return float(loss.detach()), grads


def borderline(cfg: oracle.Config, packed_f32: np.ndarray, tok: np.ndarray, lab: np.ndarray, K: int, fmt: int,
               u: float):
    """{tensor: relative L2} by which a step's gradients may lie from step()'s
    because its residuals are not the float64 ones: values near the border of
    two codes round to the other one.

    Let the residual x carry an error e, |e| <= u |x - embedding| (the embedded
    row is exact, what the layers add is not). x + e rounds to another code
    than x with probability |e| / d, d the distance of the codes, and then d
    away: a mean square of d |e|. The rounding itself has its known mean square
    and moves a tensor's gradient by a known amount (the step with that block
    rounded against the step without). Both are errors of the same values,
    uncorrelated with them and small, so they move the gradient in proportion
    to their root mean squares; the blocks' shares are added."""
    inputs: list = []
    _, plain = step(cfg, packed_f32, tok, lab, K, None, inputs_out=inputs)
    out = {k: 0.0 for k in plain}
    for b, h in enumerate(inputs[:-1]):
        added = np.abs(h - inputs[0])
        scale = np.repeat(2.0 ** (ref.scales_of(h.astype(np.float32), fmt).astype(np.float64) - 127), 32, 1)[:, :cfg.hidden]
        rounded = ref.values_of(h.astype(np.float32), fmt)
        if fmt == ref.I8:
            d = scale
        else:  # eight codes a binade, the lowest one's below 2^-6
            d = scale * 2.0 ** (np.maximum(np.floor(np.log2(np.maximum(np.abs(h) / scale, 2.0 ** -30))), -6) - 3)
        ratio = np.sqrt((d * np.minimum(u * added, d)).mean() / ((rounded - h) ** 2).mean())
        _, moved = step(cfg, packed_f32, tok, lab, K, fmt, only=b)
        for k in out:
            out[k] += ratio * np.linalg.norm(moved[k] - plain[k]) / np.linalg.norm(plain[k])
    return out
