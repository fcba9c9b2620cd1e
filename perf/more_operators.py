"""Operators of a training step around its blocks, its loss and its weights,
as measured: the norm after a block with the block's gate and the scaled
residual, fused with the norm before the next block; the cross entropy of a
head over a large vocabulary from its inputs and weights, without keeping the
logits, with the gradients of both; and the update of weight matrices by
orthogonalised momentum (Newton-Schulz products).

``own`` false computes them in plain torch, ``own`` true calls the library's
kernel-level entry points. Shapes come from the repository's configurations
(small: hidden 1024, FFN 2816, vocabulary 32000; 8B: hidden 4096, FFN 14336,
8 KV heads of 128, vocabulary 128256, 8192 tokens; mixture of experts: expert
width 1536, vocabulary 151936).

Kinds of case:
 norms  x' = a x + sigmoid(s) * (w_post * y / rms(y)), n = w_pre * x' / rms(x')
        for a residual x [T, h], a block's output y and its gate's values s
        (or no gate); with "train", the gradients of x, y, s and both weights
 ce     per row of X [T, h]: the loss logsumexp(z) - (1 - e) z_label
        - e mean(z) + c logsumexp(z)^2 of z = X W^T (W [V, h]) and the
        log-sum-exp; with "train", dX and dW for given gradients of the losses
 ortho  the orthogonalised form of each of `batch` matrices [rows, cols]
 muon   the same of momentum with a gradient, applied to the weights
"""
import math

import torch

own = False

QUINTIC = (3.4445, -4.7750, 2.0315)
EPS = 1e-5


def listed():
    return [
        # the small decoder's norms on a short batch: latency
        {"name": "norms_few", "kind": "norms", "T": 77, "h": 1024, "dtype": "bf16", "gate": True, "train": True},
        # the 8B norms of one prompt token by token: the form without gradients, a single row
        {"name": "norms_one", "kind": "norms", "T": 1, "h": 4096, "dtype": "bf16", "gate": True, "train": False},
        # one block of the 8B step
        {"name": "norms_8b", "kind": "norms", "T": 8192, "h": 4096, "dtype": "bf16", "gate": True, "train": True},
        # fp32 block outputs without a gate, width and tokens off the powers of two
        {"name": "norms_wide", "kind": "norms", "T": 4095, "h": 5636, "dtype": "f32", "gate": False, "train": True},
        # the small decoder's head on a few tokens: W is read and dW written, latency of the chain
        {"name": "ce_few", "kind": "ce", "T": 7, "V": 32000, "h": 1024, "smooth": 0.0, "z": 0.0, "train": True},
        # the small decoder's head, ragged token count, smoothed labels and a penalty on the log-sum-exp
        {"name": "ce_small", "kind": "ce", "T": 2047, "V": 32000, "h": 1024, "smooth": 0.1, "z": 1e-4, "train": True},
        # a held-out batch of the mixture of experts' head: losses alone
        {"name": "ce_eval", "kind": "ce", "T": 4095, "V": 151936, "h": 4096, "smooth": 0.0, "z": 0.0, "train": False},
        # the 8B head, one step
        {"name": "ce_8b", "kind": "ce", "T": 8192, "V": 128256, "h": 4096, "smooth": 0.0, "z": 0.0, "train": True},
        # one square weight of the small decoder: a chain of small products
        {"name": "muon_small", "kind": "muon", "batch": 1, "rows": 1024, "cols": 1024, "grad": "f32", "steps": 5},
        # the 8B key projection's gradient, orthogonalised
        {"name": "ortho_kv", "kind": "ortho", "batch": 1, "rows": 1024, "cols": 4096, "grad": "bf16", "steps": 5},
        # the 8B gate projection (tall)
        {"name": "muon_ffn", "kind": "muon", "batch": 1, "rows": 14336, "cols": 4096, "grad": "f32", "steps": 5},
        # down projections of sixteen experts in one call
        {"name": "ortho_experts", "kind": "ortho", "batch": 16, "rows": 4096, "cols": 1536, "grad": "f32", "steps": 5},
    ]


def _spread(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["norms", "ce", "ce", "ortho", "muon"])
    if kind == "norms":
        h = 4 * _spread(rng, 16, 2048)
        return {"kind": kind, "T": min(_spread(rng, 1, 16384), (8192 * 4096) // h), "h": h, "dtype": rng.choice(["bf16", "f32"]),
                "gate": rng.random() < 0.6, "train": rng.random() < 0.7}
    if kind == "ce":
        V, h = _spread(rng, 256, 151936), 8 * _spread(rng, 8, 640)
        T = min(_spread(rng, 1, 16384), (8192 * 128256 * 4096) // (2 * V * h))
        plain = rng.random() < 0.5
        return {"kind": kind, "T": T, "V": V, "h": h, "smooth": 0.0 if plain else 0.1, "z": 0.0 if plain else 1e-4,
                "train": rng.random() < 0.7}
    rows, cols = _spread(rng, 24, 8192), _spread(rng, 24, 8192)
    one = 3 * min(rows, cols) * rows * cols + min(rows, cols) ** 3
    batch = max(1, min(_spread(rng, 1, 32), int(4e11 / one)))
    return {"kind": kind, "batch": batch, "rows": rows, "cols": cols, "grad": rng.choice(["f32", "bf16"]), "steps": rng.choice([5, 5, 6])}


def _torch_type(name):
    return torch.float32 if name == "f32" else torch.bfloat16


def _normal(gen, *shape, std=1.0, dtype=torch.float32):
    return torch.empty(shape, device="cuda", dtype=dtype).normal_(0.0, std, generator=gen)


def _activation(gen, T, n, dtype=torch.float32):
    """A residual stream's values: tokens of different size, a few channels far above the others."""
    x = _normal(gen, T, n)
    x *= torch.exp(0.5 * _normal(gen, T, 1))
    loud = torch.rand(n, device="cuda", generator=gen) < 0.004
    x *= torch.where(loud, 30.0, 1.0)
    return x.to(dtype)


def _gradient(gen, batch, rows, cols):
    """A weight's gradient: products of tokens' errors of very different size with activations that share a mean,
    and the rounding of what went before."""
    n = 256
    e = _normal(gen, batch, n, rows) * torch.exp(1.5 * _normal(gen, batch, n, 1))
    a = _normal(gen, batch, n, cols) + _normal(gen, batch, 1, cols)
    return torch.bmm(e.transpose(1, 2), a) * 1e-4 + _normal(gen, batch, rows, cols, std=1e-3)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed) * 1000003 + 29)
    s = {"case": dict(case)}
    kind = case["kind"]
    new = lambda *shape, dtype=torch.float32: torch.empty(shape, device="cuda", dtype=dtype)  # noqa: E731
    bf = torch.bfloat16
    if kind == "norms":
        T, h, dt = case["T"], case["h"], _torch_type(case["dtype"])
        s["x"], s["y"] = _activation(gen, T, h), _activation(gen, T, h, dt)
        s["gate"] = _normal(gen, T, h, std=2.0, dtype=dt) if case["gate"] else None
        s["w_post"], s["w_pre"] = 1.0 + 0.1 * _normal(gen, h), 1.0 + 0.1 * _normal(gen, h)
        s["alpha"] = 0.875
        s["x_out"], s["n"], s["r_post"], s["r_pre"] = new(T, h), new(T, h, dtype=bf), new(T), new(T)
        if case["train"]:
            s["dn"], s["dres"] = _normal(gen, T, h, std=0.01), _normal(gen, T, h, std=0.01)
            s["dx"], s["dy"], s["dgate"] = new(T, h), new(T, h, dtype=dt), new(T, h, dtype=dt) if case["gate"] else None
            s["dw_post"], s["dw_pre"] = new(h), new(h)
            if own:
                import layer_streamed_gb300 as mt
                s["work"] = new(mt.mt_op_sandwich_norm_bwd_workspace(T, h))
    elif kind == "ce":
        T, V, h = case["T"], case["V"], case["h"]
        s["W"] = _normal(gen, V, h, std=0.02, dtype=bf)
        labels = torch.randint(0, V, (T,), device="cuda", generator=gen)
        # inputs as a norm leaves them, leaning towards the label's row
        lean = 8.0 * torch.rand(T, 1, device="cuda", generator=gen) / (0.02 * math.sqrt(h))
        s["X"] = (_normal(gen, T, h) + lean * (s["W"][labels].float() / (0.02 * math.sqrt(h)))).to(bf)
        if T >= 8:  # padding and prompt positions
            labels = torch.where(torch.rand(T, device="cuda", generator=gen) < 0.05, -1, labels)
        s["labels"] = labels.to(torch.int32)
        s["loss"], s["lse"] = new(T), new(T)
        if case["train"]:
            s["g"] = (0.5 + torch.rand(T, device="cuda", generator=gen)) / T  # weights of the tokens over their number
            s["dX"], s["dW"] = new(T, h, dtype=bf), new(V, h, dtype=bf)
        if own:
            import layer_streamed_gb300 as mt
            n = mt.mt_op_linear_ce_fwd_workspace(T, V, h)
            if case["train"]:
                n = max(n, mt.mt_op_linear_ce_bwd_workspace(T, V, h))
            s["work"] = new(n, dtype=torch.uint8)
    else:
        b, rows, cols = case["batch"], case["rows"], case["cols"]
        s["G"] = _gradient(gen, b, rows, cols).to(_torch_type(case["grad"]))
        if kind == "muon":
            s["M"] = 4.0 * _gradient(gen, b, rows, cols)
            s["W"] = _normal(gen, b, rows, cols, std=0.02, dtype=bf)
            s["mu"], s["lr"], s["decay"], s["scale"] = 0.95, 2e-3, 0.1, 0.2 * math.sqrt(max(rows, cols))
        else:
            s["O"] = new(b, rows, cols, dtype=bf)
        if own:
            import layer_streamed_gb300 as mt
            s["work"] = new(mt.mt_op_orthogonalize_workspace(b, rows, cols), dtype=torch.uint8)
    return s


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------
def _plain_ortho(u, steps):
    wide = u.shape[1] <= u.shape[2]
    x = u if wide else u.transpose(1, 2)
    x = x / (x.square().sum((1, 2), keepdim=True).sqrt() + 1e-7)
    a, b, c = QUINTIC
    for _ in range(steps):
        g = torch.bmm(x, x.transpose(1, 2))
        x = a * x + torch.bmm(b * g + c * torch.bmm(g, g), x)
    return x if wide else x.transpose(1, 2)


def _run_plain(s):
    c = s["case"]
    kind = c["kind"]
    if kind == "norms":
        x, y, wa, wb, al = s["x"], s["y"].float(), s["w_post"], s["w_pre"], s["alpha"]
        ra = torch.rsqrt(y.square().mean(-1, keepdim=True) + EPS)
        yh = y * ra
        sg = 1 / (1 + torch.exp(-s["gate"].float())) if c["gate"] else 1.0
        xo = al * x + sg * (yh * wa)
        rb = torch.rsqrt(xo.square().mean(-1, keepdim=True) + EPS)
        xh = xo * rb
        out = {"x_out": xo, "n": (xh * wb).to(torch.bfloat16), "rstd_post": ra[:, 0], "rstd_pre": rb[:, 0]}
        if c["train"]:
            g = s["dn"] * wb
            d = s["dres"] + rb * (g - xh * (g * xh).mean(-1, keepdim=True))
            k = d * sg
            g = k * wa
            dy = ra * (g - yh * (g * yh).mean(-1, keepdim=True))
            out |= {"dx": al * d, "dy": dy.to(s["y"].dtype), "dw_post": (k * yh).sum(0), "dw_pre": (s["dn"] * xh).sum(0)}
            if c["gate"]:
                out["dgate"] = (d * (yh * wa) * sg * (1 - sg)).to(s["gate"].dtype)
        return out
    if kind == "ce":
        X, W, e, zc = s["X"].float(), s["W"].float(), c["smooth"], c["z"]
        keep = s["labels"] >= 0
        i = s["labels"].long().clamp(min=0)[:, None]
        z = X @ W.T
        m = z.amax(-1, keepdim=True)
        p = torch.exp(z - m)
        total = p.sum(-1, keepdim=True)
        lse = m + torch.log(total)
        loss = lse - (1 - e) * z.gather(1, i) - e * z.mean(-1, keepdim=True) + zc * lse.square()
        out = {"loss": torch.where(keep, loss[:, 0], 0.0), "lse": torch.where(keep, lse[:, 0], 0.0)}
        if c["train"]:
            g = torch.where(keep, s["g"], 0.0)[:, None]
            p = p * (g / total * (1 + 2 * zc * lse)) - g * (e / c["V"])
            p.scatter_add_(1, i, -(1 - e) * g)
            out |= {"dX": (p @ W).to(torch.bfloat16), "dW": (p.T @ X).to(torch.bfloat16)}
        return out
    G = s["G"].float()
    if kind == "ortho":
        return {"O": _plain_ortho(G, c["steps"]).to(torch.bfloat16)}
    s["M"].mul_(s["mu"]).add_(G)
    w = s["W"].float()
    w = w - s["lr"] * (s["scale"] * _plain_ortho(G + s["mu"] * s["M"], c["steps"]) + s["decay"] * w)
    s["W"].copy_(w)
    return {"M": s["M"], "W": s["W"]}


# ---------------------------------------------------------------------------
# the library's operators
# ---------------------------------------------------------------------------
def _run_own(s):
    import layer_streamed_gb300 as mt
    c = s["case"]
    kind = c["kind"]
    code = lambda t: mt.MT_F32 if t.dtype == torch.float32 else mt.MT_BF16  # noqa: E731
    if kind == "norms":
        T, h, dt = c["T"], c["h"], code(s["y"])
        mt.mt_op_sandwich_norm_fwd(s["x"], s["y"], s["gate"], dt, s["w_post"], s["w_pre"], s["alpha"], EPS, s["x_out"], s["n"],
                                   s["r_post"], s["r_pre"], T, h)
        out = {"x_out": s["x_out"], "n": s["n"], "rstd_post": s["r_post"], "rstd_pre": s["r_pre"]}
        if c["train"]:
            mt.mt_op_sandwich_norm_bwd(s["x_out"], s["y"], s["gate"], dt, s["w_post"], s["w_pre"], s["alpha"], s["r_post"],
                                       s["r_pre"], s["dn"], s["dres"], s["dx"], s["dy"], s["dgate"], s["dw_post"], s["dw_pre"],
                                       s["work"], T, h)
            out |= {"dx": s["dx"], "dy": s["dy"], "dw_post": s["dw_post"], "dw_pre": s["dw_pre"]}
            if c["gate"]:
                out["dgate"] = s["dgate"]
        return out
    if kind == "ce":
        T, V, h = c["T"], c["V"], c["h"]
        mt.mt_op_linear_ce_fwd(s["X"], s["W"], s["labels"], 1.0, c["smooth"], c["z"], s["loss"], s["lse"], s["work"], T, V, h,
                               h, h)
        out = {"loss": s["loss"], "lse": s["lse"]}
        if c["train"]:
            mt.mt_op_linear_ce_bwd(s["X"], s["W"], s["labels"], 1.0, c["smooth"], c["z"], s["lse"], s["g"], s["dX"], mt.MT_BF16,
                                   s["dW"], mt.MT_BF16, 0, s["work"], T, V, h, h, h)
            out |= {"dX": s["dX"], "dW": s["dW"]}
        return out
    b, rows, cols = c["batch"], c["rows"], c["cols"]
    if kind == "ortho":
        mt.mt_op_orthogonalize(s["G"], code(s["G"]), s["O"], mt.MT_BF16, None, c["steps"], 1e-7, s["work"], b, rows, cols)
        return {"O": s["O"]}
    mt.mt_op_muon_update(s["W"], mt.MT_BF16, s["M"], s["G"], code(s["G"]), s["mu"], 1, s["lr"], s["decay"], s["scale"], None,
                         c["steps"], 1e-7, s["work"], b, rows, cols)
    return {"M": s["M"], "W": s["W"]}


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---------------------------------------------------------------------------
# what a pass cannot do without, and the values by definition
# ---------------------------------------------------------------------------
def work(case):
    size = lambda name: 4 if name == "f32" else 2  # noqa: E731
    kind = case["kind"]
    if kind == "norms":  # forward: x, y, gate in, x', n out; backward: x', y, gate, dn, the residual's gradient in, dx, dy, dgate out
        T, h, b = case["T"], case["h"], size(case["dtype"]) * (2 if case["gate"] else 1)
        n = T * h * (4 + b + 4 + 2) + 2 * 4 * h + 2 * 4 * T
        if case["train"]:
            n += T * h * (4 + b + 4 + 4 + 4 + b) + 4 * 4 * h + 2 * 4 * T
        return {"bytes": n, "flops": (46 if case["train"] else 14) * T * h}
    if kind == "ce":  # X, W once a direction, dX, dW once; the logits' product, again backward, and the gradients' two
        T, V, h = case["T"], case["V"], case["h"]
        n = 2 * (T + V) * h
        return {"bytes": n * (3 if case["train"] else 1) + 4 * T * (5 if case["train"] else 3),
                "flops": (8 if case["train"] else 2) * T * V * h}
    # a step: a symmetric product [m, m] over n, its square (both half as much as in full), and one [m, m] with [m, n]
    b, m, n = case["batch"], min(case["rows"], case["cols"]), max(case["rows"], case["cols"])
    e = size(case["grad"]) + (2 if kind == "ortho" else 4 + 4 + 2 + 2)
    return {"bytes": b * m * n * e, "flops": b * case["steps"] * (3 * m * m * n + m ** 3)}


def _exact_ortho(u, steps):
    flip = u.shape[1] > u.shape[2]
    x = u.mT if flip else u
    x = x / (torch.linalg.matrix_norm(x)[:, None, None] + 1e-7)
    eye = torch.eye(x.shape[1], device="cuda", dtype=torch.float64)
    a, b, c = QUINTIC
    for _ in range(steps):  # p(x) = a x + b (x x^T) x + c (x x^T)^2 x
        g = x @ x.mT
        x = (a * eye + (b * eye + c * g) @ g) @ x
    return x.mT if flip else x


def exact(case, seed):
    s = prepare(case, seed)
    kind = case["kind"]
    f32 = lambda v: float(torch.tensor(v, dtype=torch.float32))  # noqa: E731
    if kind == "norms":
        h = case["h"]
        x, y, wa, wb = (s[k].double() for k in ("x", "y", "w_post", "w_pre"))
        sg = torch.sigmoid(s["gate"].double()) if case["gate"] else torch.ones_like(y)
        ra = 1 / torch.sqrt(torch.einsum("th,th->t", y, y) / h + f32(EPS))
        u = y * ra[:, None] * wa
        xo = s["alpha"] * x + sg * u
        rb = 1 / torch.sqrt(torch.einsum("th,th->t", xo, xo) / h + f32(EPS))
        v = xo * rb[:, None]
        out = {"x_out": xo, "n": v * wb, "rstd_post": ra, "rstd_pre": rb}
        if case["train"]:
            dn, dres = s["dn"].double(), s["dres"].double()
            d = dres + rb[:, None] * (dn * wb - v * (torch.einsum("th,h,th->t", dn, wb, v) / h)[:, None])
            du = d * sg
            yh = y * ra[:, None]
            out["dx"] = s["alpha"] * d
            out["dy"] = ra[:, None] * (du * wa - yh * (torch.einsum("th,h,th->t", du, wa, yh) / h)[:, None])
            out["dw_post"], out["dw_pre"] = torch.einsum("th,th->h", du, yh), torch.einsum("th,th->h", dn, v)
            if case["gate"]:
                out["dgate"] = d * u * sg * (1 - sg)
        return out
    if kind == "ce":
        T, V, h, e, zc = (case[k] for k in ("T", "V", "h", "smooth", "z"))
        X, W = s["X"].double(), s["W"].double()
        kept = torch.nonzero(s["labels"] >= 0)[:, 0]
        out = {"loss": torch.zeros(T, device="cuda", dtype=torch.float64), "lse": torch.zeros(T, device="cuda", dtype=torch.float64)}
        grads = case["train"] and 6 * T * V * h < 1.2e13
        if case["train"]:
            out["dX"] = torch.zeros_like(X) if grads else None
            out["dW"] = torch.zeros_like(W) if grads else None
        for part in kept.split(1024):
            z = X[part] @ W.mT
            lab = s["labels"][part].long()
            lse = torch.logsumexp(z, 1)
            at = torch.arange(part.numel(), device="cuda")
            out["lse"][part] = lse
            out["loss"][part] = lse + zc * lse ** 2 - (1 - e) * z[at, lab] - (e * z.sum(1) / V if e else 0.0)
            if grads:  # of g * loss by z: (1 + 2 c lse) softmax - (1 - e) [label] - e / V
                dz = torch.softmax(z, 1) * (1 + 2 * zc * lse)[:, None] - e / V
                dz[at, lab] -= 1 - e
                dz *= s["g"][part].double()[:, None]
                out["dX"][part] = dz @ W
                out["dW"] += dz.mT @ X[part]
        return out
    if kind == "ortho":
        return {"O": _exact_ortho(s["G"].double(), case["steps"])}
    G, mu = s["G"].double(), f32(s["mu"])
    M = mu * s["M"].double() + G
    W = s["W"].double()
    step = f32(s["scale"]) * _exact_ortho(G + mu * M, case["steps"]) + f32(s["decay"]) * W
    return {"M": M, "W": W - f32(s["lr"]) * step}
