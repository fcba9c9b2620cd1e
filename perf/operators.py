"""The operators around the recomputing decoder step, as measured: 8-bit
activation checkpoints and their use in the backward pass, log probabilities
of given tokens with entropy and top alternatives, and the embedding lookup
with its gradient by sorted tokens.

``own`` false computes them in plain torch, ``own`` true calls the library's
kernel-level entry points. Shapes come from the repository's configurations
(small: hidden 1024, FFN 2816, vocabulary 32000; 8B: hidden 4096, FFN 14336,
vocabulary 128256, 8192 tokens; mixture of experts: vocabulary 151936).

Kinds of case:
 ckpt    an activation [T, n] kept in 8 bits (blocks of 32 columns, one
         power-of-two scale each) and restored: pack, then unpack
 norm    RMSNorm forward that keeps its input in 8 bits, and the backward that
         reads it from there: y, rstd, dx (fp32 and bf16), dw
 swiglu  SwiGLU forward that keeps g|u in 8 bits, and the backward that reads
         them from there: act, d(g|u)
 logp    log probability of one given token per row of logits, the row's
         log-sum-exp and entropy, its k most likely tokens; with "train", also
         the gradient of the logits for given gradients of both
 embed   rows of the table for given tokens, times a scale, and the table's
         gradient (dense, summed per token)
"""
import math

import numpy as np
import torch

own = False

BLOCK = 32
FMT = {"i8": 1, "e4m3": 2}


def listed():
    return [
        # a checkpoint of a few tokens, ragged last block: latency
        {"name": "ckpt_few", "kind": "ckpt", "T": 65, "n": 1000, "fmt": "i8", "dtype": "bf16"},
        # one residual checkpoint of the 8B step
        {"name": "ckpt_8b", "kind": "ckpt", "T": 8192, "n": 4096, "fmt": "e4m3", "dtype": "f32"},
        # the small decoder's norm on a short batch: latency
        {"name": "norm_few", "kind": "norm", "T": 77, "h": 1024, "fmt": "e4m3"},
        # one norm of the 8B step
        {"name": "norm_8b", "kind": "norm", "T": 8192, "h": 4096, "fmt": "i8"},
        # the small decoder's MLP, ragged token count
        {"name": "swiglu_small", "kind": "swiglu", "T": 2047, "F": 2816, "fmt": "e4m3"},
        # the 8B MLP
        {"name": "swiglu_8b", "kind": "swiglu", "T": 8192, "F": 14336, "fmt": "i8"},
        # one token scored while sampling, with 20 alternatives: latency
        {"name": "logp_one", "kind": "logp", "T": 1, "V": 151936, "dtype": "bf16", "k": 20, "train": False},
        # a scored batch of the 8B model
        {"name": "logp_8b", "kind": "logp", "T": 8192, "V": 128256, "dtype": "f32", "k": 8, "train": False},
        # a policy-gradient micro-batch: log probability, entropy, and their gradient
        {"name": "logp_train", "kind": "logp", "T": 4095, "V": 151936, "dtype": "bf16", "k": 0, "train": True},
        # the small decoder's embedding, a short batch
        {"name": "embed_few", "kind": "embed", "T": 64, "V": 32000, "h": 1024, "dtype": "f32", "grad": "f32"},
        # the 8B embedding, one step
        {"name": "embed_8b", "kind": "embed", "T": 8192, "V": 128256, "h": 4096, "dtype": "bf16", "grad": "f32"},
        # one long sequence, bf16 gradients
        {"name": "embed_long", "kind": "embed", "T": 16384, "V": 151936, "h": 4096, "dtype": "bf16", "grad": "bf16"},
    ]


def _spread(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["ckpt", "norm", "swiglu", "logp", "logp", "embed", "embed"])
    fmt = rng.choice(["i8", "e4m3"])
    dtype = rng.choice(["f32", "bf16"])
    if kind == "ckpt":
        n = _spread(rng, 24, 14336)
        return {"kind": kind, "T": min(_spread(rng, 1, 16384), (8192 * 4096) // n), "n": n, "fmt": fmt, "dtype": dtype}
    if kind == "norm":
        h = 4 * _spread(rng, 16, 2048)
        return {"kind": kind, "T": min(_spread(rng, 1, 16384), (8192 * 4096) // h), "h": h, "fmt": fmt}
    if kind == "swiglu":
        F = _spread(rng, 40, 14336)
        return {"kind": kind, "T": min(_spread(rng, 1, 16384), (8192 * 14336) // F), "F": F, "fmt": fmt}
    if kind == "logp":
        V, train = _spread(rng, 256, 151936), rng.random() < 0.5
        T = min(_spread(rng, 1, 16384), (8192 * 128256) // (2 * V))
        return {"kind": kind, "T": T, "V": V, "dtype": dtype, "k": rng.choice([0, 1, 5, 8, 20]), "train": train}
    V, h = _spread(rng, 256, 151936), 8 * _spread(rng, 8, 1024)
    h = min(h, (128256 * 4096) // V // 8 * 8)
    T = min(_spread(rng, 1, 32768), (16384 * 4096) // h)
    return {"kind": "embed", "T": T, "V": V, "h": h, "dtype": dtype, "grad": rng.choice(["f32", "bf16"])}


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


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed) * 1000003 + 17)
    s = {"case": dict(case)}
    kind, T = case["kind"], case["T"]
    new = lambda *shape, dtype=torch.float32: torch.empty(shape, device="cuda", dtype=dtype)  # noqa: E731
    u8, bf = torch.uint8, torch.bfloat16
    if kind == "ckpt":
        n = case["n"]
        s["x"] = _activation(gen, T, n, _torch_type(case["dtype"]))
        s["codes"], s["scales"] = new(T, n, dtype=u8), new(T, -(-n // BLOCK), dtype=u8)
        s["back"] = torch.empty_like(s["x"])
    elif kind == "norm":
        h = case["h"]
        s["x"] = _activation(gen, T, h)
        s["w"] = 1.0 + 0.1 * _normal(gen, h)
        s["dy"], s["resid"] = _normal(gen, T, h, std=0.01), _normal(gen, T, h, std=0.01)
        s["codes"], s["scales"] = new(T, h, dtype=u8), new(T, -(-h // BLOCK), dtype=u8)
        s["y"], s["rstd"], s["dx"], s["dxb"], s["dw"] = new(T, h, dtype=bf), new(T), new(T, h), new(T, h, dtype=bf), new(h)
        if own:
            import layer_streamed_gb300 as mt
            s["work"] = new(max(1, mt.mt_op_rmsnorm_bwd_ckpt8_workspace(T, h)))
    elif kind == "swiglu":
        F = case["F"]
        s["gu"] = _activation(gen, T, 2 * F, bf)
        s["dact"] = _normal(gen, T, F, std=0.01, dtype=bf)
        s["codes"], s["scales"] = new(T, 2 * F, dtype=u8), new(T, 2 * -(-F // BLOCK), dtype=u8)
        s["act"], s["dgu"] = new(T, F, dtype=bf), new(T, 2 * F, dtype=bf)
    elif kind == "logp":
        V, k, dt = case["V"], case["k"], _torch_type(case["dtype"])
        z = _normal(gen, T, V, std=2.5, dtype=dt)
        ids = torch.randint(0, V, (T,), device="cuda", generator=gen)
        # the scored token is usually a likely one
        z[torch.arange(T, device="cuda"), ids] += (8.0 * torch.rand(T, device="cuda", generator=gen)).to(dt)
        if V >= 1024:  # entries that may not be sampled
            z[:, V - V // 64:] = float("-inf")
            ids = torch.where(ids >= V - V // 64, ids - V // 64, ids)
        if T >= 8:  # positions of the prompt are not scored
            ids = torch.where(torch.rand(T, device="cuda", generator=gen) < 0.05, -1, ids)
        s["z"], s["ids"], s["inv_temp"] = z, ids.to(torch.int32), 1.0 if case["train"] else 1.25
        s["lse"], s["logp"], s["ent"] = new(T), new(T), new(T)
        s["top_ids"], s["top_logp"] = new(T, k, dtype=torch.int32), new(T, k)
        if case["train"]:
            s["g_logp"], s["g_ent"] = _normal(gen, T), torch.full((T,), -0.01, device="cuda")
            s["dz"] = torch.empty_like(z)
    else:
        V, h, dt = case["V"], case["h"], _torch_type(case["dtype"])
        s["table"] = _normal(gen, V, h, std=0.02, dtype=dt)
        # token frequencies fall off with their rank, ranks spread over the vocabulary
        rank = torch.exp(torch.rand(T, device="cuda", generator=gen, dtype=torch.float64) * math.log(V)).long() - 1
        ids = (rank.clamp_(0, V - 1) * 7919) % V
        if T >= 8:  # padding
            ids = torch.where(torch.rand(T, device="cuda", generator=gen) < 0.03, -1, ids)
        s["ids"], s["scale"] = ids.to(torch.int32), math.sqrt(h)
        s["dout"] = _normal(gen, T, h, std=0.01)
        s["out"], s["dtable"] = new(T, h), new(V, h, dtype=_torch_type(case["grad"]))
        if own:
            import layer_streamed_gb300 as mt
            s["work"] = new(mt.mt_op_embed_bwd_workspace(T, V, h), dtype=u8)
    return s


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------
def _times_pow2(x, e):
    """x * 2^e for whole e in [-252, 252], in two exact steps."""
    half = torch.div(e, 2, rounding_mode="floor")
    for part in (half, e - half):
        x = x * ((part + 127) << 23).view(torch.float32)
    return x


def _plain_round8(x, fmt):
    """x (float32, last axis in blocks of 32) as its 8-bit block form stands for it."""
    n = x.shape[-1]
    pad = -n % BLOCK
    b = torch.nn.functional.pad(x, (0, pad)).view(*x.shape[:-1], -1, BLOCK)
    m, e = torch.frexp(b.abs().amax(-1, keepdim=True))
    # smallest power of two that brings the block's largest value within 127 = 0.9921875 * 2^7 (448 = 0.875 * 2^9)
    limit, bits = (0.9921875, 7) if fmt == "i8" else (0.875, 9)
    e = (e - bits + (m > limit).to(e.dtype)).clamp_(min=-127)
    q = _times_pow2(b, -e)
    q = torch.round(q) if fmt == "i8" else q.to(torch.float8_e4m3fn).float()
    return _times_pow2(q, e).reshape(*x.shape[:-1], n + pad)[..., :n]


def _plain_logp(s, k):
    z, ids, it = s["z"], s["ids"].long(), s["inv_temp"]
    T, V = z.shape
    lse, logp, ent = torch.zeros(T, device="cuda"), torch.zeros(T, device="cuda"), torch.zeros(T, device="cuda")
    top_ids = torch.full((T, k), -1, device="cuda", dtype=torch.int32)
    top_logp = torch.zeros(T, k, device="cuda")
    dz = torch.empty_like(z) if "g_logp" in s else None
    column = torch.arange(V, device="cuda", dtype=torch.int32)
    for r in range(0, T, 1024):
        rows = slice(r, min(T, r + 1024))
        keep = ids[rows] >= 0
        i = ids[rows].clamp(min=0)[:, None]
        x = z[rows].float()
        m = x.amax(-1, keepdim=True)
        d = (x - m) * it
        p = torch.exp(d)
        total = p.sum(-1, keepdim=True)
        log_total = torch.log(total)
        p = p / total
        log_p = d - log_total
        h = -torch.where(p > 0, p * log_p, 0.0).sum(-1, keepdim=True)
        lse[rows] = torch.where(keep, (m * it + log_total)[:, 0], 0.0)
        logp[rows] = torch.where(keep, log_p.gather(1, i)[:, 0], 0.0)
        ent[rows] = torch.where(keep, h[:, 0], 0.0)
        x = x.clone() if k else x  # the search below strikes out what it has found; the logits stay
        for j in range(k):
            best = x.amax(-1, keepdim=True)
            at = torch.where(x == best, column, V).amin(-1, keepdim=True)
            there = keep & (best[:, 0] > float("-inf"))
            top_ids[rows, j] = torch.where(there, at[:, 0], -1)
            top_logp[rows, j] = torch.where(keep, log_p.gather(1, at.long())[:, 0], 0.0)
            x.scatter_(1, at.long(), float("-inf"))
        if dz is not None:
            gl, ge = s["g_logp"][rows, None], s["g_ent"][rows, None]
            g = -gl * p - ge * torch.where(p > 0, p * (log_p + h), 0.0)
            g.scatter_add_(1, i, gl)
            dz[rows] = torch.where(keep[:, None], g * it, 0.0).to(z.dtype)
    out = {"lse": lse, "logp": logp, "entropy": ent, "top_ids": top_ids, "top_logp": top_logp}
    if dz is not None:
        out["dlogits"] = dz
    return out


def _run_plain(s):
    c = s["case"]
    kind = c["kind"]
    if kind == "ckpt":
        return {"x": _plain_round8(s["x"].float(), c["fmt"]).to(s["x"].dtype)}
    if kind == "norm":
        x, w, dy = s["x"], s["w"], s["dy"]
        r = torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-5)
        y = (x * r * w).to(torch.bfloat16)
        xh = _plain_round8(x, c["fmt"]) * r
        g = dy * w
        dx = s["resid"] + r * (g - xh * (g * xh).mean(-1, keepdim=True))
        return {"y": y, "rstd": r[:, 0], "dx": dx, "dx_bf16": dx.to(torch.bfloat16), "dw": (dy * xh).sum(0)}
    if kind == "swiglu":
        F = c["F"]
        g, u = s["gu"][:, :F].float(), s["gu"][:, F:].float()
        act = (g / (1 + torch.exp(-g)) * u).to(torch.bfloat16)
        g, u = _plain_round8(g, c["fmt"]), _plain_round8(u, c["fmt"])
        d = s["dact"].float()
        sg = 1 / (1 + torch.exp(-g))
        dgu = torch.cat([d * u * sg * (1 + g * (1 - sg)), d * g * sg], 1).to(torch.bfloat16)
        return {"act": act, "dgu": dgu}
    if kind == "logp":
        return _plain_logp(s, c["k"])
    ids = s["ids"].long()
    keep = (ids >= 0)[:, None]
    i = ids.clamp(min=0)
    out = torch.where(keep, s["table"][i].float() * s["scale"], 0.0)
    d = torch.zeros(c["V"], c["h"], device="cuda")
    d.index_add_(0, i, torch.where(keep, s["dout"], 0.0))
    return {"out": out, "dtable": (d * s["scale"]).to(_torch_type(c["grad"]))}


# ---------------------------------------------------------------------------
# the library's operators
# ---------------------------------------------------------------------------
def _run_own(s):
    import layer_streamed_gb300 as mt
    c = s["case"]
    kind, T = c["kind"], c["T"]
    code = lambda t: mt.MT_F32 if t.dtype == torch.float32 else mt.MT_BF16  # noqa: E731
    if kind == "ckpt":
        n, fmt = c["n"], FMT[c["fmt"]]
        mt.mt_op_ckpt8_pack(s["x"], code(s["x"]), fmt, s["codes"], s["scales"], T, n, n, n)
        mt.mt_op_ckpt8_unpack(s["codes"], s["scales"], fmt, s["back"], code(s["back"]), T, n, n, n)
        return {"x": s["back"]}
    if kind == "norm":
        h, fmt = c["h"], FMT[c["fmt"]]
        mt.mt_op_rmsnorm_fwd_ckpt8(s["x"], s["w"], s["y"], s["rstd"], s["codes"], s["scales"], fmt, T, h, 1e-5)
        mt.mt_op_rmsnorm_bwd_ckpt8(s["codes"], s["scales"], fmt, s["w"], s["rstd"], s["dy"], s["resid"], s["dx"], s["dxb"],
                                   s["dw"], s["work"], T, h)
        return {"y": s["y"], "rstd": s["rstd"], "dx": s["dx"], "dx_bf16": s["dxb"], "dw": s["dw"]}
    if kind == "swiglu":
        F, fmt = c["F"], FMT[c["fmt"]]
        mt.mt_op_swiglu_fwd_ckpt8(s["gu"], s["act"], s["codes"], s["scales"], fmt, T, F, F)
        mt.mt_op_swiglu_bwd_ckpt8(s["codes"], s["scales"], fmt, s["dact"], s["dgu"], T, F, F)
        return {"act": s["act"], "dgu": s["dgu"]}
    if kind == "logp":
        V, k, z = c["V"], c["k"], s["z"]
        mt.mt_op_token_logprobs(z, code(z), s["ids"], s["inv_temp"], k, s["lse"], s["logp"], s["ent"], s["top_ids"],
                                s["top_logp"], T, V, V)
        out = {"lse": s["lse"], "logp": s["logp"], "entropy": s["ent"], "top_ids": s["top_ids"], "top_logp": s["top_logp"]}
        if c["train"]:
            mt.mt_op_token_logprobs_bwd(z, code(z), s["ids"], s["inv_temp"], s["lse"], s["ent"], s["g_logp"], s["g_ent"],
                                        s["dz"], code(s["dz"]), T, V, V, V)
            out["dlogits"] = s["dz"]
        return out
    V, h = c["V"], c["h"]
    mt.mt_op_embed_fwd(s["table"], code(s["table"]), s["ids"], s["scale"], s["out"], mt.MT_F32, T, V, h)
    mt.mt_op_embed_bwd(s["ids"], s["dout"], mt.MT_F32, s["scale"], s["dtable"], code(s["dtable"]), 0, s["work"], T, V, h)
    return {"out": s["out"], "dtable": s["dtable"]}


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---------------------------------------------------------------------------
# what a pass cannot do without, and the values by definition
# ---------------------------------------------------------------------------
def work(case):
    kind, T = case["kind"], case["T"]
    size = lambda name: 4 if name == "f32" else 2  # noqa: E731
    if kind == "ckpt":  # read x, write codes and scales, read them, write x
        n, b = case["n"], size(case["dtype"])
        return {"bytes": T * n * 2 * b + 2 * T * (n + -(-n // BLOCK)), "flops": 4 * T * n}
    if kind == "norm":  # forward: x, y, the checkpoint; backward: the checkpoint, dy, residual, dx twice
        h = case["h"]
        return {"bytes": T * h * (4 + 2 + 4 + 4 + 4 + 2) + 2 * T * (h + -(-h // BLOCK)) + 2 * 4 * h + 2 * 4 * T,
                "flops": 18 * T * h}
    if kind == "swiglu":  # forward: g|u, act, the checkpoint; backward: the checkpoint, dact, d(g|u)
        F = case["F"]
        return {"bytes": T * F * (4 + 2 + 2 + 4) + 2 * 2 * T * (F + -(-F // BLOCK)), "flops": 20 * T * F}
    if kind == "logp":  # the logits once a direction, the gradient written once
        V, b = case["V"], size(case["dtype"])
        return {"bytes": T * V * b * (3 if case["train"] else 1) + T * (4 * 4 + 8 * case["k"]),
                "flops": (14 if case["train"] else 6) * T * V}
    V, h = case["V"], case["h"]  # the used rows of the table, T rows out, T rows in, the whole gradient
    share = np.diff(np.log(np.arange(1, V + 1))) / math.log(V)  # of the tokens, by rank
    used = min(T, int(np.sum(1 - (1 - share) ** (0.97 * T))))
    return {"bytes": used * h * size(case["dtype"]) + T * h * (4 + 4) + V * h * size(case["grad"]) + 2 * 4 * T, "flops": 2 * T * h}


def _exact_round8(x, fmt):
    """The 8-bit block form's values of x (float64): the scale is the least power of two 2^e, e >= -127, with
    max|x| <= limit * 2^e; int8 rounds x / 2^e to the nearest whole number, e4m3 to a 4-bit significand with least
    exponent -6, both to even."""
    out = torch.empty_like(x)
    limit = 127.0 if fmt == "i8" else 448.0
    pow2 = lambda e: ((e.long() + 1023) << 52).view(torch.float64)  # noqa: E731
    for c in range(0, x.shape[1], BLOCK):
        v = x[:, c:c + BLOCK]
        a = v.abs().max(dim=1, keepdim=True).values
        e = torch.ceil(torch.log2(torch.where(a > 0, a, 1.0) / limit))
        # the logarithm may be off by a hair at the border: put it right by the definition itself
        e = torch.where(a <= limit * pow2(e - 1), e - 1, e)
        e = torch.where(a > limit * pow2(e), e + 1, e)
        e = torch.where(a > 0, e, -127.0).clamp(min=-127.0)
        q = v * pow2(-e)
        if fmt == "i8":
            q = torch.round(q)
        else:
            step = pow2(torch.frexp(q.abs())[1].clamp(min=-5) - 4)
            q = torch.round(q / step) * step
        out[:, c:c + BLOCK] = q * pow2(e)
    return out


def _exact_logp(s, k):
    z, ids, it = s["z"], s["ids"].long(), float(s["inv_temp"])
    T, V = z.shape
    f8 = dict(device="cuda", dtype=torch.float64)
    lse, logp, ent = torch.zeros(T, **f8), torch.zeros(T, **f8), torch.zeros(T, **f8)
    top_ids, top_logp = torch.full((T, k), -1, device="cuda", dtype=torch.int64), torch.zeros(T, k, **f8)
    dz = torch.zeros(T, V, **f8) if "g_logp" in s else None
    kept = torch.nonzero(ids >= 0)[:, 0]
    for part in kept.split(512):
        a = z[part].double()
        norm = torch.logsumexp(a * it, 1)
        lp = a * it - norm[:, None]
        p = torch.exp(lp)
        plp = torch.where(p > 0, p * lp.clamp(min=-1e300), 0.0)
        h = -plp.sum(1)
        lse[part], ent[part] = norm, h
        row = torch.arange(part.numel(), device="cuda")
        logp[part] = lp[row, ids[part]]
        if k:
            kth = torch.topk(a, k, dim=1).values[:, -1:]
            r, c = torch.nonzero((a >= kth) & (a > float("-inf")), as_tuple=True)  # in the order of rows, then columns
            order = torch.sort(a[r, c], descending=True, stable=True).indices
            order = order[torch.sort(r[order], stable=True).indices]
            r, c = r[order], c[order]
            first = torch.searchsorted(r, row)
            place = torch.arange(r.numel(), device="cuda") - first[r]
            r, c, place = r[place < k], c[place < k], place[place < k]
            ti = torch.full((part.numel(), k), -1, device="cuda")
            tl = torch.full((part.numel(), k), float("-inf"), **f8)
            ti[r, place], tl[r, place] = c, lp[r, c]
            top_ids[part], top_logp[part] = ti, tl
        if dz is not None:
            gl, ge = s["g_logp"][part].double(), s["g_ent"][part].double()
            # d logp_t / dz_j = [j = t] - p_j;  dH / dz_j = -p_j log p_j - p_j H
            g = -gl[:, None] * p - ge[:, None] * (plp + p * h[:, None])
            g[row, ids[part]] += gl
            dz[part] = g * it
    out = {"lse": lse, "logp": logp, "entropy": ent, "top_ids": top_ids.to(torch.int32), "top_logp": top_logp}
    if dz is not None:
        out["dlogits"] = dz
    return out


def exact(case, seed):
    s = prepare(case, seed)
    kind = case["kind"]
    if kind == "ckpt":
        return {"x": _exact_round8(s["x"].double(), case["fmt"])}
    if kind == "norm":
        x, w, dy = s["x"].double(), s["w"].double(), s["dy"].double()
        T, h = x.shape
        r = 1.0 / torch.sqrt((x * x).sum(1) / h + float(torch.tensor(1e-5)))
        y = x * w * r[:, None]
        n = _exact_round8(x, case["fmt"]) * r[:, None]
        dot = torch.einsum("th,h,th->t", dy, w, n) / h
        dx = s["resid"].double() + r[:, None] * (dy * w - n * dot[:, None])
        return {"y": y, "rstd": r, "dx": dx, "dx_bf16": dx, "dw": torch.einsum("th,th->h", dy, n)}
    if kind == "swiglu":
        F = case["F"]
        gu = s["gu"].double()
        act = gu[:, :F] * torch.sigmoid(gu[:, :F]) * gu[:, F:]
        g, u = _exact_round8(gu[:, :F], case["fmt"]), _exact_round8(gu[:, F:], case["fmt"])
        d, sg = s["dact"].double(), torch.sigmoid(g)
        dgu = torch.empty_like(gu)
        dgu[:, :F] = d * u * (sg + g * sg * (1 - sg))
        dgu[:, F:] = d * g * sg
        return {"act": act, "dgu": dgu}
    if kind == "logp":
        return _exact_logp(s, case["k"])
    ids = s["ids"].long()
    used = torch.nonzero(ids >= 0)[:, 0]
    scale = float(torch.tensor(s["scale"], dtype=torch.float32))
    out = torch.zeros(case["T"], case["h"], device="cuda", dtype=torch.float64)
    out[used] = s["table"][ids[used]].double() * scale
    grad = torch.zeros(case["V"], case["h"], device="cuda", dtype=torch.float64)
    grad.index_add_(0, ids[used], s["dout"][used].double() * scale)
    return {"out": out, "dtable": grad}
