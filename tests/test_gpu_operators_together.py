"""The checkpoint, token and embedding operators run together, as a scored
and trained one-layer model would: lookup, norm with an 8-bit checkpoint,
vocabulary product, log probabilities and entropy, and back.

Against float64 the chain carries a few independent bf16 roundings (the norm's
output, the logits' gradient: RMS 2^-9.8 each, into the logits and from there
into every gradient), held to the step's bar of rel-L2 2e-2. Captured into a
graph, on other streams and side by side the operators give the same bits.
"""
import subprocess
import sys
from pathlib import Path

import numpy as np
import pytest

from tests import ckpt8_ref as ref
from tests.common import rel_l2
from tests.gpu_util import from_dev, need_gpu

pytestmark = pytest.mark.gpu


class Chain:
    """Buffers of one model and batch; run() issues every operator once on the current stream."""

    def __init__(self, torch, mt, T, V, h, fmt, k, seed):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        n = lambda *s, std=1.0: torch.empty(s, device="cuda").normal_(0, std, generator=g)  # noqa: E731
        e = lambda *s, dt=torch.float32: torch.full(s, 7, device="cuda").to(dt)  # noqa: E731
        bf, u8 = torch.bfloat16, torch.uint8
        self.torch, self.mt, self.dims = torch, mt, (T, V, h, fmt, k)
        self.table = n(V, h, std=0.02).to(bf)
        self.norm_w = 1 + 0.1 * n(h)
        self.head = n(V, h, std=0.05).to(bf)
        self.new_batch(seed)
        self.x, self.y, self.rstd = e(T, h), e(T, h, dt=bf), e(T)
        self.codes, self.scales = e(T, h, dt=u8), e(T, -(-h // 32), dt=u8)
        self.z, self.dz = e(T, V), e(T, V, dt=bf)
        self.lse, self.logp, self.ent = e(T), e(T), e(T)
        self.top_ids, self.top_logp = e(T, k, dt=torch.int32), e(T, k)
        self.dy, self.dx, self.dw = e(T, h), e(T, h), e(h)
        self.dhead, self.dtable = e(V, h), e(V, h)
        self.ws_norm = e(mt.mt_op_rmsnorm_bwd_ckpt8_workspace(T, h))
        self.ws_embed = e(mt.mt_op_embed_bwd_workspace(T, V, h), dt=u8)

    def new_batch(self, seed):
        T, V = self.dims[:2]
        rng = np.random.default_rng(seed)
        ids, nxt = rng.integers(0, V, T), rng.integers(0, V, T)
        ids[: T // 4] = 3  # a frequent token
        nxt[T // 3] = -1   # one position is not scored
        put = lambda name, a: (getattr(self, name).copy_(a) if hasattr(self, name) else setattr(self, name, a.clone()))  # noqa: E731
        put("ids", self.torch.from_numpy(ids.astype(np.int32)).cuda())
        put("next", self.torch.from_numpy(nxt.astype(np.int32)).cuda())
        put("g_logp", self.torch.from_numpy(rng.standard_normal(T).astype(np.float32)).cuda())
        put("g_ent", self.torch.from_numpy(0.1 * rng.standard_normal(T).astype(np.float32)).cuda())

    def run(self):
        mt = self.mt
        T, V, h, fmt, k = self.dims
        scale = float(np.float32(np.sqrt(h)))
        mt.mt_op_embed_fwd(self.table, mt.MT_BF16, self.ids, scale, self.x, mt.MT_F32, T, V, h)
        mt.mt_op_rmsnorm_fwd_ckpt8(self.x, self.norm_w, self.y, self.rstd, self.codes, self.scales, fmt, T, h, 1e-5)
        mt.mt_op_gemm(mt.MT_GEMM_NT, mt.MT_EPI_F32, self.y, self.head, self.z, None, T, V, h, h, h, V)
        mt.mt_op_token_logprobs(self.z, mt.MT_F32, self.next, 1.0, k, self.lse, self.logp, self.ent, self.top_ids,
                                self.top_logp, T, V, V)
        mt.mt_op_token_logprobs_bwd(self.z, mt.MT_F32, self.next, 1.0, self.lse, self.ent, self.g_logp, self.g_ent,
                                    self.dz, mt.MT_BF16, T, V, V, V)
        mt.mt_op_gemm(mt.MT_GEMM_NN, mt.MT_EPI_F32, self.dz, self.head, self.dy, None, T, h, V, V, h, h)
        mt.mt_op_gemm(mt.MT_GEMM_TN, mt.MT_EPI_F32, self.dz, self.y, self.dhead, None, V, h, T, V, h, h)
        mt.mt_op_rmsnorm_bwd_ckpt8(self.codes, self.scales, fmt, self.norm_w, self.rstd, self.dy, None, self.dx, None,
                                   self.dw, self.ws_norm, T, h)
        mt.mt_op_embed_bwd(self.ids, self.dx, mt.MT_F32, scale, self.dtable, mt.MT_F32, 0, self.ws_embed, T, V, h)

    OUT = ("y", "rstd", "codes", "scales", "lse", "logp", "ent", "top_ids", "top_logp", "dz", "dx", "dw", "dhead", "dtable")

    def outputs(self):
        return {n: getattr(self, n).clone() for n in self.OUT}


def _same(torch, a, b):
    return all(torch.equal(a[n], b[n]) for n in Chain.OUT)


@pytest.mark.parametrize("fmt", [ref.I8, ref.E4M3])
def test_chain_against_float64(fmt):
    torch, mt = need_gpu()
    T, V, h, k = 96, 1000, 128, 5
    c = Chain(torch, mt, T, V, h, fmt, k, 3)
    c.run()
    E, H = from_dev(c.table).astype(np.float64), from_dev(c.head).astype(np.float64)
    w, ids, nxt = from_dev(c.norm_w).astype(np.float64), c.ids.cpu().numpy(), c.next.cpu().numpy()
    gl, ge = from_dev(c.g_logp).astype(np.float64), from_dev(c.g_ent).astype(np.float64)
    scale = float(np.float32(np.sqrt(h)))
    x = E[ids] * scale
    r = 1 / np.sqrt((x ** 2).mean(axis=1, keepdims=True) + 1e-5)
    y = x * r * w
    z = y @ H.T
    lp = z - np.log(np.exp(z).sum(axis=1, keepdims=True))
    p = np.exp(lp)
    ent = -(p * lp).sum(axis=1)
    keep = nxt >= 0
    logp = np.where(keep, lp[np.arange(T), np.maximum(nxt, 0)], 0)
    assert np.max(np.abs(from_dev(c.logp) - logp)) < 2e-2
    assert rel_l2(from_dev(c.ent), np.where(keep, ent, 0)) < 2e-2
    hot = np.zeros((T, V))
    hot[np.arange(T), np.maximum(nxt, 0)] = 1
    dz = gl[:, None] * (hot - p) - ge[:, None] * p * (lp + ent[:, None])
    dz[~keep] = 0
    dy, dhead = dz @ H, dz.T @ y
    xh = ref.values_of((x).astype(np.float32), fmt) * r
    g = dy * w
    dx = r * (g - xh * (g * xh).mean(axis=1, keepdims=True))
    dE = np.zeros((V, h))
    np.add.at(dE, ids, dx * scale)
    assert rel_l2(from_dev(c.dhead), dhead) < 2e-2
    assert rel_l2(from_dev(c.dw), (dy * xh).sum(axis=0)) < 2e-2
    assert rel_l2(from_dev(c.dx), dx) < 2e-2
    assert rel_l2(from_dev(c.dtable), dE) < 2e-2
    # the listed tokens are the largest logits the product gave
    zz = from_dev(c.z)
    want = np.stack([np.lexsort((np.arange(V), -zz[t]))[:k] for t in range(T)])
    want[~keep] = -1
    assert np.array_equal(c.top_ids.cpu().numpy(), want)
    assert mt.mt_op_device_error() == 0


@pytest.mark.parametrize("T,V,h", [(96, 1000, 128), (5, 40008, 256), (3000, 512, 64)])
def test_chain_in_a_graph(T, V, h):
    """Captured once, replayed on changed inputs: the bits of the direct calls."""
    torch, mt = need_gpu()
    c = Chain(torch, mt, T, V, h, ref.E4M3, 8, 1)
    c.run()
    first = c.outputs()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.run()
    graph.replay()
    torch.cuda.synchronize()
    assert _same(torch, c.outputs(), first)
    c.new_batch(2)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    replayed = c.outputs()
    assert not torch.equal(replayed["logp"], first["logp"])
    c.run()
    assert _same(torch, c.outputs(), replayed)
    assert mt.mt_op_device_error() == 0


def test_chains_side_by_side_on_other_streams():
    torch, mt = need_gpu()
    a = Chain(torch, mt, 700, 3000, 256, ref.I8, 4, 7)
    b = Chain(torch, mt, 64, 32000, 128, ref.E4M3, 20, 8)
    a.run(), b.run()
    want = a.outputs(), b.outputs()
    torch.cuda.synchronize()
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(5):
        with torch.cuda.stream(s):
            a.run()
        with torch.cuda.stream(t):
            b.run()
    torch.cuda.synchronize()
    assert _same(torch, a.outputs(), want[0]) and _same(torch, b.outputs(), want[1])
    assert mt.mt_op_device_error() == 0


FIRST_CALLS = {
    "norm": "mt.mt_op_rmsnorm_bwd_ckpt8(c, c, 2, x, x, x, x, y, None, y[-h:], ws, 77, h)",
    "norm_no_residual": "mt.mt_op_rmsnorm_bwd_ckpt8(c, c, 1, x, x, x, None, y, None, y[-h:], ws, 777, 2 * h)",
    "logp": "mt.mt_op_token_logprobs(x, 1, ids, 1.0, 32, y, y[9:], None, ids[64:], y[64:], 1, 151936, 151936)",
    "embed": "mt.mt_op_embed_bwd(ids, x, 1, 1.0, y, 0, 0, ws, 17000, 100, h)",
    "embed_odd": "mt.mt_op_embed_bwd(ids, x, 0, 1.0, y, 1, 0, ws, 2000, 100, h + 1)",
}


@pytest.mark.parametrize("call", sorted(FIRST_CALLS))
def test_first_call_of_a_process(call):
    """A kernel's shared memory is asked for by the call that needs it, not
    by an earlier one of another size."""
    need_gpu()
    code = ("import torch, layer_streamed_gb300 as mt\n"
            "h, z = 1024, lambda n, t=torch.float32: torch.zeros(n, dtype=t, device='cuda')\n"
            "x, y, ws = z(20 << 20), z(20 << 20), z(20 << 20)\n"
            "c, ids = z(4 << 20, torch.uint8), z(1 << 20, torch.int32)\n"
            f"{FIRST_CALLS[call]}\n"
            "torch.cuda.synchronize()\n"
            "assert mt.mt_op_device_error() == 0 and bool(torch.isfinite(y).all())\n")
    r = subprocess.run([sys.executable, "-c", code], cwd=Path(__file__).resolve().parent.parent, capture_output=True,
                       text=True, timeout=120)
    assert r.returncode == 0, r.stderr


@pytest.mark.parametrize("captured", [False, True])
def test_inputs_from_copies_fills_and_other_streams(captured):
    """Kernels that may begin early still wait for whatever wrote their
    inputs: a copy, a fill, a library kernel, another stream's event, and the
    operator before them; what they write is waited for in turn."""
    torch, mt = need_gpu()
    T, n = 4096, 2048
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    rounds = [torch.randn((T, n), device="cuda", generator=g) for _ in range(3)]
    x, back = torch.empty((T, n), device="cuda"), torch.empty((T, n), device="cuda")
    y = torch.empty((T, n), device="cuda")
    codes, scales = (torch.empty(s, dtype=torch.uint8, device="cuda") for s in ((T, n), (T, n // 32)))
    ids = torch.zeros(T, dtype=torch.int32, device="cuda")
    lse, logp = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    side, outs = torch.cuda.Stream(), [torch.empty((T, n), device="cuda") for _ in range(4)]

    def pack_unpack(out):
        mt.mt_op_ckpt8_pack(x, mt.MT_F32, 1, codes, scales, T, n, n, n)
        mt.mt_op_ckpt8_unpack(codes, scales, 1, back, mt.MT_F32, T, n, n, n)
        out.copy_(back)  # a copy reads what the operator writes; the next round writes it again

    def issue():
        main = torch.cuda.current_stream()
        for r, out in zip(rounds, outs):
            x.copy_(r)
            pack_unpack(out)
        x.zero_()
        mt.mt_op_token_logprobs(x, mt.MT_F32, ids, 1.0, 0, lse, logp, None, None, None, T, n, n)
        side.wait_stream(main)
        with torch.cuda.stream(side):
            torch.mul(rounds[0], 3.0, out=y)
            for _ in range(20):
                y.add_(rounds[1])
        main.wait_stream(side)
        mt.mt_op_ckpt8_pack(y, mt.MT_F32, 2, codes, scales, T, n, n, n)
        mt.mt_op_ckpt8_unpack(codes, scales, 2, back, mt.MT_F32, T, n, n, n)
        outs[3].copy_(back)

    if captured:
        graph = torch.cuda.CUDAGraph()
        warm = torch.cuda.Stream()
        with torch.cuda.stream(warm):
            issue()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            issue()
        run = graph.replay
    else:
        run = issue
    z = rounds[0] * 3.0
    for _ in range(20):
        z.add_(rounds[1])
    want = []
    for r, fmt in [(q, 1) for q in rounds] + [(z, 2)]:
        torch.cuda.synchronize()
        w = torch.empty((T, n), device="cuda")
        mt.mt_op_ckpt8_pack(r, mt.MT_F32, fmt, codes, scales, T, n, n, n)
        torch.cuda.synchronize()
        mt.mt_op_ckpt8_unpack(codes, scales, fmt, w, mt.MT_F32, T, n, n, n)
        torch.cuda.synchronize()
        want.append(w)
    for _ in range(10):
        for o in outs:
            o.fill_(7.0)
        lse.fill_(7.0)
        run()
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            assert torch.equal(o, w)
        assert np.allclose(from_dev(lse), np.log(n), rtol=0, atol=2e-6)  # S = n exactly; ln n to a few units of 2^-22
    assert mt.mt_op_device_error() == 0
