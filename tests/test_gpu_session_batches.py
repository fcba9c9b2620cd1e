"""A session steps any batch up to the one it was made for: a smaller step
has the bits of a session of its own size and meets the oracle's bar, whatever
ran before it in the same arena."""
import numpy as np
import pytest

import oracle
from tests.common import TINY, TINY_GQA, TINY_MOE, make_params, make_tokens, with_layers
from tests.gpu_util import need_gpu
from tests.test_gpu_e2e import compare
from tests.test_gpu_train import _master_f32

pytestmark = pytest.mark.gpu


def _session(mt, cfg, B, S, K, dtype, **kw):
    shape = mt.ModelShape(cfg.n_layers, cfg.hidden, cfg.n_heads, cfg.n_kv_heads, cfg.head_dim, cfg.ffn_dim,
                          cfg.vocab, cfg.rope_theta, cfg.norm_eps, cfg.n_experts, cfg.top_k, cfg.expert_ffn)
    return mt.Session(shape, B, S, K, dtype, **kw)


def _same(a, b):
    return np.array_equal(np.asarray(a).view(np.uint8), np.asarray(b).view(np.uint8))


@pytest.mark.parametrize("B,S", [(1, 1), (1, 32), (3, 7), (3, 31), (2, 32)])
def test_a_smaller_first_step_meets_the_oracle(B, S):
    torch, mt = need_gpu()
    cfg = with_layers(TINY_GQA, 3)
    tok, lab = make_tokens(cfg, B, S, 201)
    packed = make_params(cfg, 202)
    with _session(mt, cfg, 3, 32, 2, mt.MT_F32) as s:
        s.params[:] = packed
        loss = s.step(tok, lab, 2)
        grads = s.grads.copy()
    l_ref, g_ref = oracle.forward_backward(cfg, packed, tok, lab)
    assert abs(loss - l_ref) <= 1e-3 * l_ref
    compare(cfg, grads, g_ref, tok, loss, l_ref)
    assert mt.mt_op_device_error() == 0


RUNS = [(1, 2, 32), (4, 2, 32), (2, 1, 32), (5, 2, 17), (3, 2, 32), (1, 1, 5), (2, 2, 32), (4, 1, 1)]


@pytest.mark.parametrize("cfg,bf16", [(with_layers(TINY, 5), False), (with_layers(TINY_GQA, 5), False),
                                      (with_layers(TINY_MOE, 5), True)], ids=["tiny", "tiny_gqa", "tiny_moe"])
def test_steps_of_changing_interval_and_batch(cfg, bf16):
    torch, mt = need_gpu()
    dt = mt.MT_BF16 if bf16 else mt.MT_F32
    packed = make_params(cfg, 224, bf16=bf16)
    with _session(mt, cfg, 2, 32, 5, dt) as s:
        s.params[:] = packed
        got = []
        for i, (K, B, S) in enumerate(RUNS):
            got.append((s.step(*make_tokens(cfg, B, S, 225 + i), K), s.grads.copy()))
    for i, (K, B, S) in enumerate(RUNS):
        with _session(mt, cfg, B, S, K, dt) as s:
            s.params[:] = packed
            assert s.step(*make_tokens(cfg, B, S, 225 + i), K) == got[i][0], RUNS[i]
            assert _same(s.grads, got[i][1]), RUNS[i]
    assert mt.mt_op_device_error() == 0


@pytest.mark.parametrize("fmt", [0, 1], ids=["fp32", "i8"])
def test_steps_of_changing_length(fmt):
    """Sequences of several attention tiles, whole and ragged, below the session's longest."""
    torch, mt = need_gpu()
    cfg = with_layers(TINY_GQA, 3)
    packed = make_params(cfg, 234)
    runs = [(1, 2, 129), (2, 2, 300), (1, 1, 200), (3, 2, 128), (2, 1, 257), (2, 2, 1), (1, 2, 300)]
    with _session(mt, cfg, 2, 300, 3, mt.MT_F32, ckpt_format=fmt) as s:
        s.params[:] = packed
        got = [(s.step(*make_tokens(cfg, B, S, 235 + i), K), s.grads.copy()) for i, (K, B, S) in enumerate(runs)]
    for i, (K, B, S) in enumerate(runs):
        with _session(mt, cfg, B, S, K, mt.MT_F32, ckpt_format=fmt) as s:
            s.params[:] = packed
            assert s.step(*make_tokens(cfg, B, S, 235 + i), K) == got[i][0], runs[i]
            assert _same(s.grads, got[i][1]), runs[i]
    assert mt.mt_op_device_error() == 0


def test_smaller_training_steps():
    """Synchronous and asynchronous steps of the host optimizer on batches below the session's."""
    torch, mt = need_gpu()
    cfg = with_layers(TINY_GQA, 3)
    packed = make_params(cfg, 244)
    opt = mt.adamw_cfg(3e-3, 0.9, 0.999, 1e-8, 0.01)
    batches = [make_tokens(cfg, B, S, 245 + i) for i, (B, S) in enumerate([(1, 9), (2, 32), (2, 8)])]
    for form in ("train_step", "train_step_async"):
        ends = []
        for size in ((2, 32), None):  # one session for all, then each step's losses from sessions of its own size
            if size:
                with _session(mt, cfg, *size, 2, mt.MT_F32) as s:
                    s.params[:] = packed
                    s.bind_optimizer(opt, _master_f32(cfg, packed, False), n_threads=3)
                    losses = [getattr(s, form)(tok, lab, 2) for tok, lab in batches]
                    if form.endswith("async"):
                        s.optimizer_flush()
                    ends.append((losses, s.params.copy(), s.opt_m.copy(), s.opt_v.copy()))
            else:
                params, master = packed.copy(), _master_f32(cfg, packed, False)
                m, v = np.zeros_like(master), np.zeros_like(master)
                losses, grads = [], []
                lag = 1 if form.endswith("async") else 0

                def update(k):
                    mt.mt_adamw_update(c, opt, k, 0, cfg.n_layers + 2, master.ctypes.data, m.ctypes.data, v.ctypes.data,
                                       grads[k - 1].ctypes.data, params.ctypes.data, mt.MT_F32, 2)

                for k, (tok, lab) in enumerate(batches, 1):
                    with _session(mt, cfg, *tok.shape, 2, mt.MT_F32) as s:
                        c = s.cfg
                        s.params[:] = params
                        losses.append(s.step(tok, lab, 2))
                        grads.append(s.grads.copy())
                    if k > lag:
                        update(k - lag)
                if lag:
                    update(len(batches))
                ends.append((losses, params, m, v))
        assert ends[0][0] == ends[1][0], form
        for a, b in zip(ends[0][1:], ends[1][1:]):
            assert _same(a, b), form


@pytest.mark.parametrize("cfg,bf16", [(with_layers(TINY, 4), False), (with_layers(TINY_MOE, 4), True)],
                         ids=["tiny", "tiny_moe"])
@pytest.mark.parametrize("fmt", [0, 1, 2], ids=["fp32", "i8", "e4m3"])
def test_what_the_arena_held_before_does_not_matter(cfg, bf16, fmt):
    """An arena of NaN bits (and of whole numbers -1): every value that a step reads, it has written."""
    torch, mt = need_gpu()
    dt = mt.MT_BF16 if bf16 else mt.MT_F32
    packed = make_params(cfg, 264, bf16=bf16)
    out = []
    for fill in (None, 0xff):
        shape = mt.make_cfg(cfg.n_layers, cfg.hidden, cfg.n_heads, cfg.n_kv_heads, cfg.head_dim, cfg.ffn_dim, cfg.vocab,
                            cfg.rope_theta, cfg.norm_eps, 2, 32, 3, dt, cfg.n_experts, cfg.top_k, cfg.expert_ffn,
                            ckpt_format=fmt)
        kw = {}
        if fill is not None:
            arena = torch.full((mt.mt_required_budget(shape),), fill, dtype=torch.uint8, device="cuda")
            torch.cuda.synchronize()
            kw = dict(device_arena=arena.data_ptr())
        runs = []
        for K, B, S in ((1, 1, 9), (3, 2, 32), (2, 2, 5)):
            if fill is not None:
                arena.fill_(fill)
                torch.cuda.synchronize()
            with _session(mt, cfg, 2, 32, 3, dt, ckpt_format=fmt, **kw) as s:
                s.params[:] = packed
                runs.append((s.step(*make_tokens(cfg, B, S, 265 + K), K), s.grads.copy()))
        out.append(runs)
    for (l0, g0), (l1, g1) in zip(*out):
        assert l0 == l1 and _same(g0, g1)
    assert mt.mt_op_device_error() == 0
