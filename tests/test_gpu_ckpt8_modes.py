"""8-bit residual checkpoints together with what else a step can do: against
the float64 step with the same rounding, with bf16 gradients, FP8 weights, the
host optimizer in both its forms, and sessions whose K and batch change."""
import numpy as np
import pytest

import oracle
from tests import ckpt8_ref as ref
from tests import ckpt8_step_ref
from tests.bounds import U16
from tests.common import SMALL, TINY, TINY_GQA, TINY_MOE, f32_to_bf16_bits, make_params, make_tokens, with_layers
from tests.gpu_util import need_gpu
from tests.test_gpu_fp8 import TINY176, _fp8_and_bf16_models
from tests.test_gpu_train import _master_f32

pytestmark = pytest.mark.gpu
both_formats = pytest.mark.parametrize("fmt", [ref.I8, ref.E4M3], ids=["i8", "e4m3"])


def _session(mt, cfg, B, S, K, fmt, dtype=None, **kw):
    shape = mt.ModelShape(cfg.n_layers, cfg.hidden, cfg.n_heads, cfg.n_kv_heads, cfg.head_dim, cfg.ffn_dim,
                          cfg.vocab, cfg.rope_theta, cfg.norm_eps, cfg.n_experts, cfg.top_k, cfg.expert_ffn)
    return mt.Session(shape, B, S, K, mt.MT_F32 if dtype is None else dtype, ckpt_format=fmt, **kw)


def _same(a, b):
    return np.array_equal(np.asarray(a).view(np.uint8), np.asarray(b).view(np.uint8))


@both_formats
@pytest.mark.parametrize("cfg,B,S,K", [(with_layers(TINY, 5), 2, 32, 1), (with_layers(TINY, 5), 3, 37, 2),
                                       (with_layers(TINY_GQA, 4), 2, 32, 3), (with_layers(SMALL, 3), 1, 96, 1)],
                         ids=["tiny_k1", "tiny_k2_ragged", "gqa_k3", "small_widths_k1"])
def test_gradients_against_the_step_with_the_same_rounding(fmt, cfg, B, S, K):
    """The bar of the step with fp32 checkpoints (relative L2 2e-2), held
    against the float64 step whose checkpoints are rounded alike, and past it
    only by what values at the border of two codes can do: the residual that
    is rounded here comes from bf16 products, each rounding of its operands off
    by at most U16. (E4M3's rounding moves the first layer's gradients by 3e-2
    to 5e-2, and its input has no such values, so a step that left the rounding
    out, or rounded something else, is outside.)"""
    torch, mt = need_gpu()
    tok, lab = make_tokens(cfg, B, S, 115)
    packed = make_params(cfg, 114)
    with _session(mt, cfg, B, S, K, fmt) as s:
        s.params[:] = packed
        loss = s.step(tok, lab, K)
        got = s.grads.copy()
    want, g = ckpt8_step_ref.step(cfg, packed, tok, lab, K, fmt)
    border = ckpt8_step_ref.borderline(cfg, packed, tok, lab, K, fmt, U16)
    assert abs(loss - want) <= 1e-2 * want
    worst = {}
    for name, a in oracle.unpack(cfg, got).items():
        err, bar = np.linalg.norm(a - g[name]) / np.linalg.norm(g[name]), 2e-2 + border[name]
        worst[name] = (f"{err:.2e}", f"{bar:.2e}")
        assert err <= bar, worst
    print(worst)
    assert mt.mt_op_device_error() == 0


@both_formats
def test_a_session_whose_interval_and_batch_change(fmt):
    """Every step gives the bits of a session of its own, whatever K, batch and
    length ran before it in the same arena."""
    torch, mt = need_gpu()
    cfg = with_layers(TINY_GQA, 5)
    packed = make_params(cfg, 124)
    runs = [(1, 2, 32), (4, 2, 32), (2, 1, 32), (5, 2, 17), (3, 2, 32), (1, 1, 5), (2, 2, 32)]
    with _session(mt, cfg, 2, 32, 5, fmt) as s:
        s.params[:] = packed
        got = []
        for i, (K, B, S) in enumerate(runs):
            tok, lab = make_tokens(cfg, B, S, 125 + i)
            got.append((s.step(tok, lab, K), s.grads.copy()))
    for i, (K, B, S) in enumerate(runs):
        tok, lab = make_tokens(cfg, B, S, 125 + i)
        with _session(mt, cfg, B, S, K, fmt) as s:
            s.params[:] = packed
            assert s.step(tok, lab, K) == got[i][0], runs[i]
            assert _same(s.grads, got[i][1]), runs[i]
    assert mt.mt_op_device_error() == 0


@both_formats
@pytest.mark.parametrize("cfg,bf16", [(with_layers(TINY, 3), False), (with_layers(TINY_MOE, 3), True)],
                         ids=["tiny", "tiny_moe"])
def test_bf16_gradients_are_the_rounded_fp32_ones(fmt, cfg, bf16):
    torch, mt = need_gpu()
    tok, lab = make_tokens(cfg, 2, 32, 135)
    packed = make_params(cfg, 134, bf16=bf16)
    res = []
    for gd in (mt.MT_F32, mt.MT_BF16):
        with _session(mt, cfg, 2, 32, 1, fmt, mt.MT_BF16 if bf16 else mt.MT_F32, grad_dtype=gd) as s:
            s.params[:] = packed
            res.append((s.step(tok, lab, 1), s.grads.copy()))
    (l32, g32), (l16, g16) = res
    assert l16 == l32
    want = np.zeros_like(g16)
    for unit, t, name, shape, _ in oracle.tensor_list(cfg):
        o16, n16 = oracle.tensor_offset(cfg, unit, t, True)
        o32, _ = oracle.tensor_offset(cfg, unit, t, False)
        want[o16 // 2:(o16 + n16) // 2] = f32_to_bf16_bits(g32[o32 // 4:o32 // 4 + n16 // 2])
    assert np.array_equal(g16, want)


@both_formats
@pytest.mark.parametrize("cfg", [TINY176, with_layers(TINY_MOE, 3)], ids=["dense", "moe"])
def test_fp8_weights_are_the_step_on_the_dequantised_ones(fmt, cfg):
    torch, mt = need_gpu()
    fp8, deq = _fp8_and_bf16_models(mt, cfg, 144, 2, 32, 1)
    tok, lab = make_tokens(cfg, 2, 32, 145)
    out = []
    for dtype, params in ((mt.MT_FP8, fp8), (mt.MT_BF16, deq)):
        with _session(mt, cfg, 2, 32, 1, fmt, dtype) as s:
            s.params[:] = params
            out.append((s.step(tok, lab, 1), s.grads.copy()))
    assert out[0][0] == out[1][0] and _same(out[0][1], out[1][1])


@both_formats
@pytest.mark.parametrize("cfg,bf16", [(with_layers(TINY_GQA, 4), False), (with_layers(TINY_MOE, 3), True)],
                         ids=["tiny_gqa", "tiny_moe"])
def test_train_step_is_step_then_update(fmt, cfg, bf16):
    torch, mt = need_gpu()
    dt = mt.MT_BF16 if bf16 else mt.MT_F32
    tok, lab = make_tokens(cfg, 2, 32, 151)
    packed = make_params(cfg, 152, bf16=bf16)
    opt = mt.adamw_cfg(2e-3, 0.9, 0.999, 1e-8, 0.01)
    units = cfg.n_layers + 2
    with _session(mt, cfg, 2, 32, 1, fmt, dt) as s:
        s.params[:] = packed
        s.bind_optimizer(opt, _master_f32(cfg, packed, bf16), n_threads=3)
        runs = [(s.train_step(tok, lab, 1), s.grads.copy(), s.params.copy(), s.opt_master.copy()) for _ in range(2)]
    with _session(mt, cfg, 2, 32, 1, fmt, dt) as s:
        s.params[:] = packed
        master = _master_f32(cfg, packed, bf16)
        m, v = np.zeros_like(master), np.zeros_like(master)
        for i in range(2):
            assert s.step(tok, lab, 1) == runs[i][0]
            mt.mt_adamw_update(s.cfg, opt, i + 1, 0, units, master.ctypes.data, m.ctypes.data, v.ctypes.data,
                               s.grads_ptr, s.params_ptr, dt, 2)
            for a, b in zip((s.grads, s.params, master), runs[i][1:]):
                assert _same(a, b)


@both_formats
def test_async_steps_follow_the_staleness_one_schedule(fmt):
    torch, mt = need_gpu()
    cfg = with_layers(TINY_GQA, 5)
    batches = [make_tokens(cfg, 2, 32, 160 + k) for k in range(3)]
    packed = make_params(cfg, 164)
    opt = mt.adamw_cfg(3e-3, 0.9, 0.999, 1e-8, 0.01)
    units = cfg.n_layers + 2
    with _session(mt, cfg, 2, 32, 2, fmt) as s:
        s.params[:] = packed
        s.bind_optimizer(opt, _master_f32(cfg, packed, False), n_threads=3)
        got = [(s.train_step_async(tok, lab, 2), s.grads.copy()) for tok, lab in batches]
        s.optimizer_flush()
        final = (s.params.copy(), s.opt_master.copy(), s.opt_m.copy(), s.opt_v.copy())
    with _session(mt, cfg, 2, 32, 2, fmt) as s:
        s.params[:] = packed
        master = _master_f32(cfg, packed, False)
        m, v = np.zeros_like(master), np.zeros_like(master)

        def update(k, g):
            mt.mt_adamw_update(s.cfg, opt, k, 0, units, master.ctypes.data, m.ctypes.data, v.ctypes.data,
                               g.ctypes.data, s.params_ptr, mt.MT_F32, 2)

        for k, (tok, lab) in enumerate(batches):
            assert s.step(tok, lab, 2) == got[k][0]
            assert _same(s.grads, got[k][1])
            if k >= 1:
                update(k, got[k - 1][1])
        update(3, got[2][1])
        for x, y in zip((s.params, master, m, v), final):
            assert _same(x, y)
