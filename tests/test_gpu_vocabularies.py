"""Vocabularies off a multiple of eight, in one slice of the head and in
several: the step meets the oracle's bar with fp32, bf16 and FP8 weights."""
import numpy as np
import pytest

import oracle
from tests.common import TINY_GQA, TINY_MOE, make_params, make_tokens, with_layers
from tests.gpu_util import need_gpu
from tests.test_gpu_e2e import compare
from tests.test_gpu_fp8 import _fp8_and_bf16_models

pytestmark = pytest.mark.gpu


def _with(cfg, **kw):
    return oracle.Config(**{**cfg.__dict__, **kw})


def _step(mt, cfg, dtype, params, tok, lab, K):
    shape = mt.ModelShape(cfg.n_layers, cfg.hidden, cfg.n_heads, cfg.n_kv_heads, cfg.head_dim, cfg.ffn_dim,
                          cfg.vocab, cfg.rope_theta, cfg.norm_eps, cfg.n_experts, cfg.top_k, cfg.expert_ffn)
    with mt.Session(shape, *tok.shape, K, dtype) as s:
        s.params[:] = params
        return s.step(tok, lab, K), s.grads.copy()


@pytest.mark.parametrize("V", [1, 7, 97, 300, 1001, 2049])
@pytest.mark.parametrize("bf16", [False, True])
def test_any_vocabulary_meets_the_oracle(V, bf16):
    torch, mt = need_gpu()
    cfg = _with(with_layers(TINY_GQA, 2), vocab=V, ffn_dim=176)
    tok, lab = make_tokens(cfg, 2, 25, 301 + V)
    packed = make_params(cfg, 302, bf16=bf16)
    loss, grads = _step(mt, cfg, mt.MT_BF16 if bf16 else mt.MT_F32, packed, tok, lab, 1)
    l_ref, g_ref = oracle.forward_backward(cfg, packed, tok, lab, bf16=bf16)
    if V == 1:  # one token is certain: no loss and no gradient, up to the rounding of lse
        assert abs(loss) <= 1e-6 and l_ref == 0 and float(np.abs(grads).max()) <= 1e-5
    else:
        compare(cfg, grads, g_ref, tok, loss, l_ref)
    assert mt.mt_op_device_error() == 0


@pytest.mark.parametrize("cfg", [_with(with_layers(TINY_GQA, 2), vocab=301, ffn_dim=176),
                                 _with(with_layers(TINY_MOE, 2), vocab=301)], ids=["dense", "moe"])
def test_fp8_weights(cfg):
    torch, mt = need_gpu()
    fp8, deq = _fp8_and_bf16_models(mt, cfg, 311, 2, 25, 1)
    tok, lab = make_tokens(cfg, 2, 25, 312)
    l8, g8 = _step(mt, cfg, mt.MT_FP8, fp8, tok, lab, 1)
    lb, gb = _step(mt, cfg, mt.MT_BF16, deq, tok, lab, 1)
    assert l8 == lb and np.array_equal(g8.view(np.uint32), gb.view(np.uint32))


def test_several_slices_and_an_odd_last_one():
    """A layer buffer that holds 256 rows of the head at a time."""
    torch, mt = need_gpu()
    cfg = _with(with_layers(TINY_GQA, 2), vocab=2049, ffn_dim=8)
    tok, lab = make_tokens(cfg, 2, 25, 321)
    packed = make_params(cfg, 322)
    loss, grads = _step(mt, cfg, mt.MT_F32, packed, tok, lab, 2)
    l_ref, g_ref = oracle.forward_backward(cfg, packed, tok, lab)
    compare(cfg, grads, g_ref, tok, loss, l_ref)
