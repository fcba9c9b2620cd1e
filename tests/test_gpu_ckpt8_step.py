"""8-bit residual checkpoints in the streamed step (ckpt_format).

Exact properties: the forward and the top block never touch a rounded value,
so the loss, the head's gradients and the top block's are the bits of fp32
checkpoints, and everything is when one block holds all layers. Where the
checkpointed residual is exactly representable in 8 bits the recompute sees
the same values too: only the first layer's attention-norm backward, which
reads the packed form and adds in another order, may differ, by the rounding
of its fp32 sums.
"""
import numpy as np
import pytest

import oracle
from tests import ckpt8_ref as ref
from tests.bounds import acc
from tests.common import TINY, TINY_GQA, TINY_MOE, make_params, make_tokens, with_layers
from tests.gpu_util import need_gpu

pytestmark = pytest.mark.gpu


def _step(mt, cfg, packed, tok, lab, K, fmt, bf16=False, steps=1):
    shape = mt.ModelShape(cfg.n_layers, cfg.hidden, cfg.n_heads, cfg.n_kv_heads, cfg.head_dim, cfg.ffn_dim,
                          cfg.vocab, cfg.rope_theta, cfg.norm_eps, cfg.n_experts, cfg.top_k, cfg.expert_ffn)
    B, S = tok.shape
    with mt.Session(shape, B, S, K, mt.MT_BF16 if bf16 else mt.MT_F32, ckpt_format=fmt) as s:
        s.params[:] = packed
        for _ in range(steps):
            loss = s.step(tok, lab, K)
        g = s.grads.copy()
        plan = s.memory_plan()
    assert mt.mt_op_device_error() == 0
    return loss, g, plan


def _tensors(cfg, g):
    for unit, t, name, shape, _ in oracle.tensor_list(cfg):
        off, nb = oracle.tensor_offset(cfg, unit, t, False)
        yield unit, t, name, g[off // 4:(off + nb) // 4]


def _whole_embedding(cfg, packed, seed, bf16):
    """Embedding rows of whole numbers within +-15 times 2^-9: exact in both formats."""
    off, nb = oracle.tensor_offset(cfg, 0, 0, bf16)
    e = np.random.default_rng(seed).integers(-15, 16, cfg.vocab * cfg.hidden).astype(np.float32) * 2.0 ** -9
    view = packed[off:off + nb]
    if bf16:
        view.view(np.uint16)[:] = (e.view(np.uint32) >> 16).astype(np.uint16)
    else:
        view.view(np.float32)[:] = e


@pytest.mark.parametrize("fmt", [ref.I8, ref.E4M3])
@pytest.mark.parametrize("cfg,bf16", [(TINY, False), (TINY_MOE, True)], ids=["tiny", "tiny_moe"])
def test_one_block_is_bitwise_the_fp32_step(fmt, cfg, bf16):
    torch, mt = need_gpu()
    tok, lab = make_tokens(cfg, 2, 32, 5)
    packed = make_params(cfg, 4, bf16=bf16)
    l0, g0, _ = _step(mt, cfg, packed, tok, lab, cfg.n_layers, mt.MT_CKPT_F32, bf16)
    l1, g1, _ = _step(mt, cfg, packed, tok, lab, cfg.n_layers, fmt, bf16)
    assert l0 == l1 and np.array_equal(g0, g1)


@pytest.mark.parametrize("fmt", [ref.I8, ref.E4M3])
@pytest.mark.parametrize("cfg,bf16,K", [(with_layers(TINY, 5), False, 1), (with_layers(TINY_GQA, 5), False, 2),
                                        (with_layers(TINY_GQA, 4), False, 3), (with_layers(TINY_MOE, 3), True, 1)])
def test_loss_and_top_block_are_bitwise_and_the_rest_close(fmt, cfg, bf16, K):
    torch, mt = need_gpu()
    tok, lab = make_tokens(cfg, 2, 32, 15)
    packed = make_params(cfg, 14, bf16=bf16)
    l0, g0, p0 = _step(mt, cfg, packed, tok, lab, K, mt.MT_CKPT_F32, bf16)
    l1, g1, p1 = _step(mt, cfg, packed, tok, lab, K, fmt, bf16, steps=2)
    assert l0 == l1
    nb = -(-cfg.n_layers // K)
    top = (nb - 1) * K + 1
    rel = {1: 2.0 ** -6, 2: 2.0 ** -4}[fmt]  # at most, of a block's maximum (i8) or of the value (e4m3)
    for (unit, t, name, a), (_, _, _, b) in zip(_tensors(cfg, g0), _tensors(cfg, g1)):
        if unit >= top:
            assert np.array_equal(a, b), (unit, name)
        else:  # the rounded residual enters every lower gradient a few times over
            assert np.linalg.norm(a - b) <= 8 * rel * np.linalg.norm(a), (unit, name)
    assert p1["checkpoints"] <= p0["checkpoints"] // 3
    # repeated steps and sessions give the same bits
    l2, g2, _ = _step(mt, cfg, packed, tok, lab, K, fmt, bf16)
    assert l2 == l1 and np.array_equal(g1, g2)


@pytest.mark.parametrize("fmt", [ref.I8, ref.E4M3])
@pytest.mark.parametrize("cfg,bf16", [(TINY, False), (TINY_GQA, False), (TINY_MOE, True)],
                         ids=["tiny", "tiny_gqa", "tiny_moe"])
def test_representable_checkpoint_gives_the_fp32_gradients(fmt, cfg, bf16):
    torch, mt = need_gpu()
    tok, lab = make_tokens(cfg, 2, 32, 25)
    packed = make_params(cfg, 24, bf16=bf16)
    _whole_embedding(cfg, packed, 23, bf16)
    l0, g0, _ = _step(mt, cfg, packed, tok, lab, 1, mt.MT_CKPT_F32, bf16)
    l1, g1, _ = _step(mt, cfg, packed, tok, lab, 1, fmt, bf16)
    assert l0 == l1
    for (unit, t, name, a), (_, _, _, b) in zip(_tensors(cfg, g0), _tensors(cfg, g1)):
        if (unit, t) in ((0, 0), (1, 0)):  # behind the norm that reads the packed form
            assert np.max(np.abs(a - b)) <= 4 * acc(max(cfg.hidden, tok.size)) * np.max(np.abs(a)), name
        else:
            assert np.array_equal(a, b), (unit, name)


def test_recomputed_top_block(monkeypatch):
    """With the top block recomputed too (MT_FUSE_TOP_BLOCK=0) its checkpoint is packed as well."""
    torch, mt = need_gpu()
    monkeypatch.setenv("MT_FUSE_TOP_BLOCK", "0")
    cfg = with_layers(TINY, 3)
    tok, lab = make_tokens(cfg, 2, 32, 35)
    packed = make_params(cfg, 34)
    l0, g0, _ = _step(mt, cfg, packed, tok, lab, 2, mt.MT_CKPT_F32)
    l1, g1, _ = _step(mt, cfg, packed, tok, lab, 2, mt.MT_CKPT_I8)
    assert l0 == l1
    same = {(u, t): np.array_equal(a, b) for (u, t, _, a), (_, _, _, b) in zip(_tensors(cfg, g0), _tensors(cfg, g1))}
    assert same[(cfg.n_layers + 1, 0)] and same[(cfg.n_layers + 1, 1)]
    assert not same[(3, 1)]
    assert np.linalg.norm(g0 - g1) <= 8 * 2.0 ** -6 * np.linalg.norm(g0)
