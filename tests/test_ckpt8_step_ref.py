"""The float64 step with rounded checkpoints: without the rounding it is the
oracle's step, and the rounding moves only what lies below the top block."""
import numpy as np
import pytest

import oracle
from tests import ckpt8_ref, ckpt8_step_ref
from tests.common import TINY, TINY_GQA, make_params, make_tokens, params_f64, with_layers


@pytest.mark.parametrize("cfg", [TINY, with_layers(TINY_GQA, 4)], ids=["tiny", "tiny_gqa_4l"])
@pytest.mark.parametrize("K", [1, 2, 3])
def test_without_rounding_it_is_the_oracle(cfg, K):
    tok, lab = make_tokens(cfg, 2, 19, 5)
    packed = make_params(cfg, 6)
    loss, g = ckpt8_step_ref.step(cfg, packed, tok, lab, K, None)
    want, flat = oracle.forward_backward_f64(cfg, params_f64(cfg, packed), tok, lab)
    assert abs(loss - want) < 1e-12 * want
    for unit, t, name, shape, _ in oracle.tensor_list(cfg):
        off, nb = oracle.tensor_offset(cfg, unit, t)
        w = flat[off // 4:(off + nb) // 4].reshape(shape)
        assert np.abs(g[name] - w).max() <= 1e-10 * np.abs(w).max(), name


@pytest.mark.parametrize("fmt", [ckpt8_ref.I8, ckpt8_ref.E4M3])
def test_rounding_moves_what_lies_below_the_top_block(fmt):
    cfg = with_layers(TINY_GQA, 4)
    tok, lab = make_tokens(cfg, 2, 19, 7)
    packed = make_params(cfg, 8)
    l0, a = ckpt8_step_ref.step(cfg, packed, tok, lab, 2, None)
    l1, b = ckpt8_step_ref.step(cfg, packed, tok, lab, 2, fmt)
    assert l0 == l1
    for name in a:
        same = name in ("w_final_norm", "w_out") or name.startswith(("layer2", "layer3"))
        assert np.array_equal(a[name], b[name]) == same, name
