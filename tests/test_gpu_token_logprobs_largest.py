"""Token log probabilities of a row of 2^31 - 1 logits: the last index that
an int32 names, on and off the 16-byte boundary."""
import numpy as np
import pytest

from tests.bounds import U32, acc
from tests.gpu_util import from_dev, need_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture
def emptied():
    """Gives the large buffers back to the device."""
    yield
    import torch
    torch.cuda.empty_cache()


@pytest.mark.parametrize("bf16,off", [(True, 0), (True, 3), (False, 0), (False, 1)])
def test_largest_row(emptied, bf16, off):
    """A few logits stand out, the last two among them. The rest are equal:
    a thread adds 2^18 equal terms a sum, each rounding by half a step at
    most, so 2^18 * 2^-24 of the sum, which acc(V) covers."""
    torch, mt = need_gpu()
    V, k = (1 << 31) - 1, 5
    dt, code = (torch.bfloat16, mt.MT_BF16) if bf16 else (torch.float32, mt.MT_F32)
    flat = torch.zeros(V + off, dtype=dt, device="cuda")
    z = flat[off:]
    tops = {V - 1: 20.0, 0: 19.0, V - 2: 18.0, (1 << 30) + 1: 17.0, V - 9: 16.0}
    for i, v in tops.items():
        z[i] = v
    ids = torch.tensor([V - 1], dtype=torch.int32, device="cuda")
    lse, logp, ent = (torch.full((1,), 7.0, device="cuda") for _ in range(3))
    ti, tl = torch.zeros((1, k), dtype=torch.int32, device="cuda"), torch.zeros((1, k), device="cuda")
    mt.mt_op_token_logprobs(z, code, ids, 1.0, k, lse, logp, ent, ti, tl, 1, V, V)
    values = np.array(list(tops.values()))
    S = np.exp(values - 20).sum() + (V - len(tops)) * np.exp(-20.0)
    want = 20 + np.log(S)
    bound = acc(V) + 2.0 ** -20 + 4 * U32 * want
    assert abs(float(lse) - want) <= bound
    assert abs(float(logp) - (20 - want)) <= bound
    assert ti.tolist() == [list(tops)]
    assert np.all(np.abs(from_dev(tl)[0] - (values - want)) <= bound)
    # a NaN in the last place makes the row NaN, one in front of the row does not
    if off:
        flat[off - 1] = float("nan")
        mt.mt_op_token_logprobs(z, code, ids, 1.0, 0, lse, logp, None, None, None, 1, V, V)
        assert abs(float(lse) - want) <= bound
    z[V - 1] = float("nan")
    mt.mt_op_token_logprobs(z, code, ids, 1.0, 0, lse, logp, ent, None, None, 1, V, V)
    assert bool(torch.isnan(lse).all() and torch.isnan(logp).all() and torch.isnan(ent).all())
    assert mt.mt_op_device_error() == 0
