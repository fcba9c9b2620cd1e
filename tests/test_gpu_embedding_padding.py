"""Padding of the embedding lookup: zero bits for negative ids and for ids
past the table, whatever the scale."""
import pytest

from tests.gpu_util import need_gpu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("scale", [float("inf"), float("-inf"), float("nan"), -2.0, 0.0, 3.0e38])
@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("h", [1, 7, 64, 1028])
def test_padding_is_zero_under_every_scale(scale, bf16, h):
    torch, mt = need_gpu()
    V = 11
    dt, code = (torch.bfloat16, mt.MT_BF16) if bf16 else (torch.float32, mt.MT_F32)
    table = torch.ones((V, h), device="cuda").to(dt)
    ids = torch.tensor([3, -1, V - 1, -7, V, 0, -(1 << 31), (1 << 31) - 1], dtype=torch.int32, device="cuda")
    T = ids.numel()
    out = torch.full((T, h), 7.0, device="cuda").to(dt)
    mt.mt_op_embed_fwd(table, code, ids, scale, out, code, T, V, h)
    bits = out.view(torch.int16 if bf16 else torch.int32)
    padded = (ids < 0) | (ids >= V)
    assert int(torch.count_nonzero(bits[padded])) == 0
    want = torch.full((1,), scale, device="cuda").to(dt)  # one times the scale, rounded to the type
    got = out[~padded]
    assert torch.equal(got.nan_to_num(nan=5.0), want.nan_to_num(nan=5.0).expand_as(got))
    assert mt.mt_op_device_error() != 0  # ids past the table
    assert mt.mt_op_device_error() == 0
