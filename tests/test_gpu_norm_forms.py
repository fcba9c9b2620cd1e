"""RMSNorm forward with and without the checkpoint: one formula, the sum of
squares added in two orders. Each sum of h squares (no cancellation) is within
acc(h) of itself, half of that in the root, and each form rounds y once."""
import numpy as np
import pytest

from tests.bounds import U16, U32, acc, check
from tests.gpu_util import from_dev, need_gpu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", [1, 2])
@pytest.mark.parametrize("T,h", [(1, 4), (3, 36), (77, 1024), (500, 4096), (33, 8192)])
def test_both_norm_forwards_agree_within_their_roundings(fmt, T, h):
    torch, mt = need_gpu()
    gen = torch.Generator(device="cuda").manual_seed(T * h)
    x = torch.randn((T, h), device="cuda", generator=gen) * 3
    w = 1 + 0.1 * torch.randn(h, device="cuda", generator=gen)
    y, y8 = (torch.empty((T, h), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    r, r8 = (torch.empty(T, device="cuda") for _ in range(2))
    codes = torch.empty((T, h), dtype=torch.uint8, device="cuda")
    scales = torch.empty((T, -(-h // 32)), dtype=torch.uint8, device="cuda")
    mt.mt_op_rmsnorm_fwd(x, w, y, r, T, h, 1e-5)
    mt.mt_op_rmsnorm_fwd_ckpt8(x, w, y8, r8, codes, scales, fmt, T, h, 1e-5)
    e = acc(h) + 8 * U32
    a, b = from_dev(r).astype(np.float64), from_dev(r8).astype(np.float64)
    check(b, a, e * a, "rstd")
    a, b = from_dev(y).astype(np.float64), from_dev(y8).astype(np.float64)
    check(b, a, (2 * U16 + 2 * e) * (1 + 2 * U16) * np.abs(a), "y")
