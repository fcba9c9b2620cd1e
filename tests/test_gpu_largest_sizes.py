"""The row counts that the checkpoint, token and embedding operators accept,
at their largest: narrow rows, checked at both ends (and as a whole where a
comparison on the device is cheap). Values are chosen so that results are
exact, or bounded as beside each check."""
import math

import pytest

from tests.bounds import U16, U32
from tests.gpu_util import need_gpu

pytestmark = pytest.mark.gpu
EDGE = 1000


@pytest.fixture(autouse=True)
def emptied():
    """Gives the large buffers back to the device."""
    yield
    import torch
    torch.cuda.empty_cache()


def _ends(T):
    return (slice(0, EDGE), slice(T // 2, T // 2 + EDGE), slice(T - EDGE, T))


def _mod(torch, T, m, dtype):
    """0, 1, .., m - 1, 0, .. of length T."""
    return torch.arange(m, device="cuda").to(dtype).repeat(-(-T // m))[:T]


@pytest.mark.parametrize("fmt", [1, 2])
def test_checkpoint_of_2_to_30_rows(fmt):
    """Whole numbers up to 15 are exact in both forms, a block a row."""
    torch, mt = need_gpu()
    T = 1 << 30
    x = _mod(torch, T, 31, torch.float32) - 15
    codes, scales = (torch.empty(T, dtype=torch.uint8, device="cuda") for _ in range(2))
    mt.mt_op_ckpt8_pack(x, mt.MT_F32, fmt, codes, scales, T, 1, 1, 1)
    back = torch.full((T,), float("nan"), device="cuda")
    mt.mt_op_ckpt8_unpack(codes, scales, fmt, back, mt.MT_F32, T, 1, 1, 1)
    assert torch.equal(back, x)


def test_swiglu_of_2_to_30_rows():
    """One column: act and both gradients at the ends against float64, one bf16 rounding and the sigmoid's few ulp."""
    torch, mt = need_gpu()
    T, fmt = 1 << 30, 1
    gu = (_mod(torch, 2 * T, 31, torch.bfloat16) - 15) / 4  # exact in 8 bits too
    act = torch.empty(T, dtype=torch.bfloat16, device="cuda")
    codes, scales = (torch.empty(2 * T, dtype=torch.uint8, device="cuda") for _ in range(2))
    mt.mt_op_swiglu_fwd_ckpt8(gu, act, codes, scales, fmt, T, 1, 1)
    dgu = torch.empty(2 * T, dtype=torch.bfloat16, device="cuda")
    dact = torch.full((T,), 2.0, dtype=torch.bfloat16, device="cuda")
    mt.mt_op_swiglu_bwd_ckpt8(codes, scales, fmt, dact, dgu, T, 1, 1)
    for e in _ends(T):
        g, u = gu.view(T, 2)[e].double().unbind(1)
        s = torch.sigmoid(g)
        for got, want in ((act[e], g * s * u), (dgu.view(T, 2)[e, 0], 2 * u * s * (1 + g * (1 - s))),
                          (dgu.view(T, 2)[e, 1], 2 * g * s)):
            # (1 + g (1 - s)) cancels for g about -1.28: its error is of the terms' size
            mag = want.abs() + (u * s).abs() * 2 ** -16
            assert bool(((got.double() - want).abs() <= (U16 + 2.0 ** -14) * mag).all())


def test_norm_backward_of_2_to_30_rows():
    """Rows of four; a gradient arrives at the ends only, so the sums of dw have few terms."""
    torch, mt = need_gpu()
    T, h, fmt = 1 << 30, 4, 1
    codes = (_mod(torch, T * h, 13, torch.int8) + 65).view(torch.uint8)  # 65..77 at scale 1
    scales = torch.full((T,), 127, dtype=torch.uint8, device="cuda")
    rstd = torch.full((T,), 2.0 ** -6, device="cuda")
    w = torch.tensor([1.0, 2.0, 0.5, 1.0], device="cuda")
    dy = torch.zeros((T, h), device="cuda")
    for e in _ends(T):
        dy[e] = torch.randn((EDGE, h), device="cuda", generator=torch.Generator("cuda").manual_seed(e.start % 97))
    dx, dw = torch.full((T, h), float("nan"), device="cuda"), torch.empty(h, device="cuda")
    ws = torch.empty(mt.mt_op_rmsnorm_bwd_ckpt8_workspace(T, h), device="cuda")
    mt.mt_op_rmsnorm_bwd_ckpt8(codes, scales, fmt, w, rstd, dy, None, dx, None, dw, ws, T, h)
    assert mt.mt_op_device_error() == 0
    want_dw, mag_dw = torch.zeros(h, dtype=torch.float64, device="cuda"), 0
    for e in _ends(T):
        x, d = codes.view(torch.int8).view(T, h)[e].double(), dy[e].double()
        xh = x * 2.0 ** -6
        dot = (d * w.double() * xh).sum(1, keepdim=True) / h
        want = 2.0 ** -6 * (d * w.double() - xh * dot)
        mag = 2.0 ** -6 * ((d * w.double()).abs() + xh * (d * w.double() * xh).abs().sum(1, keepdim=True) / h)
        assert bool(((dx[e].double() - want).abs() <= 16 * U32 * mag).all())
        want_dw += (d * xh).sum(0)
        mag_dw = mag_dw + (d * xh).abs().sum(0)
    assert bool(((dw.double() - want_dw).abs() <= 3 * EDGE * U32 * mag_dw).all())
    for e in _ends(T):
        dx[e] = 0
    assert int(torch.count_nonzero(dx)) == 0


def test_logits_gradient_of_2_to_30_rows():
    """Two equal logits: p is 1/2, good to 2^-22 (lse is fp32)."""
    torch, mt = need_gpu()
    T, V = 1 << 30, 2
    z = torch.zeros((T, V), dtype=torch.bfloat16, device="cuda")
    ids = _mod(torch, T, 3, torch.int32) - 1  # not scored, first, second
    lse = torch.full((T,), math.log(2.0), device="cuda")
    g = torch.full((T,), 4.0, device="cuda")
    mt.mt_op_token_logprobs_bwd(z, mt.MT_BF16, ids, 1.0, lse, None, g, None, z, mt.MT_BF16, T, V, V, V)
    want = torch.tensor([[0.0, 0.0], [2.0, -2.0], [-2.0, 2.0]], device="cuda")  # rounds to bf16 exactly
    for e in _ends(T):
        assert torch.equal(z[e].float(), want[(ids[e] + 1).long()])
    assert int(torch.count_nonzero(z)) == 2 * int(torch.count_nonzero(ids >= 0))


def test_log_probabilities_of_2_to_28_rows():
    torch, mt = need_gpu()
    T, V, k = 1 << 28, 2, 2
    z = torch.zeros((T, V), dtype=torch.bfloat16, device="cuda")
    z[:, 1] = 1.0
    ids = _mod(torch, T, 3, torch.int32) - 1
    lse, logp, ent = (torch.full((T,), float("nan"), device="cuda") for _ in range(3))
    ti, tl = torch.full((T, k), 9, dtype=torch.int32, device="cuda"), torch.full((T, k), float("nan"), device="cuda")
    mt.mt_op_token_logprobs(z, mt.MT_BF16, ids, 1.0, k, lse, logp, ent, ti, tl, T, V, V)
    L = math.log(1 + math.e)
    p = 1 / (1 + math.exp(-1))
    H = -(p * math.log(p) + (1 - p) * math.log(1 - p))
    on = ids >= 0
    for got, want in ((lse, on * L), (logp, on * (ids.double() - L)), (ent, on * H)):
        assert bool(((got.double() - want.double()).abs() <= 2.0 ** -20).all())
    assert bool((ti[on] == torch.tensor([1, 0], device="cuda")).all()) and bool((ti[~on] == -1).all())
    want = on[:, None] * torch.tensor([1 - L, -L], device="cuda", dtype=torch.float64)
    assert bool(((tl.double() - want).abs() <= 2.0 ** -20).all())


def test_embedding_of_2_to_28_rows():
    """Counts below 2^24 are exact sums."""
    torch, mt = need_gpu()
    T, V, h = 1 << 28, 7, 1
    ids = _mod(torch, T, 9, torch.int32) - 1  # -1 is padding, 7 lies outside the table
    table = torch.arange(1, V + 1, device="cuda").float()
    out = torch.full((T,), float("nan"), device="cuda")
    mt.mt_op_embed_fwd(table, mt.MT_F32, ids, 2.0, out, mt.MT_F32, T, V, h)
    on = (ids >= 0) & (ids < V)
    assert torch.equal(out, on * 2.0 * (ids + 1))
    assert mt.mt_op_device_error() != 0
    out.zero_()
    out[::64] = 1.0
    out[T - 1] = 1.0
    ws = torch.empty(mt.mt_op_embed_bwd_workspace(T, V, h), dtype=torch.uint8, device="cuda")
    dE = torch.full((V,), float("nan"), device="cuda")
    mt.mt_op_embed_bwd(ids, out, mt.MT_F32, 1.0, dE, mt.MT_F32, 0, ws, T, V, h)
    one = on & (out > 0)
    assert torch.equal(dE.double(), torch.bincount(ids[one].long(), minlength=V).double())
    assert mt.mt_op_device_error() != 0


@pytest.mark.parametrize("fmt", [1, 2])
@pytest.mark.parametrize("n,ld", [((1 << 29), 1 << 29), ((1 << 29) - 5, (1 << 29) - 1)])
def test_checkpoint_of_the_widest_rows(fmt, n, ld):
    torch, mt = need_gpu()
    T = 2
    x = (_mod(torch, T * ld, 31, torch.float32) - 15).view(T, ld)
    codes = torch.full((T, ld), 77, dtype=torch.uint8, device="cuda")
    scales = torch.empty((T, -(-n // 32)), dtype=torch.uint8, device="cuda")
    mt.mt_op_ckpt8_pack(x, mt.MT_F32, fmt, codes, scales, T, n, ld, ld)
    back = torch.full((T, ld), 1e9, device="cuda")
    mt.mt_op_ckpt8_unpack(codes, scales, fmt, back, mt.MT_F32, T, n, ld, ld)
    assert torch.equal(back[:, :n], x[:, :n])
    assert bool((codes[:, n:] == 77).all()) and bool((back[:, n:] == 1e9).all())


@pytest.mark.parametrize("F,ld", [((1 << 29), 1 << 29), ((1 << 29) - 5, (1 << 29) - 1)])
def test_swiglu_of_the_widest_rows(F, ld):
    """Padding columns 0, and the values at the row's ends as above."""
    torch, mt = need_gpu()
    T, fmt = 1, 2
    gu = ((_mod(torch, 2 * ld, 31, torch.bfloat16) - 15) / 4).view(2, ld)
    act = torch.full((ld,), 7.0, dtype=torch.bfloat16, device="cuda")
    codes = torch.full((2, ld), 77, dtype=torch.uint8, device="cuda")
    scales = torch.empty(2 * -(-F // 32), dtype=torch.uint8, device="cuda")
    mt.mt_op_swiglu_fwd_ckpt8(gu, act, codes, scales, fmt, T, F, ld)
    dgu = torch.full((2, ld), 7.0, dtype=torch.bfloat16, device="cuda")
    dact = torch.full((ld,), 2.0, dtype=torch.bfloat16, device="cuda")
    mt.mt_op_swiglu_bwd_ckpt8(codes, scales, fmt, dact, dgu, T, F, ld)
    for e in _ends(F):
        g, u = gu[0, e].double(), gu[1, e].double()
        s = torch.sigmoid(g)
        for got, want in ((act[e], g * s * u), (dgu[0, e], 2 * u * s * (1 + g * (1 - s))), (dgu[1, e], 2 * g * s)):
            mag = want.abs() + (u * s).abs() * 2 ** -16
            assert bool(((got.double() - want).abs() <= (U16 + 2.0 ** -14) * mag).all())
    for pad in (act[F:], codes[:, F:], dgu[:, F:]):
        assert int(torch.count_nonzero(pad)) == 0
