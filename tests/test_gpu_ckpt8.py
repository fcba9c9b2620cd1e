"""8-bit activation checkpoints: the packed form against its definition
(exactly: the scale is a power of two, so the only rounding is the code's),
and the RMSNorm and SwiGLU passes that write and read it against float64.

Bounds (tests/bounds.py): U32 per fp32 rounding, U16 for the bf16 outputs,
acc(n) for fp32 sums; __expf(x) is within 2 + 1.2|x| units of 2^-23.
"""
import numpy as np
import pytest

from tests import ckpt8_ref as ref
from tests.bounds import U16, U32, acc, check, silu_parts
from tests.common import bf16_round
from tests.gpu_util import from_dev, need_gpu, to_dev_bf16, to_dev_f32

pytestmark = pytest.mark.gpu
FMTS = [ref.I8, ref.E4M3]
FLUSH = 2.0 ** -126


def _activation(T, n, seed):
    """Rows of different size, a few columns far above the others, exact zeros."""
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((T, n)) * np.exp(rng.standard_normal((T, 1)))
    x[:, rng.random(n) < 0.02] *= 100.0
    x[rng.random((T, n)) < 0.05] = 0.0
    return x.astype(np.float32)


def _pack(torch, mt, X, fmt, T, n, ldx, ldc, dtype):
    codes = torch.full((T, ldc), 0x55, dtype=torch.uint8, device="cuda")
    scales = torch.full((T, -(-n // 32)), 0x55, dtype=torch.uint8, device="cuda")
    mt.mt_op_ckpt8_pack(X, dtype, fmt, codes, scales, T, n, ldx, ldc)
    return codes, scales


SHAPES = [(1, 1, 1, 1), (3, 7, 7, 7), (5, 32, 32, 32), (2, 33, 33, 40), (9, 64, 72, 64), (4, 100, 101, 103),
          (130, 1000, 1000, 1000), (7, 4096, 4096, 4096), (300, 40, 48, 64), (1, 14336, 14336, 14336)]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("T,n,ldx,ldc", SHAPES)
def test_pack_and_unpack_follow_the_definition(fmt, bf16, T, n, ldx, ldc):
    torch, mt = need_gpu()
    full = _activation(T, ldx, 11 * T + n)
    X, x32 = to_dev_bf16(torch, full) if bf16 else (to_dev_f32(torch, full), full)
    dtype = mt.MT_BF16 if bf16 else mt.MT_F32
    x = x32[:, :n]
    codes, scales = _pack(torch, mt, X, fmt, T, n, ldx, ldc, dtype)
    c, s = codes.cpu().numpy(), scales.cpu().numpy()
    assert np.array_equal(s, ref.scales_of(x, fmt))
    want = ref.values_of(x, fmt)
    assert np.array_equal(ref.decode(c[:, :n].copy(), s, fmt), want)
    assert np.all(c[:, n:] == 0x55)  # columns past n are left as they were
    back = torch.full((T, ldx), -7.0, dtype=X.dtype, device="cuda")
    mt.mt_op_ckpt8_unpack(codes, scales, fmt, back, dtype, T, n, ldc, ldx)
    got = from_dev(back)
    assert np.array_equal(got[:, :n], bf16_round(want.astype(np.float32)) if bf16 else want.astype(np.float32))
    assert np.all(got[:, n:] == -7.0)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("T,n,ldx,ldc,x0,c0", [(5, 777, 777, 777, 1, 1), (40, 1003, 1004, 1010, 3, 5), (3, 224, 225, 231, 2, 7),
                                               (9, 4097, 4097, 4099, 5, 3), (200, 33, 35, 33, 7, 2)])
def test_pack_and_unpack_off_the_boundary(fmt, bf16, T, n, ldx, ldc, x0, c0):
    """Tensors that start at any element, rows at any byte: what lies around them stays."""
    torch, mt = need_gpu()
    full = _activation(1, x0 + T * ldx + 9, 13 * T + n).reshape(-1)
    X = torch.from_numpy(full).cuda().to(torch.bfloat16 if bf16 else torch.float32)
    dtype = mt.MT_BF16 if bf16 else mt.MT_F32
    x = from_dev(X)[x0:x0 + T * ldx].reshape(T, ldx)[:, :n]
    raw = torch.full((c0 + T * ldc + 9,), 0x55, dtype=torch.uint8, device="cuda")
    scales = torch.empty((T, -(-n // 32)), dtype=torch.uint8, device="cuda")
    mt.mt_op_ckpt8_pack(X[x0:], dtype, fmt, raw[c0:], scales, T, n, ldx, ldc)
    r = raw.cpu().numpy()
    codes, s = r[c0:c0 + T * ldc].reshape(T, ldc), scales.cpu().numpy()
    assert np.all(r[:c0] == 0x55) and np.all(codes[:, n:] == 0x55) and np.all(r[c0 + T * ldc:] == 0x55)
    want = ref.values_of(x, fmt)
    assert np.array_equal(s, ref.scales_of(x, fmt))
    assert np.array_equal(ref.decode(codes[:, :n].copy(), s, fmt), want)
    back = torch.full_like(X, -7.0)
    mt.mt_op_ckpt8_unpack(raw[c0:], scales, fmt, back[x0:], dtype, T, n, ldc, ldx)
    b = from_dev(back)
    got = b[x0:x0 + T * ldx].reshape(T, ldx)
    assert np.array_equal(got[:, :n], bf16_round(want.astype(np.float32)) if bf16 else want.astype(np.float32))
    assert np.all(b[:x0] == -7.0) and np.all(got[:, n:] == -7.0) and np.all(b[x0 + T * ldx:] == -7.0)


@pytest.mark.parametrize("fmt", FMTS)
def test_pack_borders(fmt):
    """Maxima on and around the limit, ties of both formats, subnormals,
    the largest fp32 values, zeros, infinities and NaN."""
    torch, mt = need_gpu()
    lim = ref.LIMIT[fmt]
    rows = []
    for e in (-130, -126, -120, -20, 0, 30, 118 if fmt == ref.E4M3 else 120):
        for a in (lim, np.nextafter(np.float32(lim), np.float32(0)), np.nextafter(np.float32(lim), np.float32(1e9)),
                  lim / 2, 1.0):
            with np.errstate(over="ignore"):
                r = np.full(64, 1.0, np.float64)
                r[:32] = a * 2.0 ** e * np.linspace(-1, 1, 32)
                r[32:] = (np.arange(32) + 0.5) * 2.0 ** e  # ties of the whole numbers
                rows.append(np.clip(r, -3.4028234e38, 3.4028234e38).astype(np.float32))
    for bad in (np.inf, -np.inf, np.nan):
        r = np.linspace(-1, 1, 64).astype(np.float32)
        r[40] = bad
        rows.append(r)
    rows.append(np.zeros(64, np.float32))
    rows.append(np.full(64, -0.0, np.float32))
    rows.append(np.full(64, 1e-45, np.float32))
    tie = (np.arange(64) / 16 + 1 / 32).astype(np.float32)  # midpoints of e4m3 steps
    tie[0] = 448.0
    rows.append(tie)
    x = np.stack(rows)
    T, n = x.shape
    codes, scales = _pack(torch, mt, to_dev_f32(torch, x), fmt, T, n, n, n, mt.MT_F32)
    s = scales.cpu().numpy()
    assert np.array_equal(s, ref.scales_of(x, fmt))
    want = ref.values_of(x, fmt)
    np.testing.assert_array_equal(ref.decode(codes.cpu().numpy(), s, fmt), want)
    assert np.all(codes.cpu().numpy()[s.repeat(32, 1) == 255] == 0)
    back = torch.empty((T, n), device="cuda")
    mt.mt_op_ckpt8_unpack(codes, scales, fmt, back, mt.MT_F32, T, n, n, n)
    np.testing.assert_array_equal(from_dev(back), want.astype(np.float32))


def test_every_code_unpacks():
    torch, mt = need_gpu()
    for fmt in FMTS:
        c = np.tile(np.arange(256, dtype=np.uint8), (255, 1))
        if fmt == ref.E4M3:
            c[(c & 0x7f) == 0x7f] = 0  # NaN codes are never written
        s = np.tile(np.arange(255, dtype=np.uint8)[:, None], (1, 8))
        back = torch.empty((255, 256), device="cuda")
        mt.mt_op_ckpt8_unpack(torch.from_numpy(c).cuda(), torch.from_numpy(s).cuda(), fmt, back, mt.MT_F32, 255, 256,
                              256, 256)
        with np.errstate(over="ignore"):
            np.testing.assert_array_equal(from_dev(back), ref.decode(c, s, fmt).astype(np.float32))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("T,h,with_res,with_bf", [(1, 4, False, True), (5, 36, True, False), (77, 320, True, True),
                                                  (16, 96, True, True), (17, 3200, True, True), (65, 1024, False, False),
                                                  (128, 2048, True, True), (128, 3204, True, False), (129, 96, True, True),
                                                  (1, 3200, True, True), (100, 3200, True, True),
                                                  (45, 1800, False, True), (700, 64, True, True),
                                                  (33, 4096, True, True), (9, 6000, True, False),
                                                  (500, 8192, True, True), (3, 2052, False, False), (400, 7452, True, True),
                                                  (1300, 1032, False, True)])
def test_rmsnorm_through_the_checkpoint(fmt, T, h, with_res, with_bf):
    torch, mt = need_gpu()
    eps = np.float32(1e-5)
    rng = np.random.default_rng(T * h)
    x = _activation(T, h, 3 + h)
    w = (1.0 + 0.1 * rng.standard_normal(h)).astype(np.float32)
    dy = rng.standard_normal((T, h)).astype(np.float32)
    res = rng.standard_normal((T, h)).astype(np.float32) if with_res else None
    X, W, DY = to_dev_f32(torch, x), to_dev_f32(torch, w), to_dev_f32(torch, dy)
    Y = torch.empty((T, h), dtype=torch.bfloat16, device="cuda")
    R = torch.empty(T, device="cuda")
    codes = torch.empty((T, h), dtype=torch.uint8, device="cuda")
    scales = torch.empty((T, -(-h // 32)), dtype=torch.uint8, device="cuda")
    mt.mt_op_rmsnorm_fwd_ckpt8(X, W, Y, R, codes, scales, fmt, T, h, float(eps))
    x64, w64, dy64 = x.astype(np.float64), w.astype(np.float64), dy.astype(np.float64)
    r = 1.0 / np.sqrt((x64 ** 2).mean(axis=1) + float(eps))
    e_r = acc(h) + 4 * U32  # relative error of the mean of squares halves in the root; rsqrt and eps
    check(from_dev(R), r, e_r * r, "rstd")
    y = x64 * r[:, None] * w64
    check(from_dev(Y), y, (U16 + (1 + U16) * (e_r + 3 * U32)) * np.abs(y), "y")
    s = scales.cpu().numpy()
    assert np.array_equal(s, ref.scales_of(x, fmt))
    xq = ref.decode(codes.cpu().numpy(), s, fmt)
    assert np.array_equal(xq, ref.values_of(x, fmt))

    r32 = from_dev(R).astype(np.float64)
    DX = to_dev_f32(torch, res) if with_res else torch.empty((T, h), device="cuda")  # in place over the residual
    DXB = torch.empty((T, h), dtype=torch.bfloat16, device="cuda") if with_bf else None
    DW = torch.empty(h, device="cuda")
    ws = torch.full((mt.mt_op_rmsnorm_bwd_ckpt8_workspace(T, h),), float("nan"), device="cuda")
    mt.mt_op_rmsnorm_bwd_ckpt8(codes, scales, fmt, W, R, DY, DX if with_res else None, DX, DXB, DW, ws, T, h)
    xh = xq * r32[:, None]
    g = dy64 * w64
    mean = (g * xh).mean(axis=1, keepdims=True)
    mean_abs = np.abs(g * xh).mean(axis=1, keepdims=True)
    rr = r32[:, None]
    dx = rr * (g - xh * mean) + (res if with_res else 0)
    bound = rr * (6 * U32 * (np.abs(g) + np.abs(xh * mean)) + np.abs(xh) * (acc(h) + 8 * U32) * mean_abs)
    check(from_dev(DX), dx, bound + 2 * U32 * (np.abs(dx) + (np.abs(res) if with_res else 0)) + 1e-37, "dx")
    if with_bf:
        assert np.array_equal(from_dev(DXB), bf16_round(from_dev(DX)))
    dw = (dy64 * xh).sum(axis=0)
    check(from_dev(DW), dw, (acc(T) + 4 * U32) * np.abs(dy64 * xh).sum(axis=0) + 1e-37, "dw")
    # deterministic
    DW2, DX2 = torch.empty_like(DW), torch.empty_like(DX)
    mt.mt_op_rmsnorm_bwd_ckpt8(codes, scales, fmt, W, R, DY, None, DX2, None, DW2, ws, T, h)
    assert torch.equal(DW, DW2)


def test_rmsnorm_gradient_against_differences():
    """dx and dw of sum(dy * xh w) at the checkpoint's values, by central differences of the float64 forward."""
    torch, mt = need_gpu()
    T, h, fmt = 3, 64, ref.I8
    rng = np.random.default_rng(5)
    xq = ref.values_of(rng.standard_normal((T, h)).astype(np.float32), fmt)
    w = 1 + 0.1 * rng.standard_normal(h)
    dy = rng.standard_normal((T, h)).astype(np.float32)
    X, W = to_dev_f32(torch, xq), to_dev_f32(torch, w)
    w = from_dev(W).astype(np.float64)
    codes = torch.empty((T, h), dtype=torch.uint8, device="cuda")
    scales = torch.empty((T, 2), dtype=torch.uint8, device="cuda")
    Y, R = torch.empty((T, h), dtype=torch.bfloat16, device="cuda"), torch.empty(T, device="cuda")
    mt.mt_op_rmsnorm_fwd_ckpt8(X, W, Y, R, codes, scales, fmt, T, h, 1e-5)
    DX, DW = torch.empty((T, h), device="cuda"), torch.empty(h, device="cuda")
    ws = torch.empty(mt.mt_op_rmsnorm_bwd_ckpt8_workspace(T, h), device="cuda")
    mt.mt_op_rmsnorm_bwd_ckpt8(codes, scales, fmt, W, R, to_dev_f32(torch, dy), None, DX, None, DW, ws, T, h)

    def f(x, w):
        return float((dy * x / np.sqrt((x ** 2).mean(axis=1, keepdims=True) + 1e-5) * w).sum())

    d = 1e-5  # central differences in float64: error about d^2 and 1e-16 / d, both far below 1e-5
    for t, c in ((0, 0), (1, 17), (2, 63)):
        e = np.zeros((T, h))
        e[t, c] = d
        assert abs(float(DX[t, c]) - (f(xq + e, w) - f(xq - e, w)) / (2 * d)) < 2e-5
        ew = np.zeros(h)
        ew[c] = d
        assert abs(float(DW[c]) - (f(xq, w + ew) - f(xq, w - ew)) / (2 * d)) < 2e-5


def _act_bounds(g, u, d=None):
    """Relative error of the sigmoid (its exponential and two more roundings)
    and from it the bounds of act, or of (dg, du). A sigmoid below 2^-126 may
    be 0 (and the exponential infinite a little further out), which moves act
    and du by at most 2^-126 |g u| and |dact g|, and dg by 2^-126 |dact u|
    (1 + |g|); bf16 results below 2^-126 may be 0 too."""
    with np.errstate(over="ignore"):
        s, silu, mag = silu_parts(g)
    e = (8 + 1.2 * np.abs(g)) * 2.0 ** -23
    if d is None:
        a = silu * u
        return a, (U16 + 2 * e) * np.abs(a) + FLUSH * (1 + np.abs(g * u))
    dg = d * u * s * (1 + g * (1 - s))
    du = d * silu
    return (dg, U16 * np.abs(dg) + 3 * e * np.abs(d * u) * mag + FLUSH * (1 + np.abs(d * u) * (1 + np.abs(g))),
            du, (U16 + 2 * e) * np.abs(du) + FLUSH * (1 + np.abs(d * g)))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("T,F,ld", [(1, 1, 1), (3, 5, 8), (17, 172, 176), (5, 33, 33), (64, 256, 256), (130, 2816, 2816),
                                    (2, 40, 104), (33, 64, 200), (9, 14336, 14336)])
def test_swiglu_through_the_checkpoint(fmt, T, F, ld):
    torch, mt = need_gpu()
    rng = np.random.default_rng(7 * T + F)
    gu = np.full((T, 2 * ld), 9.0, np.float32)
    gu[:, :F] = _activation(T, F, F)
    gu[:, ld:ld + F] = _activation(T, F, F + 1)
    dact = np.full((T, ld), np.nan, np.float32)  # padding is not read
    dact[:, :F] = rng.standard_normal((T, F))
    GU, gu32 = to_dev_bf16(torch, gu)
    DA = torch.from_numpy(dact).cuda().to(torch.bfloat16)
    d = from_dev(DA)[:, :F].astype(np.float64)
    act = torch.full((T, ld), 3.0, dtype=torch.bfloat16, device="cuda")
    codes = torch.full((T, 2 * ld), 0x55, dtype=torch.uint8, device="cuda")
    nb = -(-F // 32)
    scales = torch.full((T, 2 * nb), 0x55, dtype=torch.uint8, device="cuda")
    mt.mt_op_swiglu_fwd_ckpt8(GU, act, codes, scales, fmt, T, F, ld)
    g, u = gu32[:, :F].astype(np.float64), gu32[:, ld:ld + F].astype(np.float64)
    want, bound = _act_bounds(g, u)
    check(from_dev(act)[:, :F], want, bound, "act")
    assert np.all(from_dev(act)[:, F:] == 0)
    c, s = codes.cpu().numpy(), scales.cpu().numpy()
    for part, off in ((g, 0), (u, ld)):
        k = off // ld * nb
        assert np.array_equal(s[:, k:k + nb], ref.scales_of(part, fmt))
        assert np.array_equal(ref.decode(c[:, off:off + F].copy(), s[:, k:k + nb], fmt), ref.values_of(part, fmt))
        assert np.all(c[:, off + F:off + ld] == 0)
    dgu = torch.full((T, 2 * ld), 3.0, dtype=torch.bfloat16, device="cuda")
    mt.mt_op_swiglu_bwd_ckpt8(codes, scales, fmt, DA, dgu, T, F, ld)
    dg, bg, du, bu = _act_bounds(ref.values_of(g, fmt), ref.values_of(u, fmt), d)
    got = from_dev(dgu)
    check(got[:, :F], dg, bg, "dg")
    check(got[:, ld:ld + F], du, bu, "du")
    assert np.all(got[:, F:ld] == 0) and np.all(got[:, ld + F:] == 0)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("T,F,off", [(7, 1001, 1), (65, 250, 3), (3, 4099, 6), (100, 31, 5)])
def test_swiglu_off_the_boundary(fmt, T, F, off):
    """Tensors that start at any element: the same values as from aligned ones, nothing written beside them."""
    torch, mt = need_gpu()
    gu = torch.randn((T, 2 * F), device="cuda").to(torch.bfloat16)
    da = torch.randn((T, F), device="cuda").to(torch.bfloat16)
    nb = -(-F // 32)

    def run(o):
        def place(t):
            raw = torch.full((o + t.numel() + 9,), 3, dtype=t.dtype, device="cuda")
            raw[o:o + t.numel()] = t.reshape(-1)
            return raw
        g, d = place(gu), place(da)
        act, codes, dgu = place(torch.zeros_like(da)), place(torch.zeros((T, 2 * F), dtype=torch.uint8, device="cuda")), \
            place(torch.zeros_like(gu))
        scales = torch.empty((T, 2 * nb), dtype=torch.uint8, device="cuda")
        mt.mt_op_swiglu_fwd_ckpt8(g[o:], act[o:], codes[o:], scales, fmt, T, F, F)
        mt.mt_op_swiglu_bwd_ckpt8(codes[o:], scales, fmt, d[o:], dgu[o:], T, F, F)
        out = []
        for t in (act, codes, dgu):
            assert bool((t[:o] == 3).all()) and bool((t[-9:] == 3).all())
            out.append(t[o:-9].clone())
        return out + [scales]

    for a, b in zip(run(0), run(off)):
        assert torch.equal(a, b)


def test_swiglu_non_finite_block_is_nan_in_the_gradient():
    torch, mt = need_gpu()
    T, F = 2, 64
    gu = np.ones((T, 2 * F), np.float32)
    gu[0, 3] = np.inf
    gu[1, F + 40] = np.nan
    GU = torch.from_numpy(gu).cuda().to(torch.bfloat16)
    codes = torch.empty((T, 2 * F), dtype=torch.uint8, device="cuda")
    scales = torch.empty((T, 4), dtype=torch.uint8, device="cuda")
    act, dgu = torch.empty((T, F), dtype=torch.bfloat16, device="cuda"), torch.empty_like(GU)
    mt.mt_op_swiglu_fwd_ckpt8(GU, act, codes, scales, ref.E4M3, T, F, F)
    mt.mt_op_swiglu_bwd_ckpt8(codes, scales, ref.E4M3, torch.ones_like(act), dgu, T, F, F)
    nan = np.isnan(from_dev(dgu))
    assert nan[0, :32].all() and nan[0, F:F + 32].all() and not nan[0, 32:F].any()
    assert nan[1, 32:F].all() and not nan[1, :32].any()  # dg needs u; du of that block does not
    assert not nan[1, F:].any()


@pytest.fixture
def emptied():
    """Gives the large buffers back to the device."""
    yield
    import torch
    torch.cuda.empty_cache()


@pytest.mark.parametrize("ld", [1 << 29, (1 << 29) - 3])
def test_row_offsets_past_32_bits(emptied, ld):
    """Rows 2^29 elements apart (element offsets to 2^31, byte offsets to
    2^32): the same bits as the rows close together."""
    torch, mt = need_gpu()
    T, n, bf = 5, 1000, torch.bfloat16
    x = torch.randn((T, n), device="cuda").to(bf)
    small = torch.empty((T, n), dtype=torch.uint8, device="cuda"), torch.empty((T, 32), dtype=torch.uint8, device="cuda")
    mt.mt_op_ckpt8_pack(x, mt.MT_BF16, 1, *small, T, n, n, n)
    far = torch.empty(((T - 1) * ld + n,), dtype=bf, device="cuda").as_strided((T, n), (ld, 1))
    far.copy_(x)
    codes = torch.empty(((T - 1) * ld + n,), dtype=torch.uint8, device="cuda").as_strided((T, n), (ld, 1))
    scales = torch.empty((T, 32), dtype=torch.uint8, device="cuda")
    mt.mt_op_ckpt8_pack(far, mt.MT_BF16, 1, codes, scales, T, n, ld, ld)
    assert torch.equal(codes, small[0]) and torch.equal(scales, small[1])
    want, back = torch.empty_like(x), far.zero_()
    mt.mt_op_ckpt8_unpack(*small, 1, want, mt.MT_BF16, T, n, n, n)
    mt.mt_op_ckpt8_unpack(codes, scales, 1, back, mt.MT_BF16, T, n, ld, ld)
    assert torch.equal(back, want)


def test_swiglu_row_offsets_past_32_bits(emptied):
    torch, mt = need_gpu()
    T, F, ld, bf = 3, 300, 1 << 29, torch.bfloat16
    g, u, d = (torch.randn((T, F), device="cuda").to(bf) for _ in range(3))

    def run(ld):
        e = lambda n, dt: torch.empty((T, n), dtype=dt, device="cuda")  # noqa: E731
        gu, dact = e(2 * ld, bf), e(ld, bf)
        gu[:, :F], gu[:, ld:ld + F], dact[:, :F] = g, u, d
        act, codes, scales = e(ld, bf), e(2 * ld, torch.uint8), e(20, torch.uint8)
        mt.mt_op_swiglu_fwd_ckpt8(gu, act, codes, scales, 2, T, F, ld)
        mt.mt_op_swiglu_bwd_ckpt8(codes, scales, 2, dact, gu, T, F, ld)  # over g|u, which it does not read
        return (act[:, :F].clone(), codes[:, :F].clone(), codes[:, ld:ld + F].clone(), scales, gu[:, :F].clone(),
                gu[:, ld:ld + F].clone(), act[:, F:F + 4].clone(), act[:, ld - 4:].clone(), gu[:, -4:].clone())

    for a, b in zip(run(F + 4), run(ld)):  # the last three are padding
        assert torch.equal(a, b)


def test_norm_of_more_than_2_to_32_values(emptied):
    """The last rows of 4.3e9 values: the bits of the same rows alone."""
    torch, mt = need_gpu()
    T, h, last = (1 << 19) + 11, 8192, 40
    x, dy = torch.empty((T, h), device="cuda"), torch.empty((T, h), device="cuda")
    x[-last:], dy[-last:] = torch.randn((last, h), device="cuda"), torch.randn((last, h), device="cuda")
    x[:-last], dy[:-last] = 1.0, 0.0
    w = torch.randn(h, device="cuda")

    def run(x, dy):
        T = x.shape[0]
        e = lambda *s, dt=torch.float32: torch.empty(s, dtype=dt, device="cuda")  # noqa: E731
        y, r = e(T, h, dt=torch.bfloat16), e(T)
        codes, scales = e(T, h, dt=torch.uint8), e(T, h // 32, dt=torch.uint8)
        mt.mt_op_rmsnorm_fwd_ckpt8(x, w, y, r, codes, scales, 1, T, h, 1e-5)
        dx, dxb, dw = e(T, h), e(T, h, dt=torch.bfloat16), e(h)
        ws = e(mt.mt_op_rmsnorm_bwd_ckpt8_workspace(T, h))
        mt.mt_op_rmsnorm_bwd_ckpt8(codes, scales, 1, w, r, dy, None, dx, dxb, dw, ws, T, h)
        return [t[-last:].clone() for t in (y, r, codes, scales, dx, dxb)] + [dw]

    far, near = run(x, dy), run(x[-last:].clone(), dy[-last:].clone())
    for a, b in zip(far[:-1], near[:-1]):
        assert torch.equal(a, b)
    # dw: the other rows add nothing; up to 40 terms in another order
    bound = acc(last) * (dy[-last:].abs() * x[-last:].abs() * near[1][:, None]).sum(0)
    assert bool(((far[-1] - near[-1]).abs() <= 2 * bound + 1e-30).all())
