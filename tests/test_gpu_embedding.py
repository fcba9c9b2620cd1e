"""Embedding lookup with a scale and the table's gradient by sorted tokens
against float64: the lookup exactly (one fp32 product, then the type's
rounding), the sums within acc(n) of the magnitudes they add."""
import numpy as np
import pytest

from tests.bounds import U16, U32, acc, check
from tests.common import bf16_round
from tests.gpu_util import from_dev, need_gpu, to_dev_f32

pytestmark = pytest.mark.gpu


def _typed(torch, mt, bf16):
    return (torch.bfloat16, mt.MT_BF16) if bf16 else (torch.float32, mt.MT_F32)


@pytest.mark.parametrize("tb", [False, True])
@pytest.mark.parametrize("ob", [False, True])
@pytest.mark.parametrize("T,V,h", [(1, 1, 1), (5, 3, 7), (33, 256, 64), (130, 1000, 1028), (1000, 32000, 1024), (7, 50, 4096)])
def test_lookup(tb, ob, T, V, h):
    torch, mt = need_gpu()
    (tt, tc), (ot, oc) = _typed(torch, mt, tb), _typed(torch, mt, ob)
    rng = np.random.default_rng(T + h)
    table = torch.randn((V, h), device="cuda").to(tt)
    ids = rng.integers(-1, V, T).astype(np.int32)
    scale = np.float32(np.sqrt(h))
    out = torch.full((T, h), 7.0, device="cuda").to(ot)
    mt.mt_op_embed_fwd(table, tc, torch.from_numpy(ids).cuda(), float(scale), out, oc, T, V, h)
    want = from_dev(table)[np.maximum(ids, 0)] * scale
    want[ids < 0] = 0
    assert np.array_equal(from_dev(out), bf16_round(want) if ob else want)
    assert mt.mt_op_device_error() == 0


def _grad(torch, mt, ids, dout, db, eb, scale, V, start=None):
    T, h = dout.shape
    (_, dc), (et, ec) = _typed(torch, mt, db), _typed(torch, mt, eb)
    ws = torch.full((mt.mt_op_embed_bwd_workspace(T, V, h),), 0xee, dtype=torch.uint8, device="cuda")
    dE = torch.full((V, h), float("nan"), device="cuda").to(et) if start is None else start.clone()
    mt.mt_op_embed_bwd(ids, dout, dc, scale, dE, ec, start is not None, ws, T, V, h)
    return dE


def _reference(ids, dout, V):
    h = dout.shape[1]
    s, m, n = np.zeros((V, h)), np.zeros((V, h)), np.zeros(V)
    ok = (ids >= 0) & (ids < V)
    np.add.at(s, ids[ok], dout[ok].astype(np.float64))
    np.add.at(m, ids[ok], np.abs(dout[ok].astype(np.float64)))
    np.add.at(n, ids[ok], 1)
    return s, m, n


def _check_grad(got, s, m, n, scale, eb, start=None):
    want = s * scale + (0 if start is None else start)
    e = np.array([acc(int(k)) for k in n])[:, None]
    mag = m * abs(scale) + (0 if start is None else np.abs(start))
    check(got, want, (e + 4 * U32) * mag + (U16 if eb else U32) * np.abs(want) + 1e-37, "dtable")


PATTERNS = ["uniform", "skewed", "one", "padding", "pairs"]


def _ids(pattern, T, V, rng):
    if pattern == "uniform":
        return rng.integers(0, V, T)
    if pattern == "skewed":
        return np.minimum(np.exp(rng.random(T) * np.log(V)).astype(np.int64) - 1, V - 1)
    if pattern == "one":
        return np.full(T, V - 1)
    if pattern == "padding":
        return np.where(rng.random(T) < 0.7, -1, rng.integers(0, V, T))
    return (np.arange(T) // 2) % V


@pytest.mark.parametrize("pattern", PATTERNS)
@pytest.mark.parametrize("db,eb", [(False, False), (True, True), (False, True), (True, False)])
@pytest.mark.parametrize("T,V,h", [(1, 1, 4), (2, 5, 3), (64, 256, 64), (65, 2, 8), (300, 1023, 36), (1000, 1024, 8),
                                   (5000, 3, 12), (4097, 32000, 64), (70000, 700, 4)])
def test_gradient(pattern, db, eb, T, V, h):
    torch, mt = need_gpu()
    rng = np.random.default_rng(T + V)
    ids = _ids(pattern, T, V, rng).astype(np.int32)
    dout = torch.randn((T, h), device="cuda").to(torch.bfloat16 if db else torch.float32)
    IDS = torch.from_numpy(ids).cuda()
    scale = float(np.float32(np.sqrt(h)))
    s, m, n = _reference(ids, from_dev(dout), V)
    got = _grad(torch, mt, IDS, dout, db, eb, scale, V)
    _check_grad(from_dev(got), s, m, n, scale, eb)
    assert np.all(from_dev(got)[n == 0] == 0)
    # bitwise the same again, and added to what is there
    assert torch.equal(got, _grad(torch, mt, IDS, dout, db, eb, scale, V))
    start = torch.randn((V, h), device="cuda").to(got.dtype)
    more = _grad(torch, mt, IDS, dout, db, eb, scale, V, start)
    _check_grad(from_dev(more), s, m, n, scale, eb, from_dev(start).astype(np.float64))
    assert np.array_equal(from_dev(more)[n == 0], from_dev(start)[n == 0])
    assert mt.mt_op_device_error() == 0


@pytest.mark.parametrize("db,eb,T,V,h", [(False, False, 33000, 50, 515), (True, True, 33000, 20, 516),
                                         (True, False, 40000, 30000, 516), (False, True, 9000, 700, 2052)])
def test_many_wide_rows(db, eb, T, V, h):
    """Column groups several to a lane, whole and ragged, both types."""
    torch, mt = need_gpu()
    rng = np.random.default_rng(T + h)
    ids = _ids("skewed", T, V, rng).astype(np.int32)
    dout = torch.randn((T, h), device="cuda").to(torch.bfloat16 if db else torch.float32)
    s, m, n = _reference(ids, from_dev(dout), V)
    got = _grad(torch, mt, torch.from_numpy(ids).cuda(), dout, db, eb, 1.0, V)
    _check_grad(from_dev(got), s, m, n, 1.0, eb)


@pytest.mark.parametrize("T,V,h", [(3, 7, 1), (257, 60, 5), (5000, 900, 33), (33000, 4000, 517)])
@pytest.mark.parametrize("db,eb", [(True, False), (True, True), (False, False)])
@pytest.mark.parametrize("off", [0, 1])
def test_rows_of_odd_widths(off, db, eb, T, V, h):
    """Rows that start anywhere, the first one an element past a boundary
    too, NaN around the rows: only they are read."""
    torch, mt = need_gpu()
    rng = np.random.default_rng(T + off)
    ids = _ids("skewed", T, V, rng).astype(np.int32)
    flat = torch.full((T * h + off + 64,), float("nan"), device="cuda").to(torch.bfloat16 if db else torch.float32)
    dout = flat[off:off + T * h].view(T, h)
    dout.copy_(torch.randn((T, h), device="cuda"))
    s, m, n = _reference(ids, from_dev(dout), V)
    got = _grad(torch, mt, torch.from_numpy(ids).cuda(), dout, db, eb, 0.5, V)
    _check_grad(from_dev(got), s, m, n, 0.5, eb)
    assert np.all(from_dev(got)[n == 0] == 0)


@pytest.mark.parametrize("V", [1 << 10, (1 << 10) - 1, 1 << 17, 151936, (1 << 20) + 3])
def test_sort_over_the_vocabulary(V):
    """Vocabularies around the digits' borders, the largest ids in use: one
    fp32 value per position, whole numbers, so every sum is exact."""
    torch, mt = need_gpu()
    T, h = 20000, 1
    rng = np.random.default_rng(V)
    ids = np.concatenate([rng.integers(0, V, T - 3), [0, V - 1, V - 1]]).astype(np.int32)
    dout = torch.from_numpy(rng.integers(-50, 50, (T, h)).astype(np.float32)).cuda()
    got = _grad(torch, mt, torch.from_numpy(ids).cuda(), dout, False, False, 1.0, V)
    assert np.array_equal(from_dev(got), _reference(ids, from_dev(dout), V)[0].astype(np.float32))


def test_sum_order_is_by_position():
    """fp32 sums of up to 32 rows are those of adding them in ascending
    position, wherever the rows lie among others."""
    torch, mt = need_gpu()
    T, V, h = 40, 4, 4
    dout = (torch.randn((T, h), device="cuda") * torch.exp(4 * torch.randn((T, 1), device="cuda")))
    x = from_dev(dout)
    for first, n in ((0, 32), (5, 32), (3, 2), (30, 10)):
        ids = np.full(T, 3, np.int32)
        ids[:first] = 0
        ids[first:first + n] = 2
        got = from_dev(_grad(torch, mt, torch.from_numpy(ids).cuda(), dout, False, False, 1.0, V))
        want = np.zeros(h, np.float32)
        for row in x[first:first + n]:
            want = want + row
        assert np.array_equal(got[2], want)


def test_ids_past_the_vocabulary_are_reported():
    torch, mt = need_gpu()
    V, h = 10, 8
    ids = torch.tensor([1, 10, 2 ** 31 - 1, -2 ** 31, 1], dtype=torch.int32, device="cuda")
    dout = torch.ones((5, h), device="cuda")
    out = torch.full((5, h), 7.0, device="cuda")
    assert mt.mt_op_device_error() == 0
    mt.mt_op_embed_fwd(torch.ones((V, h), device="cuda"), mt.MT_F32, ids, 1.0, out, mt.MT_F32, 5, V, h)
    assert mt.mt_op_device_error() != 0
    assert np.array_equal(from_dev(out)[:, 0], [1, 0, 0, 0, 1])
    got = from_dev(_grad(torch, mt, ids, dout, False, False, 1.0, V))
    assert mt.mt_op_device_error() != 0
    assert mt.mt_op_device_error() == 0
    want = np.zeros((V, h))
    want[1] = 2
    assert np.array_equal(got, want)


def test_gradient_against_differences():
    """The loss sum(dout * out) is linear in the table: its difference quotient is the gradient."""
    torch, mt = need_gpu()
    T, V, h, scale = 9, 4, 8, 2.0
    ids = torch.tensor([0, 1, 1, 3, -1, 0, 0, 3, 1], dtype=torch.int32, device="cuda")
    dout = torch.randint(-8, 8, (T, h), device="cuda").float()
    g = _grad(torch, mt, ids, dout, False, False, scale, V)
    for v, c in ((0, 0), (1, 5), (2, 2), (3, 7)):
        t0, t1 = torch.zeros((V, h), device="cuda"), torch.zeros((V, h), device="cuda")
        t1[v, c] = 1.0
        outs = []
        for t in (t0, t1):
            out = torch.empty((T, h), device="cuda")
            mt.mt_op_embed_fwd(t, mt.MT_F32, ids, scale, out, mt.MT_F32, T, V, h)
            outs.append((out * dout).sum().item())
        assert float(g[v, c]) == outs[1] - outs[0]


def test_full_size_gradient():
    """The 8B step's table and batch (the gradient's offsets pass 32 bits): a
    skewed batch, used rows against float64 and the rest exactly zero."""
    torch, mt = need_gpu()
    T, V, h = 8192, 128256, 4096
    rng = np.random.default_rng(1)
    ids = _ids("skewed", T, V, rng).astype(np.int32)
    ids[:5] = V - 1
    IDS = torch.from_numpy(ids).cuda()
    dout = torch.randn((T, h), device="cuda")
    g = _grad(torch, mt, IDS, dout, False, False, 1.0, V)
    used = np.unique(ids)
    zero = torch.ones(V, dtype=torch.bool, device="cuda")
    zero[torch.from_numpy(used.astype(np.int64)).cuda()] = False
    assert int(torch.count_nonzero(g[zero])) == 0 and not bool(torch.isnan(g).any())
    for v in (0, 1, 2, int(used[len(used) // 2]), V - 1):
        rows = from_dev(dout[IDS == v]).astype(np.float64)
        check(from_dev(g[v]), rows.sum(axis=0), (acc(len(rows)) + 2 * U32) * np.abs(rows).sum(axis=0), f"row {v}")


@pytest.fixture
def emptied():
    """Gives the large buffers back to the device."""
    yield
    import torch
    torch.cuda.empty_cache()


def test_more_than_2_to_32_values_of_rows(emptied):
    """1.1 million rows of 4096: lookup, and whole-number gradients whose sums are exact."""
    torch, mt = need_gpu()
    T, V, h = 1_100_003, 53, 4096
    ids = torch.randint(0, V, (T,), device="cuda").int()
    table = torch.randn((V, h), device="cuda").to(torch.bfloat16)
    out = torch.empty((T, h), dtype=torch.bfloat16, device="cuda")
    mt.mt_op_embed_fwd(table, mt.MT_BF16, ids, 1.0, out, mt.MT_BF16, T, V, h)
    for lo in (0, T // 2, T - 1000):
        assert torch.equal(out[lo:lo + 1000], table[ids[lo:lo + 1000].long()])
    t = (torch.arange(T, device="cuda") % 7).to(torch.bfloat16)
    c = (torch.arange(h, device="cuda") % 3).to(torch.bfloat16)
    out.copy_(t[:, None]).add_(c[None])
    ws = torch.empty(mt.mt_op_embed_bwd_workspace(T, V, h), dtype=torch.uint8, device="cuda")
    dE = torch.empty((V, h), device="cuda")
    mt.mt_op_embed_bwd(ids, out, mt.MT_BF16, 1.0, dE, mt.MT_F32, 0, ws, T, V, h)
    n = torch.bincount(ids.long(), minlength=V).double()
    s = torch.bincount(ids.long(), weights=t.double(), minlength=V)
    assert torch.equal(dE.double(), s[:, None] + n[:, None] * c.double()[None])


@pytest.mark.parametrize("V,h,eb", [(60_000_000, 1, True), (9_000_000, 4, False), (3_000_017, 12, True),
                                    (1_073_741_823, 1, True)])
def test_large_tables_of_narrow_rows(emptied, V, h, eb):
    """Cleared beside the sort and after it, up to the largest vocabulary: only
    the rows of the given ids are other than 0."""
    torch, mt = need_gpu()
    T = 3000
    rng = np.random.default_rng(V)
    ids = np.concatenate([rng.integers(0, V, T - 4), [0, V - 1, V - 1, V // 2]]).astype(np.int32)
    dout = torch.from_numpy(rng.integers(1, 9, (T, h)).astype(np.float32)).cuda()
    got = _grad(torch, mt, torch.from_numpy(ids).cuda(), dout, False, eb, 1.0, V)
    at, back = np.unique(ids, return_inverse=True)
    want = np.zeros((len(at), h))
    np.add.at(want, back, from_dev(dout))
    rows = torch.from_numpy(at).cuda().long()
    assert np.array_equal(from_dev(got[rows]), want)  # small whole numbers: exact in bf16 too
    got[rows] = 0
    assert int(torch.count_nonzero(got)) == 0
