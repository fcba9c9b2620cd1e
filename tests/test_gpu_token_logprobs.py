"""Log probabilities of given tokens, entropy, top alternatives and the
logits' gradient against float64.

Bounds: with d = c (z - max) formed in two roundings and 2^(d log2 e) good to
2^-22, a term e^d of the sum S is off by (2^-22 + 4 U32 |d|) of itself, so
S is by E_S = 2^-21 + acc(V) + 4 U32 sum p|d|, and
 lse, logp : E_S + 2 U32 (|ln S| + |d_t| + |c max|)
 entropy   : E_S (1 + B) + (2^-21 + acc(V)) B + 8 U32 (B2 + B), B = sum p |d|, B2 = sum p d^2
 gradient  : p off by (2^-21 + 6 U32 |log p|) of itself, and the roundings of the result.
"""
import numpy as np
import pytest

from tests.bounds import U16, U32, acc, check
from tests.gpu_util import from_dev, need_gpu, to_dev_bf16, to_dev_f32

pytestmark = pytest.mark.gpu
BIG = 2.0 ** 100  # at or below -BIG: masked out; at or above BIG: no distribution


def _reference(z, ids, c, k):
    """float64, with the header's conventions for rows and logits left out."""
    T, V = z.shape
    z = z.astype(np.float64)
    out = {n: np.zeros(T) for n in ("lse", "logp", "ent", "b_lse", "b_logp", "b_ent")}
    out["top_ids"] = np.full((T, k), -1)
    out["top_logp"], out["b_top"] = np.zeros((T, k)), np.zeros((T, k))
    for t in range(T):
        if ids[t] < 0:
            continue
        live = z[t] > -BIG
        if not (z[t] < BIG).all():
            for n in ("lse", "logp", "ent"):
                out[n][t] = np.nan
            out["top_logp"][t] = np.nan
            continue
        out["top_logp"][t] = -np.inf
        if not live.any():
            out["lse"][t] = out["logp"][t] = -np.inf
            continue
        m = z[t][live].max()
        d = np.where(live, c * (z[t] - m), -np.inf)
        e = np.exp(d)
        S = e.sum()
        p = e / S
        dd = np.where(p > 0, d, 0.0)
        B, B2 = (p * np.abs(dd)).sum(), (p * dd ** 2).sum()
        es = 2.0 ** -21 + acc(V) + 4 * U32 * B
        lp = d - np.log(S)
        out["lse"][t] = c * m + np.log(S)
        out["logp"][t] = lp[ids[t]]
        out["ent"][t] = np.log(S) - (p * dd).sum()
        out["b_lse"][t] = es + 2 * U32 * (abs(np.log(S)) + abs(c * m))
        tail = lambda x: es + 2 * U32 * (abs(np.log(S)) + np.where(np.isfinite(x), np.abs(x), 0))  # noqa: E731
        out["b_logp"][t] = tail(d[ids[t]])
        out["b_ent"][t] = es * (1 + B) + (2.0 ** -21 + acc(V)) * B + 8 * U32 * (B2 + B) + 2 * U32 * np.log(S)
        order = np.lexsort((np.arange(V), -z[t]))[:k]
        order = order[live[order]]
        out["top_ids"][t, :len(order)] = order
        out["top_logp"][t, :len(order)] = lp[order]
        out["b_top"][t, :len(order)] = tail(d[order])
    return out


def _run(torch, mt, Z, dtype, ids, c, k, T, V, ld, entropy=True):
    f = lambda *s: torch.full(s, 7.0, device="cuda")  # noqa: E731
    o = {"lse": f(T), "logp": f(T), "ent": f(T) if entropy else None, "top_logp": f(T, k) if k else None,
         "top_ids": torch.full((T, k), 7, dtype=torch.int32, device="cuda") if k else None}
    mt.mt_op_token_logprobs(Z, dtype, ids, c, k, o["lse"], o["logp"], o["ent"], o["top_ids"], o["top_logp"], T, V, ld)
    return o


def _close(got, want, bound, what):
    got, want = np.asarray(got, np.float64), np.asarray(want, np.float64)
    fine = np.isfinite(want)
    np.testing.assert_array_equal(got[~fine], want[~fine], what)
    check(got[fine], want[fine], np.broadcast_to(bound, want.shape)[fine], what)


def _compare(o, w, k):
    _close(from_dev(o["lse"]), w["lse"], w["b_lse"], "lse")
    _close(from_dev(o["logp"]), w["logp"], w["b_logp"], "logp")
    if o["ent"] is not None:
        _close(from_dev(o["ent"]), w["ent"], w["b_ent"], "entropy")
    if k:
        np.testing.assert_array_equal(o["top_ids"].cpu().numpy(), w["top_ids"])
        _close(from_dev(o["top_logp"]), w["top_logp"], w["b_top"], "top_logp")


CASES = [(1, 1, 1, 0), (1, 1, 5, 1), (3, 2, 2, 2), (5, 31, 31, 8), (4, 33, 40, 32), (2, 255, 257, 20),
         (33, 1000, 1000, 5), (7, 4099, 4099, 8), (3, 9000, 9001, 32), (1, 32000, 32000, 20), (2, 128256, 128256, 8),
         (400, 515, 515, 3), (1, 151936, 151936, 1), (20, 40001, 40001, 20)]


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("T,V,ld,k", CASES)
def test_forward(bf16, T, V, ld, k):
    torch, mt = need_gpu()
    rng = np.random.default_rng(V + k)
    z = (3.0 * rng.standard_normal((T, ld))).astype(np.float32)
    z[:, V:] = 1e9  # past the row: not read
    if V > 64:
        z[rng.random((T, ld)) < 0.1] = -np.inf
        z[:, V:] = 1e9
    ids = rng.integers(0, V, T).astype(np.int32)
    if T > 2:
        ids[T // 2] = -1
    Z, z32 = (torch.from_numpy(z).cuda().to(torch.bfloat16), None) if bf16 else (to_dev_f32(torch, z), z)
    z32 = from_dev(Z)[:, :V]
    IDS = torch.from_numpy(ids).cuda()
    for c in (1.0, 0.37, 2.5):
        o = _run(torch, mt, Z, mt.MT_BF16 if bf16 else mt.MT_F32, IDS, c, k, T, V, ld, entropy=c != 0.37)
        _compare(o, _reference(z32, ids, float(np.float32(c)), k), k)
    assert mt.mt_op_device_error() == 0


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("off", [1, 3, 5])
def test_unaligned_rows(bf16, off):
    """Rows that start off a 16-byte boundary, the best logits in their unaligned ends."""
    torch, mt = need_gpu()
    T, V, k = 6, 9001, 8
    rng = np.random.default_rng(off)
    flat = rng.standard_normal(T * (V + 2) + off).astype(np.float32)
    buf = torch.from_numpy(flat).cuda()
    if bf16:
        buf = buf.to(torch.bfloat16)
    Z = buf[off:].as_strided((T, V + 2), (V + 2, 1))
    Z[:, 0], Z[:, 1], Z[:, V - 1] = 9.0, 8.0, 9.0  # ties across the ends: the lower index first
    ids = rng.integers(0, V, T).astype(np.int32)
    o = _run(torch, mt, Z, mt.MT_BF16 if bf16 else mt.MT_F32, torch.from_numpy(ids).cuda(), 1.0, k, T, V, V + 2)
    w = _reference(from_dev(Z.contiguous())[:, :V], ids, 1.0, k)
    _compare(o, w, k)
    assert (w["top_ids"][:, :3] == [0, V - 1, 1]).all()


@pytest.mark.parametrize("V,k", [(70, 32), (5000, 20), (40000, 32)])
def test_ties_go_to_the_lowest_index(V, k):
    """Few distinct values, and rows of one value only."""
    torch, mt = need_gpu()
    rng = np.random.default_rng(V)
    z = rng.integers(0, 3, (4, V)).astype(np.float32)
    z[1] = 2.0
    z[2] = 0.0
    z[2, ::2] = -0.0  # equal to 0
    z[3] = np.arange(V)[::-1] // 7
    ids = np.zeros(4, np.int32)
    o = _run(torch, mt, to_dev_f32(torch, z), mt.MT_F32, torch.from_numpy(ids).cuda(), 1.0, k, 4, V, V)
    _compare(o, _reference(z, ids, 1.0, k), k)


def test_rows_left_out_and_extreme_logits():
    torch, mt = need_gpu()
    V, k = 3000, 4
    low32, lowbf = np.finfo(np.float32).min, -3.3895314e38
    rng = np.random.default_rng(0)
    rows, ids = [], []

    def row(fill, put=(), i=5):
        r = np.full(V, fill, np.float32)
        for at, v in put:
            r[at] = v
        rows.append(r)
        ids.append(i)

    row(-np.inf)                                    # nothing left
    row(low32), row(lowbf)                          # nothing left, by the types' lowest values
    row(-np.inf, [(2999, 1.5)])                     # one token left, not the given one
    row(-np.inf, [(5, 1.5)])                        # one token left, the given one
    row(low32, [(7, 0.0), (100, 1.0)], 100)         # two left
    row(0.0, [(9, np.nan)]), row(0.0, [(9, np.inf)])
    row(-np.inf, [(2998, np.nan)])
    row(0.0, [(3, np.inf)], -1)                     # not scored: not read
    row(1e29, [(8, 1.2e30), (9, -3e38)], 8)         # far apart
    row(-1e30, (), 3)                               # all near the bottom of the range
    row(-1e29, (), 2999)
    rows.append((50 * rng.standard_normal(V)).astype(np.float32)), ids.append(17)
    z, ids = np.stack(rows), np.array(ids, np.int32)
    T = len(ids)
    Z, IDS = to_dev_f32(torch, z), torch.from_numpy(ids).cuda()
    for c in (1.0, 0.5):
        o = _run(torch, mt, Z, mt.MT_F32, IDS, c, k, T, V, V)
        _compare(o, _reference(z, ids, c, k), k)
    # gradients: zero where nothing is scored or left, NaN where the row is
    o = _run(torch, mt, Z, mt.MT_F32, IDS, 1.0, 0, T, V, V)
    D = torch.full((T, V), 7.0, device="cuda")
    one = torch.ones(T, device="cuda")
    mt.mt_op_token_logprobs_bwd(Z, mt.MT_F32, IDS, 1.0, o["lse"], o["ent"], one, one, D, mt.MT_F32, T, V, V, V)
    d = from_dev(D)
    for t in (0, 1, 2, 9):
        assert np.all(d[t] == 0)
    for t in (6, 7, 8):
        assert np.all(np.isnan(d[t]))
    want = np.zeros(V)
    want[5], want[2999] = 1, -1
    assert np.array_equal(d[3], want)
    assert np.all(d[4] == 0)
    assert np.all(np.isfinite(d[[5, 10, 12, 13]]))


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("low", [-np.inf, -3.3e38, -2.0 ** 100])
@pytest.mark.parametrize("c", [1e6, 4e4, 1e-6])
def test_masked_stretches_at_the_temperatures_ends(c, low, bf16):
    """Whole threads and warps of masked logits beside few live ones, at the
    smallest and largest temperature: statistics as in float64, finite
    gradients, none where the mask is."""
    torch, mt = need_gpu()
    T, V, k = 4, 70001, 3
    z = np.full((T, V), low, np.float32)
    z[0, 5], z[0, 69990] = 1.0, 1.0
    z[1, :16] = 0.25
    z[2, 35000:35002] = (-3.0, 2.0)
    z[3, 70000] = -1e29
    Z = torch.from_numpy(z).cuda().to(torch.bfloat16 if bf16 else torch.float32)
    code = mt.MT_BF16 if bf16 else mt.MT_F32
    ids = np.array([5, 3, 35001, 0], np.int32)
    IDS, c64 = torch.from_numpy(ids).cuda(), float(np.float32(c))
    o = _run(torch, mt, Z, code, IDS, c, k, T, V, V)
    w = _reference(from_dev(Z), ids, c64, k)
    _compare(o, w, k)
    for gl, ge in ((1.0, 1e3), (0.0, 1.0)):
        D = torch.full((T, V), 7.0, device="cuda")
        GL, GE = torch.full((T,), gl, device="cuda"), torch.full((T,), ge, device="cuda")
        mt.mt_op_token_logprobs_bwd(Z, code, IDS, c, o["lse"], o["ent"], GL, GE, D, mt.MT_F32, T, V, V, V)
        d = from_dev(D).copy()
        assert np.isfinite(d).all()
        if gl:  # the given token's own term, where it is masked out itself
            assert d[3, 0] == np.float32(c)
            d[3, 0] = 0
        assert np.all(d[~(from_dev(Z) > -BIG)] == 0)


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("T,V,k", [(1, 151936, 20), (2, 32000, 32), (40, 9000, 8), (5, 40003, 1), (300, 30000, 20)])
@pytest.mark.parametrize("pattern", ["soft_mask", "half", "ascending", "descending", "plateau", "stretch", "stripes"])
def test_uneven_rows(pattern, T, V, k, bf16):
    """Rows whose largest logits sit together, or whose threads and warps see
    nothing but low ones: bounds on the k-th largest that the threads' maxima
    give are far off there."""
    torch, mt = need_gpu()
    rng = np.random.default_rng(V + k)
    z = rng.standard_normal((T, V)).astype(np.float32)
    i = np.arange(V)
    if pattern == "soft_mask":
        z[:, (i < V // 3) | (i > V // 3 + 200)] -= 1e9
    elif pattern == "half":
        z[:, :V // 2] = -np.inf
    elif pattern == "ascending":
        z = np.broadcast_to(i / 1000, (T, V)).astype(np.float32)
    elif pattern == "descending":
        z = np.broadcast_to(-i / 1000, (T, V)).astype(np.float32)
    elif pattern == "plateau":
        z = np.where(rng.random((T, V)) < 0.02, 3, rng.integers(-3, 3, (T, V))).astype(np.float32)
    elif pattern == "stretch":
        z[:, V // 2:V // 2 + 700] += 20
    else:
        z[:, (i // 1024) % 3 != 1] -= 50
    Z = torch.from_numpy(np.ascontiguousarray(z)).cuda().to(torch.bfloat16 if bf16 else torch.float32)
    ids = rng.integers(0, V, T).astype(np.int32)
    o = _run(torch, mt, Z, mt.MT_BF16 if bf16 else mt.MT_F32, torch.from_numpy(ids).cuda(), 1.0, k, T, V, V)
    _compare(o, _reference(from_dev(Z), ids, 1.0, k), k)


def test_ids_past_the_vocabulary_are_reported():
    torch, mt = need_gpu()
    V = 100
    Z = torch.zeros((3, V), device="cuda")
    ids = torch.tensor([1, V, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    assert mt.mt_op_device_error() == 0
    o = _run(torch, mt, Z, mt.MT_F32, ids, 1.0, 2, 3, V, V)
    assert mt.mt_op_device_error() != 0
    assert mt.mt_op_device_error() == 0
    assert np.isnan(from_dev(o["logp"])[1:]).all() and np.isfinite(from_dev(o["logp"])[0])
    assert (o["top_ids"].cpu().numpy()[1:] == -1).all()
    D = torch.full((3, V), 7.0, device="cuda")
    g = torch.ones(3, device="cuda")
    mt.mt_op_token_logprobs_bwd(Z, mt.MT_F32, ids, 1.0, o["lse"], o["ent"], g, g, D, mt.MT_F32, 3, V, V, V)
    assert np.all(from_dev(D)[1:] == 0)


@pytest.mark.parametrize("zb,db", [(False, False), (False, True), (True, True), (True, False)])
@pytest.mark.parametrize("T,V,ld,ldd", [(1, 1, 1, 1), (3, 7, 9, 8), (5, 1000, 1000, 1000), (2, 9001, 9001, 9003),
                                        (3, 40000, 40008, 40000), (20, 823, 823, 823), (9, 4101, 4101, 4109)])
@pytest.mark.parametrize("grads", ["both", "logp", "entropy"])
def test_backward(zb, db, T, V, ld, ldd, grads):
    torch, mt = need_gpu()
    rng = np.random.default_rng(V + T)
    z = (3.0 * rng.standard_normal((T, ld))).astype(np.float32)
    if V > 64:
        z[rng.random((T, ld)) < 0.1] = -np.inf
    Z = torch.from_numpy(z).cuda().to(torch.bfloat16 if zb else torch.float32)
    z = from_dev(Z)[:, :V].astype(np.float64)
    ids = rng.integers(0, V, T).astype(np.int32)
    if T > 2:
        ids[1] = -1
    c = 0.8
    c64 = float(np.float32(c))
    gl = rng.standard_normal(T).astype(np.float32) if grads != "entropy" else None
    ge = rng.standard_normal(T).astype(np.float32) if grads != "logp" else None
    zc = z * c64
    m = zc.max(axis=1)
    m = np.where(np.isfinite(m), m, 0)
    lse = (m + np.log(np.exp(zc - m[:, None]).sum(axis=1))).astype(np.float32)
    lp = zc - lse[:, None].astype(np.float64)  # the kernel's definition: p = e^{z - lse} with the lse it is given
    p = np.exp(lp)
    lp0 = np.where(p > 0, lp, 0.0)
    H = (-(p * lp0).sum(axis=1)).astype(np.float32)
    GL, GE = (None if g is None else to_dev_f32(torch, g) for g in (gl, ge))
    D = torch.full((T, ldd), 7.0, device="cuda").to(torch.bfloat16 if db else torch.float32)
    mt.mt_op_token_logprobs_bwd(Z, mt.MT_BF16 if zb else mt.MT_F32, torch.from_numpy(ids).cuda(), c,
                                to_dev_f32(torch, lse), to_dev_f32(torch, H), GL, GE, D,
                                mt.MT_BF16 if db else mt.MT_F32, T, V, ld, ldd)
    a = np.zeros(T) if gl is None else gl.astype(np.float64)
    b = np.zeros(T) if ge is None else ge.astype(np.float64)
    hot = np.zeros((T, V))
    hot[np.arange(T), np.maximum(ids, 0)] = 1
    A, Bm, Hc = a[:, None], b[:, None], H[:, None].astype(np.float64)
    want = c64 * (A * (hot - p) - Bm * p * (lp0 + Hc))
    mag = p * (np.abs(A) + np.abs(Bm) * (np.abs(lp0) + np.abs(Hc)))
    bound = c64 * ((2.0 ** -21 + 6 * U32 * np.abs(lp0)) * mag + 8 * U32 * (mag + np.abs(A) * hot) +
                   4 * U32 * np.abs(Bm) * p * (np.abs(lp0) + np.abs(np.where(p > 0, zc, 0.0))))
    # log p itself carries the rounding of z c - lse
    bound += (U16 if db else U32) * np.abs(want) + 1e-36
    skip = ids < 0
    want[skip] = 0
    assert np.isfinite(want).all() and np.isfinite(bound).all()
    got = from_dev(D)
    check(got[:, :V], want, bound, "dlogits")
    assert np.all(got[:, V:] == 7.0)


@pytest.mark.parametrize("T,V", [(6, 5000), (11, 5003)])
def test_backward_in_place(T, V):
    torch, mt = need_gpu()
    for dt, code in ((torch.float32, mt.MT_F32), (torch.bfloat16, mt.MT_BF16)):
        Z = torch.randn((T, V), device="cuda").to(dt)
        ids = torch.randint(0, V, (T,), device="cuda").int()
        o = _run(torch, mt, Z, code, ids, 1.0, 0, T, V, V)
        g = torch.randn(T, device="cuda")
        D = torch.empty_like(Z)
        args = (code, ids, 1.0, o["lse"], o["ent"], g, g)
        mt.mt_op_token_logprobs_bwd(Z, *args, D, code, T, V, V, V)
        mt.mt_op_token_logprobs_bwd(Z, *args, Z, code, T, V, V, V)
        assert torch.equal(Z, D)


def test_gradient_against_differences():
    """d(sum_t a_t logp_t + b_t H_t)/dz by central differences of the float64 forward."""
    torch, mt = need_gpu()
    T, V, c = 2, 50, 0.7
    rng = np.random.default_rng(3)
    z = rng.standard_normal((T, V)).astype(np.float32)
    ids = np.array([4, 30], np.int32)
    a, b = np.array([0.5, -1.5]), np.array([0.25, 1.0])
    Z, IDS = to_dev_f32(torch, z), torch.from_numpy(ids).cuda()
    o = _run(torch, mt, Z, mt.MT_F32, IDS, c, 0, T, V, V)
    D = torch.empty((T, V), device="cuda")
    mt.mt_op_token_logprobs_bwd(Z, mt.MT_F32, IDS, c, o["lse"], o["ent"], to_dev_f32(torch, a), to_dev_f32(torch, b),
                                D, mt.MT_F32, T, V, V, V)
    c64 = float(np.float32(c))

    def f(x):
        y = c64 * x
        lp = y - np.log(np.exp(y).sum(axis=1, keepdims=True))
        return float((a * lp[np.arange(T), ids]).sum() - (b * (np.exp(lp) * lp).sum(axis=1)).sum())

    d = 1e-5
    for t, j in ((0, 4), (0, 9), (1, 30), (1, 0)):
        e = np.zeros((T, V))
        e[t, j] = d
        assert abs(float(D[t, j]) - (f(z + e) - f(z - e)) / (2 * d)) < 5e-6


def test_full_size_rows_sampled():
    """8192 rows of the 8B vocabulary (offsets past 32 bits in bytes): sampled rows against float64."""
    torch, mt = need_gpu()
    T, V, k = 8192, 128256, 8
    Z = torch.randn((T, V), device="cuda") * 2
    ids = torch.randint(0, V, (T,), device="cuda").int()
    o = _run(torch, mt, Z, mt.MT_F32, ids, 1.0, k, T, V, V)
    g = torch.randn(T, device="cuda")
    D = torch.empty((T, V), dtype=torch.bfloat16, device="cuda")
    mt.mt_op_token_logprobs_bwd(Z, mt.MT_F32, ids, 1.0, o["lse"], o["ent"], g, None, D, mt.MT_BF16, T, V, V, V)
    pick = [0, 1, 4095, 8190, 8191]
    w = _reference(from_dev(Z[pick]), ids.cpu().numpy()[pick], 1.0, k)
    _compare({n: v[pick] for n, v in o.items()}, w, k)
    for t in pick:
        lp = from_dev(Z[t]).astype(np.float64) - float(o["lse"][t])
        want = -np.exp(lp) * float(g[t])
        want[int(ids[t])] += float(g[t])
        check(from_dev(D[t]), want, (U16 + 2.0 ** -20) * np.abs(want) + 2.0 ** -20 * np.exp(lp) * abs(float(g[t])) + 1e-36)


@pytest.fixture
def emptied():
    """Gives the large buffers back to the device."""
    yield
    import torch
    torch.cuda.empty_cache()


def test_row_offsets_past_32_bits(emptied):
    """Rows 2^30 elements and some apart: the same bits as the rows close together."""
    torch, mt = need_gpu()
    T, V, k, far = 4, 5003, 5, (1 << 30) + 8
    ids = torch.tensor([3, 0, 5002, 77], dtype=torch.int32, device="cuda")
    z = torch.randn((T, V), device="cuda").to(torch.bfloat16)
    g = torch.randn(T, device="cuda")
    outs = []
    for ld in (5008, far):
        Z = torch.empty(((T - 1) * ld + V,), dtype=torch.bfloat16, device="cuda").as_strided((T, V), (ld, 1))
        Z.copy_(z)
        o = _run(torch, mt, Z, mt.MT_BF16, ids, 1.0, k, T, V, ld)
        mt.mt_op_token_logprobs_bwd(Z, mt.MT_BF16, ids, 1.0, o["lse"], o["ent"], g, g, Z, mt.MT_BF16, T, V, ld, ld)
        outs.append(list(o.values()) + [Z.clone()])
        del Z
    for a, b in zip(*outs):
        assert torch.equal(a, b)


def test_one_very_long_row(emptied):
    """300 million logits: sums of that many terms, and indices past 2^28."""
    torch, mt = need_gpu()
    V, k = 300_000_007, 4
    z = torch.zeros((1, V), dtype=torch.bfloat16, device="cuda")
    z[0, ::2] = 1.0
    z[0, [299_999_998, 5, 268_435_457]] = torch.tensor([9.0, 8.0, 7.0], dtype=torch.bfloat16, device="cuda")
    ids = torch.tensor([268_435_457], dtype=torch.int32, device="cuda")
    o = _run(torch, mt, z, mt.MT_BF16, ids, 1.0, k, 1, V, V)
    # 299999998 is even, the other two odd; half of the rest has 1, half 0
    ones, zeros = (V + 1) // 2 - 1, V // 2 - 2
    terms = np.array([ones, zeros, 1, 1, 1]) * np.exp(np.array([1.0, 0, 9, 8, 7]) - 9)
    S, lse = terms.sum(), 9 + np.log(terms.sum())
    es = 2.0 ** -21 + acc(V) + 4 * U32 * (terms * np.array([8, 9, 0, 1, 2])).sum() / S
    bound = es + 2 * U32 * (np.log(S) + 9)
    assert abs(float(o["lse"]) - lse) <= bound and abs(float(o["logp"]) - (7 - lse)) <= bound
    p = terms / S
    ent = -(p[:2] * (np.array([1.0, 0]) - lse)).sum() - (p[2:] * (np.array([9.0, 8, 7]) - lse)).sum()
    B = (p * np.array([8, 9, 0, 1, 2])).sum()
    assert abs(float(o["ent"]) - ent) <= es * (1 + B) + (2.0 ** -21 + acc(V)) * B + 8 * U32 * (81 + B) + 2 * U32 * np.log(S)
    assert o["top_ids"].tolist() == [[299_999_998, 5, 268_435_457, 0]]
    want = np.array([9.0, 8, 7, 1]) - lse
    assert np.all(np.abs(from_dev(o["top_logp"])[0] - want) <= bound + 2 * U32 * np.abs(want))
