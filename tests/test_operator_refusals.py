"""What the checkpoint, token and embedding entry points refuse before
anything runs (no GPU needed: the arguments are checked on the host)."""
import pytest
import torch

import layer_streamed_gb300 as mt

F, B = mt.MT_F32, mt.MT_BF16


@pytest.fixture(scope="module", autouse=True)
def built():
    mt.build()
    mt.lib()


def _refused(call, code=mt.MT_ERR_ARG):
    with pytest.raises(mt.MtError) as e:
        call()
    # with no device at all a refusal may come after the runtime has noticed that
    assert e.value.code in (code, mt.MT_ERR_CUDA)


buf = torch.zeros(4096, dtype=torch.float32)
odd = torch.zeros(4097, dtype=torch.uint8)[1:]


def test_ckpt8_refusals():
    ok = dict(x=buf, dt=F, fmt=1, codes=buf, scales=buf, T=2, n=8, ldx=8, ldc=8)
    bad = [dict(x=None), dict(codes=None), dict(scales=None), dict(dt=2), dict(dt=-1), dict(fmt=0), dict(fmt=3),
           dict(T=0), dict(T=-1), dict(n=0), dict(ldx=7), dict(ldc=7), dict(x=odd), dict(ldx=(1 << 29) + 1),
           dict(T=(1 << 30) + 1)]
    for b in bad:
        a = {**ok, **b}
        _refused(lambda: mt.mt_op_ckpt8_pack(a["x"], a["dt"], a["fmt"], a["codes"], a["scales"], a["T"], a["n"],
                                             a["ldx"], a["ldc"], 0))
        _refused(lambda: mt.mt_op_ckpt8_unpack(a["codes"], a["scales"], a["fmt"], a["x"], a["dt"], a["T"], a["n"],
                                               a["ldc"], a["ldx"], 0))


def test_rmsnorm_ckpt8_refusals():
    for T, h, fmt, x in ((0, 8, 1, buf), (1, 6, 1, buf), (1, 8196, 1, buf), (1, 8, 0, buf), (1, 8, 1, None),
                         (1, 8, 1, buf[1:])):
        _refused(lambda: mt.mt_op_rmsnorm_fwd_ckpt8(x, buf, buf, buf, buf, buf, fmt, T, h, 1e-5, 0))
        _refused(lambda: mt.mt_op_rmsnorm_bwd_ckpt8(buf, buf, fmt, buf, buf, x, None, buf, None, buf, buf, T, h, 0))
    _refused(lambda: mt.mt_op_rmsnorm_bwd_ckpt8(buf, buf, 1, buf, buf, buf, None, buf, None, buf, None, 1, 8, 0))
    _refused(lambda: mt.mt_op_rmsnorm_fwd_ckpt8(buf, buf, buf, odd, buf, buf, 1, 1, 8, 1e-5, 0))
    _refused(lambda: mt.mt_op_rmsnorm_bwd_ckpt8(buf, buf, 1, buf, odd, buf, None, buf, None, buf, buf, 1, 8, 0))
    _refused(lambda: mt.mt_op_rmsnorm_bwd_ckpt8(buf, buf, 1, buf, buf, buf, None, buf, None, odd, buf, 1, 8, 0))
    for T, h in ((0, 8), (1, 0), (1, 6), (1, 8196), (1, 1 << 20), (-1, 8), (1, -8)):
        assert mt.mt_op_rmsnorm_bwd_ckpt8_workspace(T, h) == 0
    assert mt.mt_op_rmsnorm_bwd_ckpt8_workspace(1, 8) >= 8


def test_swiglu_ckpt8_refusals():
    for T, F_, ld, fmt, p in ((0, 8, 8, 1, buf), (1, 0, 8, 1, buf), (1, 9, 8, 1, buf), (1, 8, 8, 5, buf),
                              (1, 8, 8, 1, None), (1, 8, 8, 1, odd), (1, 8, (1 << 29) + 8, 1, buf)):
        _refused(lambda: mt.mt_op_swiglu_fwd_ckpt8(p, buf, buf, buf, fmt, T, F_, ld, 0))
        _refused(lambda: mt.mt_op_swiglu_bwd_ckpt8(buf, buf, fmt, p, buf, T, F_, ld, 0))


def test_token_logprobs_refusals():
    ok = dict(z=buf, dt=F, ids=buf, c=1.0, k=2, lse=buf, logp=buf, ti=buf, tl=buf, T=2, V=8, ld=8)
    bad = [dict(z=None), dict(ids=None), dict(lse=None), dict(logp=None), dict(ti=None), dict(tl=None), dict(dt=2),
           dict(c=0.0), dict(c=-1.0), dict(c=float("nan")), dict(c=float("inf")), dict(k=-1), dict(k=9), dict(k=33, V=64, ld=64),
           dict(T=0), dict(V=0), dict(ld=7), dict(z=odd), dict(ids=odd), dict(lse=odd), dict(logp=odd), dict(ti=odd),
           dict(tl=odd)]
    for b in bad:
        a = {**ok, **b}
        _refused(lambda: mt.mt_op_token_logprobs(a["z"], a["dt"], a["ids"], a["c"], a["k"], a["lse"], a["logp"], None,
                                                 a["ti"], a["tl"], a["T"], a["V"], a["ld"], 0))
    ok = dict(z=buf, dt=F, ids=buf, c=1.0, lse=buf, ent=buf, gl=buf, ge=buf, dz=buf, ddt=B, T=2, V=8, ld=8, ldd=8)
    bad = [dict(z=None), dict(ids=None), dict(lse=None), dict(ent=None), dict(gl=None, ge=None), dict(dz=None),
           dict(dt=2), dict(ddt=3), dict(c=0.0), dict(T=0), dict(V=0), dict(ld=7), dict(ldd=7), dict(dz=odd),
           dict(ids=odd), dict(lse=odd), dict(ent=odd), dict(gl=odd), dict(ge=odd)]
    for b in bad:
        a = {**ok, **b}
        _refused(lambda: mt.mt_op_token_logprobs_bwd(a["z"], a["dt"], a["ids"], a["c"], a["lse"], a["ent"], a["gl"],
                                                     a["ge"], a["dz"], a["ddt"], a["T"], a["V"], a["ld"], a["ldd"], 0))


def test_embedding_refusals():
    for a in (dict(t=None), dict(i=None), dict(o=None), dict(dt=2), dict(od=7), dict(T=0), dict(V=0), dict(h=0),
              dict(t=odd), dict(i=odd), dict(o=odd), dict(T=(1 << 28) + 1), dict(V=1 << 30)):
        a = {**dict(t=buf, i=buf, o=buf, dt=F, od=F, T=2, V=3, h=4), **a}
        _refused(lambda: mt.mt_op_embed_fwd(a["t"], a["dt"], a["i"], 1.0, a["o"], a["od"], a["T"], a["V"], a["h"], 0))
        _refused(lambda: mt.mt_op_embed_bwd(a["i"], a["t"], a["dt"], 1.0, a["o"], a["od"], 0, buf, a["T"], a["V"],
                                            a["h"], 0))
    al = torch.zeros(8192, dtype=torch.uint8)
    off = (-al.data_ptr()) % 256 + 16  # a workspace off its 256-byte boundary
    _refused(lambda: mt.mt_op_embed_bwd(buf, buf, F, 1.0, buf, F, 0, al[off:], 2, 3, 4, 0))
    assert mt.mt_op_embed_bwd_workspace(0, 3, 4) == 0
    assert mt.mt_op_embed_bwd_workspace(2, 3, 4) > 0


def test_checkpoint_format_in_the_configuration():
    def budget(fmt):
        return mt.mt_required_budget(mt.make_cfg(4, 64, 4, 4, 16, 172, 256, max_batch=2, max_seq=512, max_K=1,
                                                 ckpt_format=fmt))
    T, h, L = 1024, 64, 4
    saved = budget(mt.MT_CKPT_F32) - budget(mt.MT_CKPT_I8)
    assert budget(mt.MT_CKPT_I8) == budget(mt.MT_CKPT_E4M3)
    # four checkpoints shrink from 4 bytes to 1 + 1/32 a value, against more partial sums of the norm backward
    parts = mt.mt_op_rmsnorm_bwd_ckpt8_workspace(T, h) - mt.mt_op_rmsnorm_bwd_workspace(T, h)
    assert saved == L * (4 * T * h - T * h - T * h // 32) - max(parts, 0) * 4
    assert budget(3) == 0 and budget(-1) == 0
