"""Every argument that the checkpoint, token and embedding entry points
refuse, one at a time, with the exact code: MT_ERR_ARG and nothing else. On a
machine without a device a request that passed the checks answers
MT_ERR_CUDA (its launch fails), so a check that is missing shows."""
import pytest
import torch

import layer_streamed_gb300 as mt

# with a device a check that is missing would launch a kernel on this file's host memory
pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="requests on host memory: only where no launch can succeed")

F, B = mt.MT_F32, mt.MT_BF16
INT_MAX = (1 << 31) - 1


def _aligned(nbytes, off=0, boundary=256):
    """A host buffer that starts `off` bytes past a boundary."""
    raw = torch.zeros(nbytes + 2 * boundary, dtype=torch.uint8)
    at = -raw.data_ptr() % boundary + off
    return raw[at:at + nbytes]


buf = _aligned(1 << 16)
off1, off2, off4, off8, off16 = (_aligned(1 << 16, k) for k in (1, 2, 4, 8, 16))

# entry point: (positional names, a request that is sound, requests that are not)
CALLS = {
    "mt_op_ckpt8_pack": (
        "x dt fmt codes scales T n ldx ldc",
        dict(x=buf, dt=F, fmt=1, codes=buf, scales=buf, T=2, n=8, ldx=8, ldc=8),
        [dict(x=None), dict(codes=None), dict(scales=None), dict(dt=2), dict(dt=-1), dict(fmt=0), dict(fmt=3),
         dict(fmt=-1), dict(T=0), dict(T=-1), dict(T=(1 << 30) + 1), dict(n=0), dict(n=-1), dict(ldx=7), dict(ldc=7),
         dict(ldx=(1 << 29) + 1), dict(ldc=(1 << 29) + 1), dict(x=off2), dict(x=off1, dt=B)]),
    "mt_op_ckpt8_unpack": (
        "codes scales fmt x dt T n ldc ldx",
        dict(x=buf, dt=F, fmt=1, codes=buf, scales=buf, T=2, n=8, ldx=8, ldc=8),
        [dict(x=None), dict(codes=None), dict(scales=None), dict(dt=2), dict(dt=-1), dict(fmt=0), dict(fmt=3),
         dict(T=0), dict(T=-1), dict(T=(1 << 30) + 1), dict(n=0), dict(ldx=7), dict(ldc=7), dict(ldx=(1 << 29) + 1),
         dict(ldc=(1 << 29) + 1), dict(x=off2), dict(x=off1, dt=B)]),
    "mt_op_rmsnorm_fwd_ckpt8": (
        "x w y rstd codes scales fmt T h eps",
        dict(x=buf, w=buf, y=buf, rstd=buf, codes=buf, scales=buf, fmt=1, T=2, h=8, eps=1e-5),
        [dict(x=None), dict(w=None), dict(y=None), dict(rstd=None), dict(codes=None), dict(scales=None), dict(fmt=0),
         dict(fmt=3), dict(T=0), dict(T=-1), dict(h=0), dict(h=6), dict(h=8196), dict(x=off8), dict(w=off8),
         dict(y=off4), dict(rstd=off2), dict(codes=off2)]),
    "mt_op_rmsnorm_bwd_ckpt8": (
        "codes scales fmt w rstd dy resid dx dxb dw ws T h",
        dict(codes=buf, scales=buf, fmt=1, w=buf, rstd=buf, dy=buf, resid=buf, dx=buf, dxb=buf, dw=buf, ws=buf, T=2, h=8),
        [dict(codes=None), dict(scales=None), dict(w=None), dict(rstd=None), dict(dy=None), dict(dx=None), dict(dw=None),
         dict(ws=None), dict(fmt=0), dict(fmt=3), dict(T=0), dict(T=-1), dict(h=0), dict(h=6), dict(h=8196),
         dict(codes=off2), dict(w=off8), dict(rstd=off2), dict(dy=off8), dict(resid=off8), dict(dx=off8), dict(dxb=off4),
         dict(dw=off2), dict(ws=off8)]),
    "mt_op_swiglu_fwd_ckpt8": (
        "gu act codes scales fmt T F ld",
        dict(gu=buf, act=buf, codes=buf, scales=buf, fmt=1, T=2, F=8, ld=8),
        [dict(gu=None), dict(act=None), dict(codes=None), dict(scales=None), dict(fmt=0), dict(fmt=3), dict(T=0),
         dict(T=(1 << 30) + 1), dict(F=0), dict(F=9), dict(ld=(1 << 29) + 8), dict(gu=off1), dict(act=off1)]),
    "mt_op_swiglu_bwd_ckpt8": (
        "codes scales fmt dact dgu T F ld",
        dict(dact=buf, dgu=buf, codes=buf, scales=buf, fmt=1, T=2, F=8, ld=8),
        [dict(dact=None), dict(dgu=None), dict(codes=None), dict(scales=None), dict(fmt=0), dict(fmt=3), dict(T=0),
         dict(T=(1 << 30) + 1), dict(F=0), dict(F=9), dict(ld=(1 << 29) + 8), dict(dact=off1), dict(dgu=off1)]),
    "mt_op_token_logprobs": (
        "z dt ids c k lse logp ent ti tl T V ld",
        dict(z=buf, dt=F, ids=buf, c=1.0, k=2, lse=buf, logp=buf, ent=buf, ti=buf, tl=buf, T=2, V=8, ld=8),
        [dict(z=None), dict(ids=None), dict(lse=None), dict(logp=None), dict(ti=None), dict(tl=None), dict(dt=2),
         dict(dt=-1), dict(c=0.0), dict(c=-1.0), dict(c=9e-7), dict(c=1.1e6), dict(c=float("nan")), dict(c=float("inf")),
         dict(k=-1), dict(k=9), dict(k=33, V=64, ld=64), dict(T=0), dict(T=-1), dict(T=(1 << 28) + 1), dict(V=0),
         dict(V=-1), dict(ld=7), dict(z=off2), dict(z=off1, dt=B), dict(ids=off2), dict(lse=off2), dict(logp=off2),
         dict(ent=off2), dict(ti=off2), dict(tl=off2)]),
    "mt_op_token_logprobs_bwd": (
        "z dt ids c lse ent gl ge dz ddt T V ld ldd",
        dict(z=buf, dt=F, ids=buf, c=1.0, lse=buf, ent=buf, gl=buf, ge=buf, dz=buf, ddt=B, T=2, V=8, ld=8, ldd=8),
        [dict(z=None), dict(ids=None), dict(lse=None), dict(ent=None), dict(gl=None, ge=None), dict(dz=None), dict(dt=2),
         dict(ddt=3), dict(c=0.0), dict(c=float("nan")), dict(T=0), dict(T=-1), dict(V=0), dict(V=(1 << 30) + 1, ld=INT_MAX, ldd=INT_MAX),
         dict(ld=7), dict(ldd=7), dict(z=off2), dict(dz=off1), dict(dz=off2, ddt=F), dict(ids=off2), dict(lse=off2),
         dict(ent=off2), dict(gl=off2), dict(ge=off2)]),
    "mt_op_embed_fwd": (
        "t dt i s o od T V h",
        dict(t=buf, dt=F, i=buf, s=1.0, o=buf, od=F, T=2, V=3, h=4),
        [dict(t=None), dict(i=None), dict(o=None), dict(dt=2), dict(od=7), dict(T=0), dict(T=(1 << 28) + 1), dict(V=0),
         dict(V=1 << 30), dict(h=0), dict(h=(1 << 22) + 1), dict(t=off2), dict(t=off1, dt=B), dict(o=off2),
         dict(o=off1, od=B), dict(i=off2)]),
    "mt_op_embed_bwd": (
        "i d dt s o od acc ws T V h",
        dict(i=buf, d=buf, dt=F, s=1.0, o=buf, od=F, acc=0, ws=buf, T=2, V=3, h=4),
        [dict(i=None), dict(d=None), dict(o=None), dict(ws=None), dict(dt=2), dict(od=7), dict(T=0), dict(T=(1 << 28) + 1),
         dict(V=0), dict(V=1 << 30), dict(h=0), dict(h=(1 << 22) + 1), dict(d=off2), dict(d=off1, dt=B), dict(o=off2),
         dict(o=off1, od=B), dict(i=off2), dict(ws=off16)]),
}


@pytest.fixture(scope="module", autouse=True)
def built():
    mt.build()
    mt.lib()


def _code(name, **change):
    names, ok, _ = CALLS[name]
    a = {**ok, **change}
    try:
        getattr(mt, name)(*[a[k] for k in names.split()], 0)
    except mt.MtError as e:
        return e.code
    return mt.MT_OK


def _cases():
    for name, (_, _, bad) in CALLS.items():
        for change in bad:
            what = "-".join(f"{k}={'tensor' if torch.is_tensor(v) else v}" for k, v in change.items())
            yield pytest.param(name, change, id=f"{name[6:]}-{what}")


@pytest.mark.parametrize("name,change", list(_cases()))
def test_a_bad_argument_is_refused_as_such(name, change):
    assert _code(name, **change) == mt.MT_ERR_ARG


@pytest.mark.parametrize("name", CALLS)
def test_a_sound_request_passes_the_checks_and_its_failed_launch_says_so(name):
    assert _code(name) == mt.MT_ERR_CUDA
    # and the error that this leaves pending does not colour the next refusal
    assert _code(name, T=0) == mt.MT_ERR_ARG


@pytest.mark.parametrize("T", [(1 << 30) + 1, INT_MAX])
@pytest.mark.parametrize("h", [4, 8192])
def test_norm_backward_refuses_rows_its_counter_would_wrap_on(T, h):
    """A block looks up to eight rounds of the grid (1216 blocks for narrow
    rows) past its row: near 2^31 rows that sum is negative and names rows in
    front of the buffers."""
    assert _code("mt_op_rmsnorm_bwd_ckpt8", T=T, h=h) == mt.MT_ERR_ARG
    assert mt.mt_op_rmsnorm_bwd_ckpt8_workspace(T, h) == 0
    assert mt.mt_op_rmsnorm_bwd_ckpt8_workspace(1 << 30, h) > 0


@pytest.mark.parametrize("T", [(1 << 30) + 1, INT_MAX - (1 << 21), INT_MAX])
def test_logits_gradient_refuses_rows_its_counter_would_wrap_on(T):
    """The row counter steps by up to 65535 * 32 rows: within that of 2^31 it
    turns negative and passes the test against T."""
    for V in (1, 8):
        assert _code("mt_op_token_logprobs_bwd", T=T, V=V) == mt.MT_ERR_ARG


@pytest.mark.parametrize("T,h", [(1 << 28, 1 << 22), (1 << 28, 1 << 13), (1 << 20, 1 << 22), (1 << 28, 4), (1, 1 << 22)])
@pytest.mark.parametrize("od,off", [(F, 0), (B, 0), (F, 4)])
def test_embedding_workspace_is_nothing_exactly_where_the_gradient_is_refused(T, h, od, off):
    """Sizes, whatever the alignment and the types: the query answers 0 for
    those that the call refuses and for no others."""
    size = mt.mt_op_embed_bwd_workspace(T, 4, h)
    code = _code("mt_op_embed_bwd", T=T, V=4, h=h, od=od, d=off4 if off else buf)
    assert code == (mt.MT_ERR_CUDA if size else mt.MT_ERR_ARG)


@pytest.mark.parametrize("h,blocks", [(8192, 1), (4096, 1), (2048, 2), (512, 8), (4, 8)])
def test_norm_backward_workspace_does_not_depend_on_the_machine_that_asks(h, blocks):
    """The parts of as many blocks as 152 SMs hold, with or without a device."""
    assert mt.mt_op_rmsnorm_bwd_ckpt8_workspace(1 << 20, h) == 152 * blocks * h
    assert mt.mt_op_rmsnorm_bwd_ckpt8_workspace(3, h) == 3 * h
