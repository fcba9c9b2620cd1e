"""Every argument that the cross entropy from a head's inputs, the
orthogonalised updates and the norms around a block refuse, one at a time:
MT_ERR_ARG exactly. On a machine without a device a request that passed the
checks answers MT_ERR_CUDA, so a check that is missing shows."""
import numpy as np
import pytest
import torch

import layer_streamed_gb300 as mt

# with a device a check that is missing would launch a kernel on this file's host memory
pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="requests on host memory: only where no launch can succeed")

F, B = mt.MT_F32, mt.MT_BF16
INT_MAX = (1 << 31) - 1
nan, inf = float("nan"), float("inf")


def _aligned(nbytes, off=0, boundary=256):
    raw = torch.zeros(nbytes + 2 * boundary, dtype=torch.uint8)
    at = -raw.data_ptr() % boundary + off
    return raw[at:at + nbytes]


buf = _aligned(1 << 16)
off1, off2, off4, off8, off16 = (_aligned(1 << 16, k) for k in (1, 2, 4, 8, 16))
_ce = [dict(X=None), dict(W=None), dict(lab=None), dict(ws=None), dict(X=off8), dict(W=off8), dict(lab=off2), dict(ws=off16),
       dict(c=0.0), dict(c=9e-7), dict(c=1.1e6), dict(c=nan), dict(c=-1.0), dict(e=-0.1), dict(e=1.0), dict(e=nan), dict(z=-1e-3),
       dict(z=nan), dict(z=inf), dict(T=0), dict(T=-1), dict(T=(1 << 24) + 1), dict(V=0), dict(V=-1), dict(V=(1 << 24) + 1),
       dict(T=1 << 24, V=1 << 17), dict(h=0), dict(h=-8), dict(h=12), dict(h=(1 << 16) + 8, ldx=1 << 17, ldw=1 << 17),
       dict(ldx=8), dict(ldw=8), dict(ldx=20), dict(ldw=20)]
_ns = [dict(ws=None), dict(ws=off16), dict(steps=0), dict(steps=33), dict(steps=-1), dict(eps=-1e-7), dict(eps=nan), dict(eps=inf),
       dict(b=0), dict(b=-1), dict(b=4097), dict(r=0), dict(r=-1), dict(r=(1 << 16) + 1), dict(cc=0), dict(cc=(1 << 16) + 1),
       dict(b=4096, r=1 << 16, cc=1 << 16), dict(coef=np.full((5, 3), nan)), dict(coef=np.full((5, 3), inf)),
       dict(coef=np.full((5, 3), 100.5)), dict(coef=np.zeros((4, 3))), dict(G=None), dict(G=off2), dict(G=off1, gd=B), dict(gd=2),
       dict(gd=-1)]
_sn = [dict(y=None), dict(wa=None), dict(wb=None), dict(dt=2), dict(dt=-1), dict(T=0), dict(T=-1), dict(T=(1 << 30) + 1), dict(h=0),
       dict(h=6), dict(h=8196), dict(h=-4), dict(y=off4), dict(y=off8, dt=F), dict(gate=off4), dict(wa=off8), dict(wb=off8),
       dict(al=nan), dict(al=inf)]

CALLS = {
    "mt_op_linear_ce_fwd": (
        "X W lab c e z loss lse ws T V h ldx ldw",
        dict(X=buf, W=buf, lab=buf, c=1.0, e=0.1, z=1e-4, loss=buf, lse=buf, ws=buf, T=2, V=8, h=16, ldx=16, ldw=24),
        _ce + [dict(loss=None), dict(lse=None), dict(loss=off2), dict(lse=off2)]),
    "mt_op_linear_ce_bwd": (
        "X W lab c e z lse g dX xd dW wd acc ws T V h ldx ldw",
        dict(X=buf, W=buf, lab=buf, c=1.0, e=0.1, z=1e-4, lse=buf, g=buf, dX=buf, xd=B, dW=buf, wd=F, acc=0, ws=buf, T=2, V=8,
             h=16, ldx=16, ldw=24),
        _ce + [dict(lse=None), dict(g=None), dict(lse=off2), dict(g=off2), dict(dX=None, dW=None), dict(dX=off8), dict(dW=off8),
               dict(xd=2), dict(wd=-1)]),
    "mt_op_orthogonalize": (
        "G gd O od coef steps eps ws b r cc",
        dict(G=buf, gd=F, O=buf, od=B, coef=None, steps=5, eps=1e-7, ws=buf, b=1, r=4, cc=6),
        _ns + [dict(O=None), dict(O=off2, od=F), dict(O=off1), dict(od=2)]),
    "mt_op_muon_update": (
        "W wd M G gd mu nes lr decay scale coef steps eps ws b r cc",
        dict(W=buf, wd=B, M=buf, G=buf, gd=F, mu=0.95, nes=1, lr=0.01, decay=0.1, scale=1.0, coef=None, steps=5, eps=1e-7, ws=buf,
             b=1, r=4, cc=6),
        _ns + [dict(W=None), dict(W=off1), dict(W=off2, wd=F), dict(wd=3), dict(M=None), dict(M=off2), dict(mu=1.0), dict(mu=-0.1),
               dict(mu=nan), dict(lr=nan), dict(lr=inf), dict(decay=nan), dict(scale=inf)]),
    "mt_op_sandwich_norm_fwd": (
        "x y gate dt wa wb al eps xo n ra rb T h",
        dict(x=buf, y=buf, gate=buf, dt=B, wa=buf, wb=buf, al=0.9, eps=1e-5, xo=buf, n=buf, ra=buf, rb=buf, T=2, h=8),
        _sn + [dict(x=None), dict(xo=None), dict(n=None), dict(ra=None), dict(rb=None), dict(x=off8), dict(xo=off8), dict(n=off4),
               dict(ra=off2), dict(rb=off2), dict(eps=-1e-9), dict(eps=nan), dict(eps=inf)]),
    "mt_op_sandwich_norm_bwd": (
        "xo y gate dt wa wb al ra rb dn dres dx dy dg dwa dwb ws T h",
        dict(xo=buf, y=buf, gate=buf, dt=B, wa=buf, wb=buf, al=0.9, ra=buf, rb=buf, dn=buf, dres=buf, dx=buf, dy=buf, dg=buf,
             dwa=buf, dwb=buf, ws=buf, T=2, h=8),
        _sn + [dict(xo=None), dict(ra=None), dict(rb=None), dict(dn=None), dict(dx=None), dict(dy=None), dict(dg=None),
               dict(gate=None), dict(dwa=None), dict(dwb=None), dict(ws=None), dict(xo=off8), dict(ra=off2), dict(rb=off2),
               dict(dn=off8), dict(dres=off8), dict(dx=off8), dict(dy=off4), dict(dg=off4), dict(dwa=off2), dict(dwb=off2),
               dict(ws=off8)]),
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
        for i, change in enumerate(bad):
            what = "-".join(f"{k}={v if isinstance(v, (int, float, type(None))) else type(v).__name__}" for k, v in change.items())
            yield pytest.param(name, change, id=f"{name[6:]}-{i}-{what}")


@pytest.mark.parametrize("name,change", list(_cases()))
def test_a_bad_argument_is_refused_as_such(name, change):
    assert _code(name, **change) == mt.MT_ERR_ARG


@pytest.mark.parametrize("name", CALLS)
def test_a_sound_request_passes_the_checks_and_its_failed_launch_says_so(name):
    assert _code(name) == mt.MT_ERR_CUDA
    # and the error that this leaves pending does not colour the next refusal
    assert _code(name, T=0, b=0) == mt.MT_ERR_ARG


def test_optional_operands():
    assert _code("mt_op_linear_ce_bwd", dX=None) == mt.MT_ERR_CUDA
    assert _code("mt_op_linear_ce_bwd", dW=None, acc=1) == mt.MT_ERR_CUDA
    assert _code("mt_op_sandwich_norm_fwd", gate=None) == mt.MT_ERR_CUDA
    assert _code("mt_op_sandwich_norm_bwd", gate=None, dg=None, dres=None) == mt.MT_ERR_CUDA
    assert _code("mt_op_orthogonalize", coef=[(1.5, -0.5, 0.0)] * 5) == mt.MT_ERR_CUDA


def test_workspaces_are_nothing_for_sizes_that_are_refused():
    for T, V, h in ((0, 8, 16), (2, 0, 16), (2, 8, 12), (2, 8, 0), ((1 << 24) + 1, 8, 16), (1 << 24, 1 << 17, 16), (2, 8, (1 << 16) + 8)):
        assert mt.mt_op_linear_ce_fwd_workspace(T, V, h) == 0 and mt.mt_op_linear_ce_bwd_workspace(T, V, h) == 0
    for a in ((0, 4, 4), (1, 0, 4), (1, 4, (1 << 16) + 1), (4097, 4, 4), (4096, 1 << 16, 1 << 16)):
        assert mt.mt_op_orthogonalize_workspace(*a) == 0
    for T, h in ((0, 8), (1, 0), (1, 6), (1, 8196), (-1, 8), ((1 << 30) + 1, 8)):
        assert mt.mt_op_sandwich_norm_bwd_workspace(T, h) == 0


@pytest.mark.parametrize("T,V,h", [(1, 1, 8), (8192, 128256, 4096), (1 << 24, 256, 8), (1 << 16, 1 << 24, 64), (7, 1 << 24, 1 << 16)])
def test_cross_entropy_keeps_less_than_the_logits(T, V, h):
    """A piece's dz (2^28 values, or 256 columns), X, and one fp32 X or the partial sums that a GPU's tiles need."""
    bwd = mt.mt_op_linear_ce_bwd_workspace(T, V, h)
    assert 0 < bwd <= 2 * max(1 << 28, 256 * T) + 6 * T * h + 152 * 2 * 65536 * 4 + (1 << 12)
    assert 0 < mt.mt_op_linear_ce_fwd_workspace(T, V, h) <= T * (24 * (V // 128 + 1) + 8) + (1 << 12)


@pytest.mark.parametrize("h", [4, 64, 4096, 4100, 6144, 8192])
def test_norm_workspace_does_not_depend_on_the_machine_that_asks(h):
    blocks = 1 if h > 2048 else min(8, 1024 // max(32, (h // 4 + 31) // 32 * 32))
    assert mt.mt_op_sandwich_norm_bwd_workspace(1 << 20, h) == 152 * blocks * 2 * h
    assert mt.mt_op_sandwich_norm_bwd_workspace(3, h) == 3 * 2 * h
