"""mt_layer_cfg keeps the size and the meaning that it had before ckpt_format:
a program built against the header without that field passes a shorter
struct, and whatever lies behind it must not choose a checkpoint format."""
import ctypes
import os
import subprocess

import pytest

import layer_streamed_gb300 as mt

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module", autouse=True)
def built():
    mt.build()
    mt.lib()


class _WithoutFormat(ctypes.Structure):
    """The struct up to a 32-bit grad_dtype, then the caller's own memory."""
    _fields_ = [("ints", ctypes.c_int32 * 7), ("rope_theta", ctypes.c_float), ("norm_eps", ctypes.c_float),
                ("more", ctypes.c_int32 * 7), ("grad_dtype", ctypes.c_int32), ("behind", ctypes.c_int32 * 4)]


@pytest.mark.parametrize("behind", [0, 1, 2, 7, -1])
@pytest.mark.parametrize("grad", [mt.MT_F32, mt.MT_BF16])
def test_memory_behind_the_shorter_struct_is_not_read(behind, grad):
    old = _WithoutFormat((4, 64, 4, 4, 16, 172, 256), 1e4, 1e-5, (2, 512, 1, mt.MT_F32, 0, 0, 0), grad, (behind,) * 4)
    got = mt.lib().mt_required_budget(ctypes.cast(ctypes.pointer(old), ctypes.POINTER(mt.mt_layer_cfg)))
    assert got == mt.mt_required_budget(mt.make_cfg(4, 64, 4, 4, 16, 172, 256, max_batch=2, max_seq=512, max_K=1,
                                                    grad_dtype=grad)) > 0


def test_layout_of_the_header(tmp_path):
    src = tmp_path / "layout.c"
    src.write_text('#include <stddef.h>\n#include "mt.h"\n'
                   "_Static_assert(sizeof(mt_layer_cfg) == 68, \"size\");\n"
                   "_Static_assert(offsetof(mt_layer_cfg, grad_dtype) == 64, \"grad_dtype\");\n"
                   "_Static_assert(offsetof(mt_layer_cfg, ckpt_format) == 66, \"ckpt_format\");\n")
    subprocess.run(["gcc", "-std=c11", "-fsyntax-only", "-I", os.path.join(ROOT, "include"), str(src)], check=True)
    assert ctypes.sizeof(mt.mt_layer_cfg) == 68
    assert mt.mt_layer_cfg.grad_dtype.offset == 64 and mt.mt_layer_cfg.ckpt_format.offset == 66


@pytest.mark.parametrize("field", ["grad_dtype", "ckpt_format"])
@pytest.mark.parametrize("value", [3, -1, 32767, 1 << 16, (1 << 16) + 1, -(1 << 16), 1 << 32])
def test_values_that_do_not_fit_are_refused_and_not_cut(field, value):
    kw = dict(max_batch=2, max_seq=512, max_K=1)
    try:
        cfg = mt.make_cfg(4, 64, 4, 4, 16, 172, 256, **kw, **{field: value})
    except mt.MtError as e:
        assert e.code == mt.MT_ERR_ARG
    else:
        assert mt.mt_required_budget(cfg) == 0
