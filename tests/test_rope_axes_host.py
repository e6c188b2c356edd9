"""Rotary positions with several axes on the host: what stof_rope_axes_init
fills, and the refusals of structs and calls (before any launch, so no GPU is
needed)."""
import ctypes
import os
import struct
import subprocess

import pytest
import torch

from sparse_mask_transformer_gb300 import build as stof_build
from sparse_mask_transformer_gb300 import stof

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 1 << 20  # never dereferenced


@pytest.fixture(scope="module")
def lib():
    stof_build.build()
    return stof.load_library()


def test_the_struct_keeps_the_plan_and_the_axes(lib):
    plan = stof.stof_rope_plan_init(12, theta=100.0, interleaved=True, amplitude=1.5)
    axes = stof.stof_rope_axes_init(plan, 3, [0, 1, 2, 2, 1, 0])
    assert (axes.made, axes.n_axes, list(axes.axis[:6])) == (1, 3, [0, 1, 2, 2, 1, 0])
    assert bytes(axes.turn) == bytes(plan)


def test_structs_match_the_header(tmp_path):
    src = tmp_path / "layout.c"
    structs = {"stof_rope_axes": stof.stof_rope_axes, "stof_caches": stof.stof_caches}
    lines = [f'  printf("{n}.{f} %zu\\n", offsetof({n}, {f}));' for n, c in structs.items() for f, _ in c._fields_]
    lines += [f'  printf("{n} %zu\\n", sizeof({n}));' for n in structs]
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "stof.h"\nint main(void) {\n' + "\n".join(lines) + "\n  return 0;\n}\n")
    exe = tmp_path / "layout"
    subprocess.check_call(["gcc", "-std=c11", f"-I{os.path.join(ROOT, 'include')}", str(src), "-o", str(exe)])
    got = dict(ln.split() for ln in subprocess.check_output([str(exe)], text=True).splitlines())
    for name, cls in structs.items():
        assert int(got[name]) == ctypes.sizeof(cls), name
        for field, _ in cls._fields_:
            assert int(got[f"{name}.{field}"]) == getattr(cls, field).offset, (name, field)


@pytest.mark.parametrize("n_axes,axis,status", [
    (0, [0] * 4, stof.STOF_ERR_INVALID_ARG), (5, [0] * 4, stof.STOF_ERR_UNSUPPORTED),
    (2, [0, 1, 2, 0], stof.STOF_ERR_INVALID_ARG), (2, [0, 1, -1, 0], stof.STOF_ERR_INVALID_ARG),
    (2, [0, 1, 0], stof.STOF_ERR_SHAPE), (2, [0, 1, 0, 1, 0], stof.STOF_ERR_SHAPE)])
def test_bad_axes_are_refused(lib, n_axes, axis, status):
    with pytest.raises(stof.StofError) as e:
        stof.stof_rope_axes_init(stof.stof_rope_plan_init(8), n_axes, axis)
    assert e.value.status == status


def test_a_plan_that_was_not_made_is_refused(lib):
    axis = (ctypes.c_int32 * 4)(0, 0, 1, 1)
    axes = stof.stof_rope_axes()
    assert lib.stof_rope_axes_init(ctypes.byref(axes), ctypes.byref(stof.stof_rope_plan()), 2, axis) == stof.STOF_ERR_INVALID_ARG
    assert axes.made == 0
    plan = stof.stof_rope_plan_init(8)
    assert lib.stof_rope_axes_init(ctypes.byref(axes), ctypes.byref(plan), 2, None) == stof.STOF_ERR_INVALID_ARG
    assert lib.stof_rope_axes_init(None, ctypes.byref(plan), 2, axis) == stof.STOF_ERR_INVALID_ARG


def _call(lib, axes, bwd=False, data=FAKE, out=FAKE, dt=1, B=1, H=2, T=4, d=16, positions=FAKE, counts=None):
    x = struct.pack("24q", *(data, 64, 16, 16), *([0] * 8), *(out, 64, 16, 16), *([0] * 8))
    if bwd:
        return lib.stof_rope_axes_bwd(axes, x, dt, B, H, 0, T, d, positions, counts, None)
    return lib.stof_rope_axes_fwd(axes, x, dt, B, H, 0, T, d, positions, counts, None, T, None, None)


@pytest.mark.parametrize("bwd", [False, True])
def test_bad_calls_are_refused(lib, bwd):
    axes = stof.stof_rope_axes_init(stof.stof_rope_plan_init(8), 2, [0, 1, 0, 1])
    assert _call(lib, stof.stof_rope_axes(), bwd) == stof.STOF_ERR_INVALID_ARG
    assert _call(lib, None, bwd) == stof.STOF_ERR_INVALID_ARG
    assert _call(lib, axes, bwd, positions=None) == stof.STOF_ERR_INVALID_ARG
    assert _call(lib, axes, bwd, positions=FAKE + 2) == stof.STOF_ERR_ALIGNMENT
    assert _call(lib, axes, bwd, data=FAKE + 1) == stof.STOF_ERR_ALIGNMENT
    assert _call(lib, axes, bwd, dt=3) == stof.STOF_ERR_DTYPE
    assert _call(lib, axes, bwd, d=6) == stof.STOF_ERR_SHAPE
    assert _call(lib, axes, bwd, d=258) == stof.STOF_ERR_UNSUPPORTED
    assert _call(lib, axes, bwd, out=0) == stof.STOF_ERR_INVALID_ARG
    assert _call(lib, axes, bwd, B=-1) == stof.STOF_ERR_INVALID_ARG
    assert _call(lib, axes, bwd, T=0, positions=None) == stof.STOF_OK  # nothing to do
    broken = stof.stof_rope_axes_init(stof.stof_rope_plan_init(8), 2, [0, 1, 0, 1])
    broken.axis[3] = 2
    assert _call(lib, broken, bwd) == stof.STOF_ERR_INVALID_ARG


def test_binding_refuses_host_tensors(lib):
    axes = stof.stof_rope_axes_init(stof.stof_rope_plan_init(8), 2, [0, 1, 0, 1])
    q = torch.zeros(1, 2, 4, 8, dtype=torch.float16)
    with pytest.raises(stof.StofError) as e:
        stof.stof_rope_axes_fwd(axes, q, None, None, q, None, None, torch.zeros(2, 1, 4, dtype=torch.int32))
    assert e.value.status == stof.STOF_ERR_INVALID_ARG
