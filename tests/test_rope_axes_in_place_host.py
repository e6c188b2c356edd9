"""stof_rope_axes_init on a struct that holds the plan itself (no GPU)."""
import ctypes

from sparse_mask_transformer_gb300 import stof
from tests.test_rope_axes_host import lib  # noqa: F401 (fixture)


def test_axes_are_filled_from_their_own_plan(lib):  # noqa: F811
    plan = stof.stof_rope_plan_init(12, theta=100.0, amplitude=1.5)
    axes = stof.stof_rope_axes_init(plan, 2, [0, 1, 0, 1, 0, 1])
    axis = (ctypes.c_int32 * 6)(2, 2, 1, 1, 0, 0)
    # (turn is the struct's first member)
    own = ctypes.cast(ctypes.pointer(axes), ctypes.POINTER(stof.stof_rope_plan))
    assert lib.stof_rope_axes_init(ctypes.byref(axes), own, 3, axis) == stof.STOF_OK
    assert (axes.made, axes.n_axes, list(axes.axis[:6])) == (1, 3, [2, 2, 1, 1, 0, 0])
    assert bytes(axes.turn) == bytes(plan)
