"""Rotary positions on the host: the plan's frequencies against their
definition in exact arithmetic, and the refusals of plans and calls (before
any launch, so no GPU is needed)."""
import ctypes
import math
import struct
from fractions import Fraction

import pytest
import torch

from sparse_mask_transformer_gb300 import build as stof_build
from sparse_mask_transformer_gb300 import stof


@pytest.fixture(scope="module")
def lib():
    stof_build.build()
    return stof.load_library()


def definition(rot, theta, scaling, factor, length, lo, hi):
    out = []
    for p in range(rot // 2):
        w = theta ** (-2 * p / rot)
        if scaling == stof.STOF_ROPE_LINEAR:
            w /= factor
        elif scaling == stof.STOF_ROPE_BY_INDEX:
            def at(n):
                return rot * math.log(length / (n * 2 * math.pi)) / (2 * math.log(theta))
            a, b = max(math.floor(at(hi)), 0), min(math.ceil(at(lo)), rot - 1)
            r = min(max((p - a) / max(b - a, 0.001), 0), 1)
            w = w * (1 - r) + w / factor * r
        elif scaling == stof.STOF_ROPE_BY_TURNS:
            s = min(max((length * w / (2 * math.pi) - lo) / (hi - lo), 0), 1)
            w = w * s + w / factor * (1 - s)
        out.append(w)
    return out


@pytest.mark.parametrize("rot,theta", [(2, 10000.0), (20, 10000.0), (64, 500000.0), (128, 10000.0), (256, 1e6)])
@pytest.mark.parametrize("scaling", [0, 1, 2, 3])
def test_plan_steps_follow_the_definition(lib, rot, theta, scaling):
    plan = stof.stof_rope_plan_init(rot, theta=theta, scaling=scaling, factor=8.0, original_length=4096, turns_lo=1.0,
                                    turns_hi=32.0, amplitude=1.25)
    assert (plan.rot_dim, plan.interleaved, plan.amplitude, plan.made) == (rot, 0, 1.25, 1)
    for p, w in enumerate(definition(rot, theta, scaling, 8.0, 4096, 1.0, 32.0)):
        # double precision on both sides: a few roundings of 2^-53 of the frequency each; and the step is a whole
        # number of 2^-64 turns, cut off: at most 2 pi 2^-64 rad (2^-33 turns at position 2^31)
        assert abs(plan.step[p] / 2.0 ** 64 * 2 * math.pi - w) <= 16 * 2.0 ** -53 * w + 2 * math.pi * 2.0 ** -64, p


def test_custom_frequencies_are_reduced_to_a_turn(lib):
    f = [0.0, 1.0, -1.0, 7.0, 100.0, -0.25, 2 * math.pi]
    plan = stof.stof_rope_plan_custom(f, interleaved=True)
    assert plan.rot_dim == 14 and plan.interleaved == 1
    pi = Fraction(31415926535897932384626433832795028841971, 10 ** 40)
    for p, w in enumerate(f):
        turns = Fraction(w) / (2 * pi)
        err = abs(Fraction(plan.step[p], 2 ** 64) - turns)
        err -= round(err)  # whole turns do not count
        assert abs(err) <= Fraction(max(1.0, abs(w)) * 2.0 ** -52), w


def test_bad_plans_are_refused(lib):
    bad = [dict(rot_dim=0), dict(rot_dim=-2), dict(rot_dim=3), dict(rot_dim=64, theta=1.0),
           dict(rot_dim=64, theta=float("nan")), dict(rot_dim=64, scaling=4), dict(rot_dim=64, scaling=1, factor=0.0),
           dict(rot_dim=64, scaling=2, factor=2.0, original_length=0),
           dict(rot_dim=64, scaling=3, factor=2.0, original_length=8, turns_lo=4.0, turns_hi=4.0),
           dict(rot_dim=64, amplitude=float("inf"))]
    for kw in bad:
        with pytest.raises(stof.StofError) as e:
            stof.stof_rope_plan_init(**kw)
        assert e.value.status == stof.STOF_ERR_INVALID_ARG, kw
    with pytest.raises(stof.StofError) as e:
        stof.stof_rope_plan_init(258)
    assert e.value.status == stof.STOF_ERR_UNSUPPORTED
    for f in ([float("nan")], [float("inf")], []):
        with pytest.raises(stof.StofError):
            stof.stof_rope_plan_custom(f)


FAKE = 1 << 20  # never dereferenced: every call below is refused first


def _call(lib, plan=None, q=True, k=True, v=True, dt=0, B=2, H=4, Hkv=2, T=8, d=64, positions=None, counts=None,
          rows=None, kv_rows=8, q_out=True, k_out=True, v_out=True, data=FAKE, err=None):
    plan = stof.stof_rope_plan_init(64) if plan is None else plan
    row = lambda on: (data or 0, 4096, 512, 64) if on else (0, 0, 0, 0)  # noqa: E731
    x = struct.pack("24q", *row(q), *row(k), *row(v), *row(q_out), *row(k_out), *row(v_out))
    return lib.stof_rope_fwd(ctypes.byref(plan), x, dt, B, H, Hkv, T, d, positions, counts, rows, kv_rows, err, None)


def test_bad_calls_are_refused(lib):
    empty = stof.stof_rope_plan()
    assert _call(lib, plan=empty) == stof.STOF_ERR_INVALID_ARG
    assert _call(lib, dt=7) == stof.STOF_ERR_DTYPE
    assert _call(lib, B=-1) == stof.STOF_ERR_INVALID_ARG
    assert _call(lib, kv_rows=-1) == stof.STOF_ERR_INVALID_ARG
    assert _call(lib, q_out=False) == stof.STOF_ERR_INVALID_ARG
    assert _call(lib, k=False, k_out=False) == stof.STOF_ERR_INVALID_ARG  # v without k
    assert _call(lib, d=63) == stof.STOF_ERR_UNSUPPORTED
    assert _call(lib, d=258) == stof.STOF_ERR_UNSUPPORTED
    assert _call(lib, d=32) == stof.STOF_ERR_SHAPE
    assert lib.stof_rope_fwd(ctypes.byref(stof.stof_rope_plan_init(64)), None, 0, 2, 4, 2, 8, 64, None, None, None, 8, None,
                             None) == stof.STOF_ERR_INVALID_ARG
    assert _call(lib, data=FAKE + 1) == stof.STOF_ERR_ALIGNMENT
    assert _call(lib, positions=FAKE + 2) == stof.STOF_ERR_ALIGNMENT
    assert _call(lib, err=FAKE + 4) == stof.STOF_ERR_ALIGNMENT
    assert _call(lib, B=1 << 20, T=1 << 20) == stof.STOF_ERR_SHAPE
    # nothing to do: no launch
    assert _call(lib, B=0) == stof.STOF_OK
    assert _call(lib, T=0) == stof.STOF_OK
    assert _call(lib, q=False, k=False, v=False, q_out=False, k_out=False, v_out=False) == stof.STOF_OK


def test_binding_refuses_tensors_it_cannot_take(lib):
    plan = stof.stof_rope_plan_init(64)
    x = torch.zeros(1, 2, 4, 64, dtype=torch.float16)
    with pytest.raises(stof.StofError) as e:
        stof.stof_rope_fwd(plan, x, None, None, x, None, None)
    assert e.value.status == stof.STOF_ERR_INVALID_ARG
    with pytest.raises(stof.StofError):
        stof.stof_rope_fwd(plan, None, None, None, None, None, None)
