"""Rotary positions with several axes (stof_rope_axes_fwd, stof_rope_axes_bwd)
against the formula in 64 bits: orders and numbers of axes, head sizes of
every access width, grids of tokens, packed and in-place tensors, cache rows,
ragged requests, the gradient.  Tolerance as for one axis
(tests/test_gpu_rope.py): the output's rounding, 2^-20 (|x_a| + |x_c|) for the
fp32 angle and products, fp16's smallest steps."""
import numpy as np
import pytest
import torch

from sparse_mask_transformer_gb300 import stof
from tests.test_gpu_rope import check, f64, frequencies, rand

pytestmark = pytest.mark.gpu


def axes_of(n_axes, pairs, order):
    if order == "blocks":
        return [min(p * n_axes // pairs, n_axes - 1) for p in range(pairs)]
    return [p % n_axes for p in range(pairs)]


def turned(x, pos, axis, w, interleaved, sign=1.0):
    """x [B, H, T, d] in 64 bits turned at pos [axes, B, T]; and the error scale of every element."""
    rot = 2 * len(axis)
    y, scale = x.copy(), np.zeros_like(x)
    ang = sign * np.stack([pos[a] for a in axis], axis=-1)[:, None].astype(np.float64) * w  # [B, 1, T, pairs]
    c, s = np.cos(ang), np.sin(ang)
    a, b = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    scale[..., a] = scale[..., b] = np.abs(x[..., a]) + np.abs(x[..., b])
    return y, scale


def grid(n_axes, B, T, seed=0):
    """Positions of frames of 3 x 5 tokens behind some text."""
    t = np.arange(T)
    at = [t // 15, t // 5 % 3, t % 5, t][:n_axes]
    return np.random.default_rng(seed).integers(0, 900, (1, B, 1)) + np.stack(at)[:, None, :]


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("d,rot", [(32, 32), (64, 64), (128, 128), (256, 256), (128, 96),  # 16 bytes an access
                                   (72, 72), (80, 40), (60, 24), (12, 8),                  # 8 bytes
                                   (64, 20), (6, 2), (62, 24)])                            # 2
def test_layouts_and_sizes(gpu_lib, dtype, interleaved, d, rot):
    B, H, Hkv, T, n = 2, 6, 2, 37, 3
    q, k, v = rand((B, H, T, d), dtype, 1), rand((B, Hkv, T, d), dtype, 2), rand((B, Hkv, T, d), dtype, 3)
    out = [torch.full_like(t, float("nan")) for t in (q, k, v)]
    axis, pos = axes_of(n, rot // 2, "blocks" if d % 64 else "turns"), grid(n, B, T)
    axes = stof.stof_rope_axes_init(stof.stof_rope_plan_init(rot, interleaved=interleaved), n, axis)
    stof.stof_rope_axes_fwd(axes, q, k, v, *out, i32(pos))
    for x, y in ((q, out[0]), (k, out[1])):
        check(y, *turned(f64(x), pos, axis, frequencies(rot), interleaved), dtype)
    assert torch.equal(out[2], v)


@pytest.mark.parametrize("n_axes", [1, 2, 4])
@pytest.mark.parametrize("order", ["blocks", "turns"])
def test_numbers_of_axes(gpu_lib, n_axes, order):
    B, H, T, d, dtype = 3, 5, 64, 64, torch.bfloat16
    axis, pos = axes_of(n_axes, d // 2, order), grid(n_axes, B, T, seed=n_axes)
    q = rand((B, H, T, d), dtype, 4)
    o = torch.empty_like(q)
    axes = stof.stof_rope_axes_init(stof.stof_rope_plan_init(d), n_axes, axis)
    stof.stof_rope_axes_fwd(axes, q, None, None, o, None, None, i32(pos))
    check(o, *turned(f64(q), pos, axis, frequencies(d), False), dtype)


def test_equal_positions_are_one_axis_bit_for_bit(gpu_lib):
    B, H, Hkv, T, d = 2, 8, 2, 133, 128
    q, k = rand((B, H, T, d), torch.bfloat16, 5), rand((B, Hkv, T, d), torch.bfloat16, 6)
    plan = stof.stof_rope_plan_init(d, theta=500000.0, amplitude=1.25)
    pos = i32(np.random.default_rng(1).integers(-2 ** 31, 2 ** 31, (B, T)))
    one, many = [torch.empty_like(t) for t in (q, k)], [torch.empty_like(t) for t in (q, k)]
    stof.stof_rope_fwd(plan, q, k, None, *one, None, positions=pos)
    stof.stof_rope_axes_fwd(stof.stof_rope_axes_init(plan, 3, axes_of(3, 64, "turns")), q, k, None, *many, None,
                            pos[None].repeat(3, 1, 1).contiguous())
    assert torch.equal(one[0], many[0]) and torch.equal(one[1], many[1])


@pytest.mark.parametrize("T,B,H,Hkv", [(1, 1, 1, 1), (1, 16, 32, 8), (1, 1, 0, 3), (3, 5, 7, 0), (1237, 1, 12, 4), (700, 24, 16, 16)])
def test_batch_shapes_with_frequencies_of_each_axis(gpu_lib, T, B, H, Hkv):
    d, dtype, n = 64, torch.bfloat16, 2
    axis = axes_of(n, d // 2, "blocks")
    w = np.concatenate([100.0 ** (-np.arange(16) / 16)] * 2)
    axes = stof.stof_rope_axes_init(stof.stof_rope_plan_custom(w), n, axis)
    q = rand((B, H, T, d), dtype, 7) if H else None
    k = rand((B, Hkv, T, d), dtype, 8) if Hkv else None
    qo, ko = (None if t is None else torch.empty_like(t) for t in (q, k))
    pos = grid(n, B, T)
    stof.stof_rope_axes_fwd(axes, q, k, None, qo, ko, None, i32(pos))
    for x, y in ((q, qo), (k, ko)):
        if x is not None:
            check(y, *turned(f64(x), pos, axis, w, False), dtype, extra=2.0 ** -40)


def test_far_positions(gpu_lib):
    d, T, n = 128, 64, 3
    pos = np.random.default_rng(2).integers(-2 ** 31, 2 ** 31, (n, 1, T))
    axis = axes_of(n, d // 2, "turns")
    q = rand((1, 3, T, d), torch.float16, 9)
    o = torch.empty_like(q)
    axes = stof.stof_rope_axes_init(stof.stof_rope_plan_init(d, theta=500000.0), n, axis)
    stof.stof_rope_axes_fwd(axes, q, None, None, o, None, None, i32(pos))
    # the definition's own 64-bit angle: position * w rounded to 2^-53 of up to 2^31 rad, and w itself on both sides
    check(o, *turned(f64(q), pos, axis, frequencies(d, 500000.0), False), torch.float16, extra=4 * 2.0 ** -53 * 2.0 ** 31)


@pytest.mark.parametrize("d,rot", [(128, 128), (72, 72), (20, 10)])
def test_packed_projection_and_in_place(gpu_lib, d, rot):
    B, H, Hkv, T, n, dtype = 2, 4, 2, 50, 3, torch.bfloat16
    packed = rand((B, T, H + 2 * Hkv, d), dtype, 10)
    before = packed.clone()
    q, k, v = (t.transpose(1, 2) for t in packed.split([H, Hkv, Hkv], dim=2))
    out = [torch.empty(B, h, T, d, dtype=dtype, device="cuda") for h in (H, Hkv, Hkv)]
    axis, pos = axes_of(n, rot // 2, "blocks"), grid(n, B, T)
    axes = stof.stof_rope_axes_init(stof.stof_rope_plan_init(rot), n, axis)
    stof.stof_rope_axes_fwd(axes, q, k, v, *out, i32(pos))
    assert torch.equal(packed, before)
    for x, y in ((q, out[0]), (k, out[1])):
        check(y, *turned(f64(x), pos, axis, frequencies(rot), False), dtype)
    assert torch.equal(out[2], v)
    stof.stof_rope_axes_fwd(axes, q, k, v, q, k, v, i32(pos))  # in place
    assert torch.equal(q, out[0]) and torch.equal(k, out[1]) and torch.equal(v, out[2])


def test_cache_rows_ragged_requests_and_bad_rows(gpu_lib):
    B, H, Hkv, T, d, cap, n = 4, 4, 2, 5, 64, 40, 3
    q, k, v = rand((B, H, T, d), torch.float16, 11), rand((B, Hkv, T, d), torch.float16, 12), rand((B, Hkv, T, d), torch.float16, 13)
    rows, counts = [0, 17, 38, -3], [5, 2, 5, 5]       # request 2 leaves the cache after two rows, 3 begins before it
    kc, vc = (torch.full((B, Hkv, cap, d), 7.0, dtype=torch.float16, device="cuda") for _ in range(2))
    qo = torch.full_like(q, 7.0)
    axis, pos = axes_of(n, d // 2, "turns"), grid(n, B, T)
    axes = stof.stof_rope_axes_init(stof.stof_rope_plan_init(d), n, axis)
    err = torch.zeros(1, dtype=torch.int64, device="cuda")
    stof.stof_rope_axes_fwd(axes, q, k, v, qo, kc, vc, i32(pos), counts=i32(counts), rows=i32(rows), device_error=err)
    assert err.item() == stof.STOF_DEVERR_BAD_LENGTH
    want_q, sq = turned(f64(q), pos, axis, frequencies(d), False)
    want_k, sk = turned(f64(k), pos, axis, frequencies(d), False)
    wk, wv, sc = np.full(kc.shape, 7.0), np.full(vc.shape, 7.0), np.zeros(kc.shape)
    for b in range(B):
        want_q[b, :, counts[b]:], sq[b, :, counts[b]:] = 7.0, 0.0
        for t in range(counts[b]):
            if 0 <= rows[b] + t < cap:
                wk[b, :, rows[b] + t], sc[b, :, rows[b] + t] = want_k[b, :, t], sk[b, :, t]
                wv[b, :, rows[b] + t] = f64(v)[b, :, t]
    check(qo, want_q, sq, torch.float16)
    check(kc, wk, sc, torch.float16)
    assert np.array_equal(f64(vc), wv)


@pytest.mark.parametrize("d,interleaved", [(64, False), (72, False), (64, True)])
def test_gradient_is_the_turn_back_and_matches_differences(gpu_lib, d, interleaved):
    """The gradient by its formula, into a packed gradient; and <grad, e> against the forward pass's own differences:
    the rotation is linear, so <y, g> of an input e is <e, gradient of g>."""
    B, H, Hkv, T, n, dtype = 2, 3, 1, 31, 3, torch.float16
    axis, pos = axes_of(n, d // 2, "blocks"), grid(n, B, T)
    axes = stof.stof_rope_axes_init(stof.stof_rope_plan_init(d, interleaved=interleaved), n, axis)
    g = [rand((B, h, T, d), dtype, 14 + i) for i, h in enumerate((H, Hkv, Hkv))]
    packed = torch.full((B, T, H + 2 * Hkv, d), float("nan"), dtype=dtype, device="cuda")
    out = [t.transpose(1, 2) for t in packed.split([H, Hkv, Hkv], dim=2)]
    stof.stof_rope_axes_bwd(axes, *g, *out, i32(pos))
    for x, y in zip(g[:2], out[:2]):
        check(y, *turned(f64(x), pos, axis, frequencies(d), interleaved, sign=-1.0), dtype)
    assert torch.equal(out[2], g[2])
    e = rand((B, H, T, d), dtype, 20)
    y = torch.empty_like(e)
    stof.stof_rope_axes_fwd(axes, e, None, None, y, None, None, i32(pos))
    a, b = (f64(y) * f64(g[0])).sum(), (f64(e) * f64(out[0])).sum()
    # each side: every term of one rounding (2^-11 and the fp32 error) of y or the gradient
    bound = (2.0 ** -11 + 2.0 ** -19) * ((np.abs(f64(y) * f64(g[0]))).sum() + np.abs(f64(e) * f64(out[0])).sum()) \
        + 2.0 ** -19 * (np.abs(f64(e)).max() * np.abs(f64(g[0])).sum() * 2)
    assert abs(a - b) <= bound


def test_capture_and_streams(gpu_lib):
    B, H, T, d, n = 2, 4, 40, 128, 3
    q = rand((B, H, T, d), torch.bfloat16, 21)
    o, want = torch.empty_like(q), torch.empty_like(q)
    axes = stof.stof_rope_axes_init(stof.stof_rope_plan_init(d), n, axes_of(n, d // 2, "turns"))
    pos = i32(grid(n, B, T))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    stof.stof_rope_axes_fwd(axes, q, None, None, o, None, None, pos, stream=side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        stof.stof_rope_axes_fwd(axes, q, None, None, o, None, None, pos)
    pos.add_(77)
    stof.stof_rope_axes_fwd(axes, q, None, None, want, None, None, pos)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(o, want)


def test_positions_of_another_shape_are_refused(gpu_lib):
    q = rand((2, 4, 6, 64), torch.bfloat16, 22)
    axes = stof.stof_rope_axes_init(stof.stof_rope_plan_init(64), 3, axes_of(3, 32, "turns"))
    for shape in ((2, 2, 6), (3, 2, 7), (2, 6)):
        with pytest.raises(stof.StofError) as e:
            stof.stof_rope_axes_fwd(axes, q, None, None, q, None, None, torch.zeros(shape, dtype=torch.int32, device="cuda"))
        assert e.value.status == stof.STOF_ERR_SHAPE
    with pytest.raises(stof.StofError):
        stof.stof_rope_axes_fwd(axes, q, None, None, q, None, None, None)
