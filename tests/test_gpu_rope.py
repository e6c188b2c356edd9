"""Rotary positions (stof_rope_fwd, stof_rope_bwd) against the formula in 64
bits: layouts, partly turned heads, scalings, far positions, packed and
in-place tensors, cache rows, ragged requests, and the gradient.

Tolerance: the output's one rounding (half a step of the type) and the fp32
angle and products: the reduced angle is rounded once (2^-24 of half a turn,
below 2^-22 rad), cosine, sine, amplitude and the two products by a few
2^-24, so an element is off by at most 2^-20 amplitude (|x_a| + |x_c|)
beside its rounding; fp16's smallest steps add 2^-25."""
import math

import numpy as np
import pytest
import torch

from sparse_mask_transformer_gb300 import stof

pytestmark = pytest.mark.gpu
HALF = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}


def frequencies(rot, theta=10000.0):
    return np.array([theta ** (-2 * p / rot) for p in range(rot // 2)])


def turned(x, pos, w, rot, interleaved, amplitude=1.0, sign=1.0):
    """x [B, H, T, d] in 64 bits turned at pos [B, T]; and the error scale of every element."""
    y, scale = x.copy(), np.zeros_like(x)
    ang = sign * pos[:, None, :, None].astype(np.float64) * w
    c, s = np.cos(ang), np.sin(ang)
    a, b = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
    y[..., a] = amplitude * (x[..., a] * c - x[..., b] * s)
    y[..., b] = amplitude * (x[..., b] * c + x[..., a] * s)
    scale[..., a] = scale[..., b] = abs(amplitude) * (np.abs(x[..., a]) + np.abs(x[..., b]))
    return y, scale


def check(got, want, scale, dtype, extra=0.0):
    g = got.double().cpu().numpy()
    err = np.abs(g - want)
    assert np.all(err <= HALF[dtype] * np.abs(want) * (1 + 2.0 ** -6) + (2.0 ** -20 + extra) * scale + 2.0 ** -25), err.max()


def f64(t):
    return t.double().cpu().numpy()


def rand(shape, dtype, seed):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("d,rot", [(32, 32), (64, 64), (64, 32), (128, 128), (256, 256), (128, 96), (64, 20), (80, 40),
                                   (6, 2), (62, 24)])
def test_layouts_and_sizes(gpu_lib, dtype, interleaved, d, rot):
    B, H, Hkv, T = 2, 6, 2, 37
    q, k, v = rand((B, H, T, d), dtype, 1), rand((B, Hkv, T, d), dtype, 2), rand((B, Hkv, T, d), dtype, 3)
    out = [torch.full_like(t, float("nan")) for t in (q, k, v)]
    plan = stof.stof_rope_plan_init(rot, interleaved=interleaved, amplitude=1.5)
    stof.stof_rope_fwd(plan, q, k, v, *out)
    pos = np.tile(np.arange(T), (B, 1))
    for x, y in ((q, out[0]), (k, out[1])):
        check(y, *turned(f64(x), pos, frequencies(rot), rot, interleaved, 1.5), dtype)
    assert torch.equal(out[2], v)


@pytest.mark.parametrize("T,B,H,Hkv", [(1, 1, 1, 1), (1, 16, 32, 8), (1, 1, 0, 3), (3, 5, 7, 0), (1237, 1, 12, 4), (700, 24, 16, 16)])
def test_batch_shapes(gpu_lib, T, B, H, Hkv):
    """From one token to enough of them that a thread owns all heads of its pairs."""
    d, dtype = 64, torch.bfloat16
    plan = stof.stof_rope_plan_init(d)
    q = rand((B, H, T, d), dtype, 4) if H else None
    k = rand((B, Hkv, T, d), dtype, 5) if Hkv else None
    qo, ko = (None if t is None else torch.empty_like(t) for t in (q, k))
    stof.stof_rope_fwd(plan, q, k, None, qo, ko, None)
    pos = np.tile(np.arange(T), (B, 1))
    for x, y in ((q, qo), (k, ko)):
        if x is not None:
            check(y, *turned(f64(x), pos, frequencies(d), d, False), dtype)


def test_far_and_negative_positions(gpu_lib):
    d, T, dtype = 128, 64, torch.float16
    rng = np.random.default_rng(0)
    pos = np.concatenate([rng.integers(-2 ** 31, 2 ** 31, T - 6), [0, 1, -1, 2 ** 31 - 1, -2 ** 31, 10 ** 7]])[None]
    q = rand((1, 3, T, d), dtype, 6)
    o = torch.empty_like(q)
    plan = stof.stof_rope_plan_init(d, theta=500000.0)
    stof.stof_rope_fwd(plan, q, None, None, o, None, None, positions=torch.tensor(pos, dtype=torch.int32, device="cuda"))
    # the definition's own 64-bit angle: position * w rounded to 2^-53 of up to 2^31 rad, and w itself on both sides
    check(o, *turned(f64(q), pos, frequencies(d, 500000.0), d, False), dtype, extra=4 * 2.0 ** -53 * 2.0 ** 31)


@pytest.mark.parametrize("d,rot", [(128, 128), (64, 32), (20, 10)])
def test_packed_projection_and_in_place(gpu_lib, d, rot):
    B, H, Hkv, T, dtype = 2, 4, 2, 50, torch.bfloat16
    packed = rand((B, T, H + 2 * Hkv, d), dtype, 7)
    before = packed.clone()
    q, k, v = (t.transpose(1, 2) for t in packed.split([H, Hkv, Hkv], dim=2))
    out = [torch.empty(B, h, T, d, dtype=dtype, device="cuda") for h in (H, Hkv, Hkv)]
    plan = stof.stof_rope_plan_init(rot)
    stof.stof_rope_fwd(plan, q, k, v, *out)
    assert torch.equal(packed, before)
    pos = np.tile(np.arange(T), (B, 1))
    for x, y in ((q, out[0]), (k, out[1])):
        check(y, *turned(f64(x), pos, frequencies(rot), rot, False), dtype)
    assert torch.equal(out[2], v)
    stof.stof_rope_fwd(plan, q, k, v, q, k, v)  # in place
    assert torch.equal(q, out[0]) and torch.equal(k, out[1]) and torch.equal(v, out[2])


@pytest.mark.parametrize("d", [64, 22])
def test_odd_offsets_take_the_narrow_path(gpu_lib, d):
    """Rows that start off a 16-byte boundary give the same values."""
    B, H, T, dtype = 1, 2, 9, torch.float16
    x = rand((B, H, T, d), dtype, 8)
    buf = torch.zeros(B * H * T * (d + 1) + 1, dtype=dtype, device="cuda")
    odd = buf[1:].as_strided((B, H, T, d), (H * T * (d + 1), T * (d + 1), d + 1, 1))
    odd.copy_(x)
    a, b = torch.empty_like(x), torch.empty_like(x)
    plan = stof.stof_rope_plan_init(d if d == 64 else 16)
    stof.stof_rope_fwd(plan, x, None, None, a, None, None)
    stof.stof_rope_fwd(plan, odd, None, None, b, None, None)
    assert torch.equal(a, b)


def test_cache_rows_and_ragged_requests(gpu_lib):
    B, H, Hkv, T, d, cap, dtype = 4, 4, 2, 5, 128, 40, torch.bfloat16
    q, k, v = rand((B, H, T, d), dtype, 1), rand((B, Hkv, T, d), dtype, 2), rand((B, Hkv, T, d), dtype, 3)
    caches = [rand((B, Hkv, cap, d), dtype, s) for s in (4, 5)]
    old = [c.clone() for c in caches]
    qo = torch.full_like(q, 7.0)
    rows, counts = [0, 35, 17, 20], [5, 5, 0, 3]
    plan = stof.stof_rope_plan_init(d)
    err = torch.zeros(1, dtype=torch.int64, device="cuda")
    stof.stof_rope_fwd(plan, q, k, v, qo, *caches, rows=torch.tensor(rows, dtype=torch.int32, device="cuda"),
                       counts=torch.tensor(counts, dtype=torch.int32, device="cuda"), device_error=err)
    assert err.item() == 0
    pos = np.array(rows)[:, None] + np.arange(T)[None, :]
    wq, sq = turned(f64(q), pos, frequencies(d), d, False)
    wk, sk = turned(f64(k), pos, frequencies(d), d, False)
    for b in range(B):
        n, r = counts[b], rows[b]
        check(qo[b, :, :n], wq[b, :, :n], sq[b, :, :n], dtype)
        assert torch.all(qo[b, :, n:] == 7.0)
        check(caches[0][b, :, r:r + n], wk[b, :, :n], sk[b, :, :n], dtype)
        assert torch.equal(caches[1][b, :, r:r + n], v[b, :, :n])
        for c, o in zip(caches, old):
            assert torch.equal(c[b, :, :r], o[b, :, :r]) and torch.equal(c[b, :, r + n:], o[b, :, r + n:])


def test_rows_outside_the_cache_are_skipped_and_reported(gpu_lib):
    B, Hkv, T, d, cap, dtype = 3, 2, 4, 64, 10, torch.float16
    k = rand((B, Hkv, T, d), dtype, 2)
    guard = torch.full((B, Hkv, cap + 8, d), 3.0, dtype=dtype, device="cuda")
    cache = guard[:, :, 4:4 + cap]
    rows = torch.tensor([-2, 8, 2], dtype=torch.int32, device="cuda")
    err = torch.zeros(1, dtype=torch.int64, device="cuda")
    stof.stof_rope_fwd(stof.stof_rope_plan_init(d), None, k, None, None, cache, None, rows=rows, device_error=err)
    assert err.item() == stof.STOF_DEVERR_BAD_LENGTH
    assert torch.all(guard[:, :, :4] == 3.0) and torch.all(guard[:, :, 4 + cap:] == 3.0)
    w, s = turned(f64(k), np.array([-2, 8, 2])[:, None] + np.arange(T), frequencies(d), d, False)
    check(cache[0, :, 0:2], w[0, :, 2:], s[0, :, 2:], dtype)   # rows -2 and -1 skipped
    check(cache[1, :, 8:10], w[1, :, :2], s[1, :, :2], dtype)  # rows 10 and 11 skipped
    check(cache[2, :, 2:6], w[2], s[2], dtype)
    assert torch.all(cache[0, :, 2:] == 3.0) and torch.all(cache[1, :, :8] == 3.0)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rot", [64, 32])
def test_gradient_is_the_formulas_and_the_differences(gpu_lib, interleaved, rot):
    B, H, T, d, dtype, amp = 1, 2, 11, 64, torch.bfloat16, 1.25
    plan = stof.stof_rope_plan_init(rot, interleaved=interleaved, amplitude=amp)
    g = rand((B, H, T, d), dtype, 9)
    pos = np.arange(100, 100 + T)[None]
    p = torch.tensor(pos, dtype=torch.int32, device="cuda")
    grads = torch.empty(B, T, 3 * H, d, dtype=dtype, device="cuda")
    out = [t.transpose(1, 2) for t in grads.split([H, H, H], dim=2)]
    stof.stof_rope_bwd(plan, g, g, g, *out, positions=p)
    want, scale = turned(f64(g), pos, frequencies(rot), rot, interleaved, amp, sign=-1.0)
    check(out[0], want, scale, dtype)
    assert torch.equal(out[0], out[1]) and torch.equal(out[2], g)
    # central differences of <g, rope(x)> in 64 bits (the function is linear: exact up to rounding)
    x = np.random.default_rng(1).standard_normal((B, H, T, d))
    w = frequencies(rot)
    for idx in [(0, 0, 0, 0), (0, 1, 5, 17), (0, 1, 10, 40), (0, 0, 3, 63)]:
        e = np.zeros_like(x)
        e[idx] = 1.0
        diff = (np.sum(f64(g) * (turned(x + e, pos, w, rot, interleaved, amp)[0] - turned(x - e, pos, w, rot, interleaved, amp)[0]))) / 2
        assert abs(float(out[0][idx]) - diff) <= 2.0 ** -8 * abs(diff) * 1.01 + 2.0 ** -20 * scale[idx] + 1e-12


def test_graph_replay_and_streams(gpu_lib):
    """Captured and replayed on changed inputs and positions; two calls on two streams."""
    B, H, T, d, dtype = 2, 4, 3, 128, torch.bfloat16
    plan = stof.stof_rope_plan_init(d)
    q, o = rand((B, H, T, d), dtype, 1), torch.empty(B, H, T, d, dtype=dtype, device="cuda")
    pos = torch.zeros(B, T, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        stof.stof_rope_fwd(plan, q, None, None, o, None, None, positions=pos)
    for seed in (2, 3):
        q.copy_(rand((B, H, T, d), dtype, seed))
        pos.copy_(torch.arange(seed, seed + B * T, dtype=torch.int32).view(B, T))
        graph.replay()
        want = torch.empty_like(o)
        stof.stof_rope_fwd(plan, q, None, None, want, None, None, positions=pos)
        torch.cuda.synchronize()
        assert torch.equal(o, want)
    streams, outs = [torch.cuda.Stream() for _ in range(2)], [torch.empty_like(o) for _ in range(2)]
    for s, y in zip(streams, outs):
        s.wait_stream(torch.cuda.current_stream())
        stof.stof_rope_fwd(plan, q, None, None, y, None, None, positions=pos, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], o) and torch.equal(outs[1], o)


@pytest.mark.parametrize("d,rot", [(64, 64), (6, 2)])
def test_head_counts_that_nothing_divides(gpu_lib, d, rot):
    """Head slots need not divide the heads: one slot per head would be the only divisor."""
    B, H, Hkv, T, dtype = 3, 60, 1, 401, torch.float16
    plan = stof.stof_rope_plan_init(rot)
    q, k = rand((B, H, T, d), dtype, 30), rand((B, Hkv, T, d), dtype, 31)
    qo, ko = torch.full_like(q, float("nan")), torch.full_like(k, float("nan"))
    stof.stof_rope_fwd(plan, q, k, None, qo, ko, None)
    pos = np.tile(np.arange(T), (B, 1))
    for x, y in ((q, qo), (k, ko)):
        check(y, *turned(f64(x), pos, frequencies(rot), rot, False), dtype)
