"""Rotary positions with several axes over the numbers of head slots that a
call may take: less than a wave of threads, one wave, a wave and a half, more
tokens than a wave; slots that do not divide the heads; with V and elements
that are only copied, for every access width, both directions.  The formula in
64 bits, on the GPU; tolerance as in tests/test_gpu_rope.py, and 2^-40 for the
frequency's own rounding (2^-53) over 2^13 positions."""
import numpy as np
import pytest
import torch

from sparse_mask_transformer_gb300 import stof
from tests.test_gpu_rope import HALF, frequencies, rand
from tests.test_gpu_rope_axes import axes_of

pytestmark = pytest.mark.gpu

WIDTHS = [(16, 16, False), (24, 16, False), (8, 8, True), (24, 8, True),  # (d, rot, interleaved): 16 bytes an access
          (8, 8, False), (20, 8, False), (12, 4, True),                   # 8
          (2, 2, False), (14, 2, True)]                                   # 2


def check(got, x, pos, axis, w, interleaved, sign=1.0):
    rot, x = 2 * len(axis), x.double()
    ang = sign * pos[torch.tensor(axis, device="cuda")].permute(1, 2, 0)[:, None].double() * torch.tensor(w, device="cuda")
    c, s = ang.cos(), ang.sin()
    a, b = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
    want, scale = x.clone(), torch.zeros_like(x)
    want[..., a] = x[..., a] * c - x[..., b] * s
    want[..., b] = x[..., b] * c + x[..., a] * s
    scale[..., a] = scale[..., b] = x[..., a].abs() + x[..., b].abs()
    err = (got.double() - want).abs()
    tol = HALF[got.dtype] * want.abs() * (1 + 2.0 ** -6) + (2.0 ** -20 + 2.0 ** -40) * scale + 2.0 ** -25
    assert bool((err <= tol).all()), float(err.max())


@pytest.mark.parametrize("waves", [0.05, 0.3, 0.45, 0.6, 0.95, 1.6])
@pytest.mark.parametrize("d,rot,interleaved", WIDTHS)
def test_slots(gpu_lib, waves, d, rot, interleaved):
    H, Hkv, n, dtype = 5, 2, 2, torch.bfloat16
    threads = 1024 * torch.cuda.get_device_properties(0).multi_processor_count  # of one wave
    wide = d % 8 == 0 and rot % (8 if interleaved else 16) == 0
    pairs = (8 if wide else 4 if d % 4 == 0 else 1) // (2 if interleaved and d % 4 == 0 else 1)
    T = int(waves * threads) * pairs // (rot // 2)
    axis, w = axes_of(n, rot // 2, "turns"), frequencies(rot)
    pos = torch.randint(-2 ** 13, 2 ** 13, (n, 1, T), generator=torch.Generator().manual_seed(T), dtype=torch.int32).cuda()
    axes = stof.stof_rope_axes_init(stof.stof_rope_plan_init(rot, interleaved=interleaved), n, axis)
    packed = rand((1, T, H + 2 * Hkv, d), dtype, 31)
    q, k, v = (t.transpose(1, 2) for t in packed.split([H, Hkv, Hkv], dim=2))
    buf = torch.full((packed.numel() + 64,), 7.0, dtype=dtype, device="cuda")
    out = [b.view(1, h, T, d) for b, h in zip(buf[:-64].split([q.numel(), k.numel(), v.numel()]), (H, Hkv, Hkv))]
    stof.stof_rope_axes_fwd(axes, q, k, v, *out, pos)
    for x, y in ((q, out[0]), (k, out[1])):
        check(y, x, pos, axis, w, interleaved)
    assert torch.equal(out[2], v) and torch.all(buf[-64:] == 7.0)
    grad = torch.full_like(packed, float("nan"))
    back = [t.transpose(1, 2) for t in grad.split([H, Hkv, Hkv], dim=2)]
    stof.stof_rope_axes_bwd(axes, *out, *back, pos)
    for x, y in ((out[0], back[0]), (out[1], back[1])):
        check(y, x, pos, axis, w, interleaved, sign=-1.0)
    assert torch.equal(back[2], v)


@pytest.mark.parametrize("T,H,Hkv,d,rot,dtype", [(9805, 16, 16, 64, 64, torch.float16), (16384, 24, 8, 80, 80, torch.bfloat16),
                                                 (1500, 16, 16, 72, 72, torch.bfloat16), (1000, 32, 8, 128, 64, torch.float16),
                                                 (6000, 9, 3, 80, 40, torch.bfloat16)])
def test_heads_that_the_slots_do_not_divide(gpu_lib, T, H, Hkv, d, rot, dtype):
    n = 3
    axis, w = axes_of(n, rot // 2, "blocks"), frequencies(rot)
    pos = torch.tensor(np.random.default_rng(T).integers(0, 5000, (n, 1, T)), dtype=torch.int32, device="cuda")
    axes = stof.stof_rope_axes_init(stof.stof_rope_plan_init(rot), n, axis)
    q, k, v = (rand((1, h, T, d), dtype, 32 + i) for i, h in enumerate((H, Hkv, Hkv)))
    out = [torch.full_like(t, float("nan")) for t in (q, k, v)]
    stof.stof_rope_axes_fwd(axes, q, k, v, *out, pos)
    for x, y in ((q, out[0]), (k, out[1])):
        check(y, x, pos, axis, w, False)
    assert torch.equal(out[2], v)
