"""fp16 rows whose softmax reference is far below 0 in some part of their keys:
scores of 2^26 to 2^30 (log2 units) are 8 to 128 apart at least, and a reference
is raised by their difference, not by a comparison in fp32 at that size (8 added
to -2^27 rounds to 16 more: P would be 2^16, past fp16).  Against the definition
in 64 bits (tests/scored_reference.py derives the tolerance)."""
import numpy as np
import pytest
import torch

from sparse_mask_transformer_gb300 import stof
from tests.conftest import gpu_encode
from tests.scored_reference import attend, default_scale, f64

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("far", [2_000_000_000, -2_000_000_000, 1_200_000_000, -800_000_000])
@pytest.mark.parametrize("softcap", [0.0, 30.0])
@pytest.mark.parametrize("d,H,T", [(64, 2, 3), (64, 10, 5), (64, 33, 9), (128, 2, 3), (128, 33, 9)])
def test_committed_keys_far_from_the_drafted_ones(gpu_lib, d, H, T, softcap, far):
    """A drafted token sees itself and the tokens before it; the shares of the cache that hold committed keys alone have
    only scores near -2^27.2, a few steps of 16 apart."""
    n, dtype = 90_000, torch.float16
    slopes = np.linspace(0.05, 0.09, H) * 2e9 / abs(far)
    g = torch.Generator().manual_seed(d + H)
    q = (torch.randn(1, H, T, d, generator=g) * 4).to(dtype)
    k, v = (torch.randn(1, 1, n + T, d, generator=g).to(dtype) for _ in range(2))
    positions = torch.tensor([[far + t for t in range(T)]], dtype=torch.int32, device="cuda")
    o = torch.full_like(q, 5.0).cuda()
    ws = torch.empty(stof.stof_tree_attn_workspace_bytes(1, H, 1, T, d), dtype=torch.uint8, device="cuda")
    score = stof.Score(softcap, torch.tensor(slopes, dtype=torch.float32, device="cuda"))
    stof.stof_tree_attn_fwd(q.cuda(), k.cuda(), v.cuda(), torch.tensor([n], dtype=torch.int32, device="cuda"), default_scale(d),
                            o, ws, positions=positions, score=score)
    assert torch.isfinite(o.float()).all()
    # the committed keys' weights are below 2^-10^7: the drafted ones alone decide
    valid = np.tril(np.ones((T, T), dtype=bool))
    dist = np.abs(np.arange(T)[:, None] - np.arange(T)[None, :]).astype(np.float64)
    for h in range(H):
        want, tol = attend(f64(q[0, h]), f64(k[0, 0, n:]), f64(v[0, 0, n:]), valid, dist, default_scale(d), softcap,
                           float(np.float32(slopes[h])), dtype)
        assert np.all(np.abs(f64(o[0, h]) - want) <= tol)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("L", [300, 2500])
def test_steep_slopes(gpu_lib, d, L):
    """Slopes of 2^20: rows whose nearest visible keys are some 100 away on both sides have two of them, with equal scores
    but for q.k, which such distances round away."""
    dtype, H = torch.float16, 2
    masks = np.zeros((1, L, L), dtype=np.uint8)
    i = np.arange(L)
    masks[0] = np.abs(i[:, None] - i[None, :]) >= 97
    g = torch.Generator().manual_seed(d)
    q = torch.randn(1, H, L, d, generator=g).to(dtype)
    k = torch.randn(1, 1, L, d, generator=g).to(dtype)
    v = torch.rand(1, 1, L, d, generator=g).to(dtype)
    fmt, ws, _ = gpu_encode(torch.from_numpy(masks).cuda(), 128, 128)
    o = torch.empty_like(q).cuda()
    score = stof.Score(0.0, torch.full((H,), 2.0 ** 20, device="cuda"))
    stof.stof_mha_fwd_score(q.cuda(), k.cuda(), v.cuda(), fmt, default_scale(d), score, 0, 0, stof.STOF_KERNEL_BLOCKWISE, o)
    assert torch.isfinite(o.float()).all()
    got, vv = f64(o[0, 0]), f64(v[0, 0])
    for r in range(97, L - 97, 31):                      # between the two nearest keys' V, up to a rounding of P and one of O
        lo, hi = np.minimum(vv[r - 97], vv[r + 97]), np.maximum(vv[r - 97], vv[r + 97])
        assert np.all(got[r] >= lo * (1 - 2.0 ** -9)) and np.all(got[r] <= hi * (1 + 2.0 ** -9))
