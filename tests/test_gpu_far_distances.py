"""Scores lowered with distance where every visible key is far from the query
(positions up to 2^31, q_start up to 2^30): neighbouring keys differ by one
slope whatever their distance.  stof_mha_fwd_score on every kernel and
stof_tree_attn_fwd, against the definition in 64 bits.

A softmax does not change when a row's scores all move by the same amount, so
the reference (tests/scored_reference.py) gets the distances less the row's
least one (slope >= 0), or what they lack to its greatest one (slope < 0, with
the slope's magnitude); its tolerance then counts 2^-22 of slope times that."""
import numpy as np
import pytest
import torch

from sparse_mask_transformer_gb300 import stof
from tests.conftest import gpu_encode
from tests.scored_reference import attend, default_scale, f64

pytestmark = pytest.mark.gpu
ROW, BLOCK = stof.STOF_KERNEL_ROWWISE, stof.STOF_KERNEL_BLOCKWISE
FAR = [1 << 24, 1 << 30, -(1 << 24), -(1 << 30)]


def relative(dist, valid, slope):
    """int64 distances [n, m] -> (float64 distances from the row's best visible one, |slope|)."""
    big = np.int64(1) << 40
    if slope >= 0:
        base = np.where(valid, dist, big).min(axis=1, keepdims=True)
        out = dist - base
    else:
        base = np.where(valid, dist, -big).max(axis=1, keepdims=True)
        out = base - dist
    return np.where(valid, out, 0).astype(np.float64), abs(slope)


def check(got, q, k, v, valid, dist, scale, softcap, slope, dtype):
    rel, a = relative(dist, valid, slope)
    want, tol = attend(f64(q), f64(k), f64(v), valid, rel, scale, softcap, a, dtype)
    err = np.abs(f64(got) - want)
    assert np.all(err <= tol), float((err / np.maximum(tol, 1e-30)).max())


@pytest.mark.parametrize("q_start", FAR)
@pytest.mark.parametrize("softcap", [0.0, 20.0])
@pytest.mark.parametrize("d,which,Lq,Lk", [(32, ROW, 90, 300), (128, ROW, 90, 300), (256, ROW, 90, 300), (64, BLOCK, 200, 300),
                                           (128, BLOCK, 200, 300), (64, BLOCK, 130, 4500), (128, BLOCK, 130, 4500)])
def test_far_queries_of_a_format(gpu_lib, d, which, Lq, Lk, softcap, q_start):
    H, Hkv, dtype = 3, 1, torch.bfloat16
    slopes = [0.5, -0.5, 0.0371]
    rng = np.random.default_rng(Lk)
    masks = (rng.random((1, Lq, Lk)) < 0.6).astype(np.uint8)
    masks[0, :, 128:256] = 1
    masks[0, 7] = 0
    g = torch.Generator().manual_seed(d)
    q = torch.randn(1, H, Lq, d, generator=g).to(dtype)
    k, v = (torch.randn(1, Hkv, Lk, d, generator=g).to(dtype) for _ in range(2))
    fmt, ws, _ = gpu_encode(torch.from_numpy(masks).cuda(), 128, 128)
    o = torch.empty_like(q).cuda()
    score = stof.Score(softcap, torch.tensor(slopes, dtype=torch.float32, device="cuda"), q_start)
    stof.stof_mha_fwd_score(q.cuda(), k.cuda(), v.cuda(), fmt, default_scale(d), score, 0, 0, which, o)
    stof.stof_format_sync(fmt)
    assert fmt.device_error == 0
    dist = np.abs(np.arange(Lq)[:, None] + q_start - np.arange(Lk)[None, :])
    for h in range(H):
        check(o[0, h], q[0, h], k[0, 0], v[0, 0], masks[0] != 0, dist, default_scale(d), softcap, float(np.float32(slopes[h])), dtype)


@pytest.mark.parametrize("start", [0, 1 << 24])
@pytest.mark.parametrize("d,which", [(64, BLOCK), (128, BLOCK), (64, ROW)])
def test_rows_whose_keys_are_all_in_far_tiles(gpu_lib, d, which, start):
    """Packed so that the listed tiles are far from the query tile, on both sides of it and behind it."""
    L, dtype = 9000, torch.bfloat16
    masks = np.zeros((1, 256, L), dtype=np.uint8)
    masks[0, :128, :40] = 1
    masks[0, :100, 8900:8950] = 1
    masks[0, 128:, 8700:8990] = 1
    g = torch.Generator().manual_seed(d)
    q = torch.randn(1, 2, 256, d, generator=g).to(dtype)
    k, v = (torch.randn(1, 1, L, d, generator=g).to(dtype) for _ in range(2))
    slopes = [0.61, -0.61]
    fmt, ws, _ = gpu_encode(torch.from_numpy(masks).cuda(), 128, 128)
    o = torch.empty_like(q).cuda()
    score = stof.Score(0.0, torch.tensor(slopes, dtype=torch.float32, device="cuda"), start)
    stof.stof_mha_fwd_score(q.cuda(), k.cuda(), v.cuda(), fmt, default_scale(d), score, 0, 0, which, o)
    dist = np.abs(np.arange(256)[:, None] + start - np.arange(L)[None, :])
    for h in range(2):
        check(o[0, h], q[0, h], k[0, 0], v[0, 0], masks[0] != 0, dist, default_scale(d), 0.0, float(np.float32(slopes[h])), dtype)


def bits_of(sees):
    T = sees.shape[-1]
    wide = np.zeros((*sees.shape[:-1], -(-T // 32) * 32), dtype=bool)
    wide[..., :T] = sees
    return torch.tensor(np.packbits(wide, axis=-1, bitorder="little").view("<i4").copy(), device="cuda")


@pytest.mark.parametrize("softcap", [0.0, 20.0])
@pytest.mark.parametrize("own", [True, False])
@pytest.mark.parametrize("base", [1 << 24, 2 ** 31 - 60, -2 ** 31 + 5_000_000])
@pytest.mark.parametrize("d,H,T", [(64, 3, 5), (64, 3, 20), (64, 6, 40), (128, 3, 5), (128, 6, 40)])
def test_drafted_tokens_far_from_the_cache(gpu_lib, d, H, T, base, own, softcap):
    """Committed keys at 0 .. len, drafted tokens far from them and from one another; tokens that do not see themselves
    (their nearest key is another drafted one, or a committed one 2^24 and more away)."""
    dtype, lens = torch.float16, [0, 300, 5000]
    B, cap = len(lens), 5000 + T + 9
    slopes = ([0.5, -0.5, 0.0371] * 2)[:H]
    rng = np.random.default_rng(T)
    sees = np.tril(rng.random((B, T, T)) < 0.5, -1)
    sees[:, T // 2] = False
    if own:
        sees |= np.eye(T, dtype=bool)
    positions = base + np.sort(rng.integers(0, 60, (B, T)), axis=1)
    positions[:, 1::4] -= 5_000_000                       # some far from the others
    g = torch.Generator().manual_seed(d + T)
    q = torch.randn(B, H, T, d, generator=g).to(dtype)
    k, v = (torch.randn(B, 1, cap, d, generator=g).to(dtype) for _ in range(2))
    o = torch.full_like(q, 5.0).cuda()
    ws = torch.empty(stof.stof_tree_attn_workspace_bytes(B, H, 1, T, d), dtype=torch.uint8, device="cuda")
    err = torch.zeros(1, dtype=torch.int64, device="cuda")
    score = stof.Score(softcap, torch.tensor(slopes, dtype=torch.float32, device="cuda"))
    stof.stof_tree_attn_fwd(q.cuda(), k.cuda(), v.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"), default_scale(d),
                            o, ws, tree=bits_of(sees), positions=torch.tensor(positions, dtype=torch.int32, device="cuda"),
                            score=score, device_error=err)
    assert err.item() == 0
    for b, n in enumerate(lens):
        valid = np.concatenate([np.ones((T, n), dtype=bool), sees[b]], axis=1)
        at = np.concatenate([np.arange(n), positions[b]])
        dist = np.abs(positions[b][:, None] - at[None, :])
        for h in range(H):
            check(o[b, h], q[b, h], k[b, 0, :n + T], v[b, 0, :n + T], valid, dist, default_scale(d), softcap,
                  float(np.float32(slopes[h])), dtype)


@pytest.mark.parametrize("d,H", [(64, 3), (64, 33), (128, 3)])
def test_a_slope_below_zero_over_a_long_cache(gpu_lib, d, H):
    """Without positions: the farthest keys weigh most, in another share than the drafted tokens."""
    T, n, dtype = 3, 70001, torch.bfloat16
    g = torch.Generator().manual_seed(d)
    q = torch.randn(1, H, T, d, generator=g).to(dtype)
    k, v = (torch.randn(1, 1, n + T, d, generator=g).to(dtype) for _ in range(2))
    slopes = [-0.77, 0.77, -0.01] * (H // 3)
    o = torch.full_like(q, 5.0).cuda()
    ws = torch.empty(stof.stof_tree_attn_workspace_bytes(1, H, 1, T, d), dtype=torch.uint8, device="cuda")
    score = stof.Score(0.0, torch.tensor(slopes, dtype=torch.float32, device="cuda"))
    stof.stof_tree_attn_fwd(q.cuda(), k.cuda(), v.cuda(), torch.tensor([n], dtype=torch.int32, device="cuda"), default_scale(d),
                            o, ws, score=score)
    valid = np.arange(n + T)[None, :] <= n + np.arange(T)[:, None]
    dist = np.abs(n + np.arange(T)[:, None] - np.arange(n + T)[None, :])
    for h in range(3):
        check(o[0, h], q[0, h], k[0, 0], v[0, 0], valid, dist, default_scale(d), 0.0, float(np.float32(slopes[h])), dtype)
