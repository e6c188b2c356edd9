"""Capped scores at and around the cap on the tensor-core kernels' capped-only
path (no slopes: the fixed reference of bf16, the polynomial taken first and
again in exact form, its masked form) and beside slopes: rows all at +cap, all
at -cap, on both sides, just inside and just past the polynomial's range;
scales of either sign; caps around the largest one with a fixed reference; V
near that reference's bounds.  Prompt and cache attention, against the
definition in 64 bits (tests/scored_reference.py derives the tolerance)."""
import numpy as np
import pytest
import torch

from sparse_mask_transformer_gb300 import stof
from tests.conftest import gpu_encode
from tests.scored_reference import attend, f64

pytestmark = pytest.mark.gpu
ROW, BLOCK = stof.STOF_KERNEL_ROWWISE, stof.STOF_KERNEL_BLOCKWISE
KINDS = ["low", "high", "sides", "edge", "some"]


def scores(kind, cap, scale, n, rng):
    """q.k of n keys, given by K's first element (q's is 1, the others 0)."""
    x = {"low": rng.uniform(-12, -8, n), "high": rng.uniform(8, 12, n), "sides": rng.choice([-1, 1], n) * rng.uniform(0.2, 9, n),
         "edge": rng.choice([-1, 1], n) * rng.uniform(0.49, 0.51, n),             # of the cap: the polynomial holds to half
         "some": np.where(rng.random(n) < 0.02, rng.uniform(-5, 5, n), rng.uniform(-0.1, 0.1, n))}[kind]
    return x * cap / scale


def inputs(kind, cap, scale, H, Lq, Lk, d, dtype, seed, rows_differ=True):
    rng = np.random.default_rng(seed)
    q, k = np.zeros((H, Lq, d)), np.zeros((1, Lk, d))
    q[..., 0] = 1.0
    k[0, :, 0] = scores(kind, cap, scale, Lk, rng)
    if rows_differ:                                      # small products of the other elements, in every row
        q[..., 1:] = rng.normal(size=(H, Lq, d - 1)) * 0.3
        k[0, :, 1:] = rng.normal(size=(Lk, d - 1)) * 0.3
    v = rng.normal(size=(1, Lk, d))
    return [torch.tensor(x[None]).to(dtype) for x in (q, k, v)]


def compare(got, q, k, v, valid, dist, scale, cap, slope, dtype):
    want, tol = attend(f64(q), f64(k), f64(v), valid, dist, scale, cap, slope, dtype)
    err = np.abs(f64(got) - want)
    assert np.all(err <= tol), float((err / np.maximum(tol, 1e-300)).max())


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("cap", [5.0, 59.0, 60.0, 61.0])
@pytest.mark.parametrize("sl", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("d,which,Lq,Lk", [(64, BLOCK, 200, 300), (128, BLOCK, 200, 300), (64, BLOCK, 130, 2100),
                                           (128, BLOCK, 130, 2100), (64, ROW, 60, 300)])
def test_prompt(gpu_lib, d, which, Lq, Lk, dtype, sl, cap, kind):
    H = 2
    for scale in (0.5, -0.5):
        q, k, v = inputs(kind, cap, scale, H, Lq, Lk, d, dtype, 7)
        rng = np.random.default_rng(1)
        masks = (rng.random((1, Lq, Lk)) < 0.6).astype(np.uint8)
        masks[0, :, 128:256] = 1
        masks[0, 3] = 0
        slopes = [0.05, -0.01] if sl else None
        fmt, ws, _ = gpu_encode(torch.from_numpy(masks).cuda(), 128, 128)
        o = torch.empty_like(q).cuda()
        score = stof.Score(cap, torch.tensor(slopes, dtype=torch.float32, device="cuda") if sl else None)
        stof.stof_mha_fwd_score(q.cuda(), k.cuda(), v.cuda(), fmt, scale, score, 0, 0, which, o)
        dist = np.abs(np.arange(Lq)[:, None] - np.arange(Lk)[None, :]).astype(np.float64)
        for h in range(H):
            compare(o[0, h], q[0, h], k[0, 0], v[0, 0], masks[0] != 0, dist, scale, cap,
                    float(np.float32(slopes[h])) if sl else 0.0, dtype)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("cap", [5.0, 60.0, 61.0])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("d,H,T", [(64, 4, 7), (64, 6, 10), (64, 9, 10), (128, 4, 7), (128, 20, 10)])  # four, two, one copies; one
def test_cache(gpu_lib, d, H, T, dtype, cap, kind):
    lens = [0, 77, 1500]
    for scale in (0.5, -0.5):
        B, most = len(lens), max(lens) + T
        qkv = [inputs(kind, cap, scale, H, T, most, d, dtype, 11 + b) for b in range(B)]
        q, k, v = (torch.cat([x[i] for x in qkv]) for i in range(3))
        o = torch.full_like(q, 5.0).cuda()
        ws = torch.empty(stof.stof_tree_attn_workspace_bytes(B, H, 1, T, d), dtype=torch.uint8, device="cuda")
        stof.stof_tree_attn_fwd(q.cuda(), k.cuda(), v.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"), scale, o, ws,
                                score=stof.Score(cap))
        for b, n in enumerate(lens):
            valid = np.arange(n + T)[None, :] <= n + np.arange(T)[:, None]
            for h in (0, H - 1):
                compare(o[b, h], q[b, h], k[b, 0, :n + T], v[b, 0, :n + T], valid, np.zeros_like(valid, dtype=float), scale, cap,
                        0.0, dtype)


@pytest.mark.parametrize("kind,size", [("high", 2.0 ** 30), ("low", 2.0 ** -34)])
@pytest.mark.parametrize("d", [64, 128])
def test_v_near_the_fixed_references_bounds(gpu_lib, d, kind, size):
    """Every score at +60 or -60 (P near 2^87 or 2^-87), V as large or small as the header allows for 300 keys."""
    H, L, dtype, scale = 2, 300, torch.bfloat16, 1.0
    q, k, v = inputs(kind, 60.0, scale, H, L, L, d, dtype, 5, rows_differ=False)
    v = (v.double().sign() * v.double().abs().clamp(0.25, 4.0) / 4.0 * size).to(dtype)
    masks = np.tril(np.ones((1, L, L), dtype=np.uint8))
    fmt, ws, _ = gpu_encode(torch.from_numpy(masks).cuda(), 128, 128)
    o = torch.empty_like(q).cuda()
    stof.stof_mha_fwd_score(q.cuda(), k.cuda(), v.cuda(), fmt, scale, stof.Score(60.0), 0, 0, BLOCK, o)
    to = torch.empty_like(q[:, :, L - 2:]).cuda()
    tws = torch.empty(stof.stof_tree_attn_workspace_bytes(1, H, 1, 2, d), dtype=torch.uint8, device="cuda")
    stof.stof_tree_attn_fwd(q[:, :, L - 2:].contiguous().cuda(), k.cuda(), v.cuda(),
                            torch.tensor([L - 2], dtype=torch.int32, device="cuda"), scale, to, tws, score=stof.Score(60.0))
    for h in range(H):
        compare(o[0, h], q[0, h], k[0, 0], v[0, 0], masks[0] != 0, np.zeros((L, L)), scale, 60.0, 0.0, dtype)
        compare(to[0, h], q[0, h, L - 2:], k[0, 0], v[0, 0], masks[0, L - 2:] != 0, np.zeros((2, L)), scale, 60.0, 0.0, dtype)
