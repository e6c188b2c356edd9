"""The row-wise kernel where key 0 of a head is masked (a left-padded batch)
and its V row holds anything: plain and scored calls, against the definition
in 64 bits (tests/scored_reference.py derives the tolerance)."""
import numpy as np
import pytest
import torch

from sparse_mask_transformer_gb300 import stof
from tests.conftest import gpu_encode
from tests.scored_reference import attend_heads, default_scale, f64, head_slopes

pytestmark = pytest.mark.gpu
ROW = stof.STOF_KERNEL_ROWWISE


@pytest.mark.parametrize("junk", [float("nan"), float("inf")])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("d", [32, 64, 128, 256])
@pytest.mark.parametrize("density", [0.02, 0.5])
def test_a_masked_first_key(gpu_lib, density, d, dtype, junk):
    """The first outer tile lists nothing; rows with few keys, many and none."""
    B, H, L = 1, 2, 330
    masks = (np.random.default_rng(d).random((1, L, L)) < density).astype(np.uint8)
    masks[0, 150:200, 128:256] = 1
    masks[0, :, :128] = 0
    masks[0, 7] = 0
    g = torch.Generator().manual_seed(d)
    q, k, v = ((torch.randn(B, H, L, d, generator=g) * s).to(dtype) for s in (2.0, 1.0, 1.0))
    vj, kj = v.clone(), k.clone()
    vj[:, :, :128] = junk
    kj[:, :, :128] = junk
    fmt, ws, _ = gpu_encode(torch.from_numpy(masks).cuda(), 128, 128)
    dist = np.abs(np.arange(L)[:, None] - np.arange(L)[None, :]).astype(np.float64)
    slopes = head_slopes(H)
    score = stof.Score(20.0, torch.tensor(slopes, dtype=torch.float32, device="cuda"))
    for sc, cap, sl in ((None, 0.0, None), (score, 20.0, slopes)):
        o = torch.empty_like(q).cuda()
        stof.stof_mha_fwd_score(q.cuda(), kj.cuda(), vj.cuda(), fmt, default_scale(d), sc, 0, 0, ROW, o)
        want, tol = attend_heads(f64(q), f64(k), f64(v), lambda b, h: masks[0] != 0, dist, default_scale(d), cap, sl, dtype)
        assert np.all(np.abs(f64(o) - want) <= tol)
        assert torch.all(o[:, :, 7] == 0)
