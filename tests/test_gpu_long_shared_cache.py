"""stof_mha_fwd_score where many query heads share few long K/V heads: what
counts is B Hkv Lk keys and B H Lq rows, not keys per query head; K and V
offsets past 2^31 elements."""
import numpy as np
import pytest
import torch

from sparse_mask_transformer_gb300 import stof
from tests.scored_reference import attend, default_scale, f64

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("which", [stof.STOF_KERNEL_AUTO, stof.STOF_KERNEL_BLOCKWISE, stof.STOF_KERNEL_ROWWISE])
def test_many_heads_on_one_long_head(gpu_lib, which):
    B, H, Hkv, Lq, Lk, d, dtype = 64, 32, 1, 5, 1 << 20, 64, torch.bfloat16
    assert B * H * Lk >= 1 << 31 and (B - 1) * Hkv * Lk * d > 1 << 31
    at = np.concatenate([np.arange(3, 40), np.arange(Lk - 200, Lk)])      # the keys of the queries' document
    g = torch.Generator().manual_seed(0)
    q = torch.randn(B, H, Lq, d, generator=g).to(dtype).cuda()
    k, v = (torch.zeros(B, Hkv, Lk, d, dtype=dtype, device="cuda") for _ in range(2))
    where = torch.tensor(at, device="cuda")
    for t in (k, v):
        t[:, :, where] = torch.randn(B, Hkv, len(at), d, generator=g).to(dtype).cuda()
    k_doc = torch.full((1, Lk), -1, dtype=torch.int32, device="cuda")
    k_doc[0, where] = 0
    q_doc = torch.zeros(1, Lq, dtype=torch.int32, device="cuda")
    ws = torch.empty(stof.stof_encode_workspace_bytes(1, Lq, Lk, 128, 128), dtype=torch.uint8, device="cuda")
    fmt = stof.stof_encode_documents(q_doc, k_doc, None, None, 128, 128, ws)
    o = torch.full_like(q, 5.0)
    stof.stof_mha_fwd_score(q, k, v, fmt, default_scale(d), stof.Score(30.0), 0, 0, which, o)
    stof.stof_format_sync(fmt)
    assert fmt.device_error == 0
    for b, h in ((0, 0), (31, 17), (63, 31)):
        want, tol = attend(f64(q[b, h]), f64(k[b, 0, where]), f64(v[b, 0, where]), np.ones((Lq, len(at)), dtype=bool),
                           np.zeros((Lq, len(at))), default_scale(d), 30.0, 0.0, dtype)
        assert np.all(np.abs(f64(o[b, h]) - want) <= tol)
    assert torch.isfinite(o.float()).all() and not torch.any(o == 5.0)
