"""stof_tune() measures the plain kernels: its cached result does not decide
which kernel a call with capped or lowered scores or shared K/V heads runs."""
import pytest
import torch

from sparse_mask_transformer_gb300 import stof

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("L,density", [(1024, 0.002), (4096, 0.002), (256, 1.0), (256, 0.05)])
def test_a_tuning_result_is_not_used(gpu_lib, L, density):
    B, H, d = (8, 12, 64) if L == 1024 else (1, 2, 64)
    g = torch.Generator(device="cuda").manual_seed(L)
    mask = (torch.rand(1, L, L, device="cuda", generator=g) < density).to(torch.uint8)
    q, k, v = (torch.randn(B, H, L, d, device="cuda", generator=g).to(torch.bfloat16) for _ in range(3))
    ws = torch.empty(stof.stof_encode_workspace_bytes(1, L, L, 128, 128), dtype=torch.uint8, device="cuda")
    fmt = stof.stof_encode_mask(mask, 128, 128, ws)
    stof.stof_format_sync(fmt)
    slopes = torch.full((H,), 0.1, device="cuda")
    calls = [(H, stof.Score(30.0)), (H, stof.Score(0.0, slopes)), (1, None)]

    def outputs():
        out = []
        for heads, score in calls:
            o = torch.empty_like(q)
            stof.stof_mha_fwd_score(q, k[:, :heads].contiguous(), v[:, :heads].contiguous(), fmt, 0.125, score, 0, 0,
                                    stof.STOF_KERNEL_AUTO, o)
            out.append(o)
        return out

    stof.stof_tune_clear()
    before = outputs()
    tune_ws = torch.empty(stof.stof_tune_workspace_bytes(1, L), dtype=torch.uint8, device="cuda")
    stof.stof_tune(mask, q, k, v, 0.125, 0, 0, tune_ws, torch.empty_like(q))
    after = outputs()
    stof.stof_tune_clear()
    for a, b in zip(before, after):
        assert torch.equal(a, b)
