"""stof_tree_attn_fwd's own error bits in the first 8 bytes of its workspace: a
call without device_error does not fail silently."""
import pytest
import torch

from sparse_mask_transformer_gb300 import stof

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("d,H,Hkv,T", [(64, 4, 2, 1), (64, 8, 2, 12), (128, 8, 2, 3), (128, 64, 1, 40)])
def test_every_call_leaves_its_error_bits(gpu_lib, d, H, Hkv, T):
    B, cap = 3, 600
    g = torch.Generator().manual_seed(d)
    q = torch.randn(B, H, T, d, generator=g).to(torch.bfloat16).cuda()
    k, v = (torch.randn(B, Hkv, cap, d, generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    ws = torch.full((stof.stof_tree_attn_workspace_bytes(B, H, Hkv, T, d),), 0xCD, dtype=torch.uint8, device="cuda")
    word, o, bad = ws[:8].view(torch.int64), torch.empty_like(q), stof.STOF_DEVERR_BAD_LENGTH
    for lens, counts, want in (([10, 500, 0], [T, T, T], 0), ([10, 601, 0], [T, T, T], bad), ([10, 500, 0], [T, 0, T], 0),
                               ([-1, 500, 0], [T, T, T], bad), ([10, 500, 0], [T, T, T + 1], bad), ([9, 8, 7], [T, T, T], 0)):
        ws.fill_(0xCD)
        stof.stof_tree_attn_fwd(q, k, v, i32(lens), 0.1, o, ws, counts=i32(counts))
        assert word.item() == want
    # captured: every replay leaves its own
    lens = i32([10, 500, 0])
    stof.stof_tree_attn_fwd(q, k, v, lens, 0.1, o, ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        stof.stof_tree_attn_fwd(q, k, v, lens, 0.1, o, ws)
    for n, want in ((10, 0), (-3, bad), (20, 0)):
        lens[0] = n
        ws.fill_(0xFF)
        graph.replay()
        assert word.item() == want
