"""Workspace sizes of stof_prefix_attn_fwd, from the layout (no GPU, no launch)."""
import pytest

from sparse_mask_transformer_gb300 import stof
from tests.test_prefix_host import lib  # noqa: F401 (fixture)


def up256(x):
    return (x + 255) // 256 * 256


@pytest.mark.parametrize("B,P,H,Hkv,T,d,megabytes", [
    (64, 1, 32, 8, 1, 128, 42.6),   # 32 requests of 4 rows fill a tile: 128 rows a slot
    (64, 1, 32, 8, 1, 64, 21.6), (64, 1, 32, 32, 1, 128, 22.4), (4, 1, 32, 8, 1, 128, 5.2), (64, 1, 32, 8, 16, 128, 74.6),
    (16, 1, 32, 8, 16, 128, 49.0), (128, 8, 12, 12, 1, 64, 23.8), (1, 1, 4, 4, 3, 128, None), (2, 2, 5, 1, 1, 64, None),
    (6, 2, 64, 2, 9, 64, None)])
def test_workspace_bytes(lib, B, P, H, Hkv, T, d, megabytes):  # noqa: F811
    rows = H // Hkv * T                                       # of a request for a K/V head
    fill = rows * min(B // P, 128 // rows) if rows < 128 else 128
    copies = 1 if d == 128 or 2 * fill > 128 else (2 if 4 * fill > 128 else 4)
    slot = 128 if copies > 1 else fill
    parts = 608 * slot + 2 * copies * B * H * T
    want = 1024 + up256(parts * d * 4) + up256(parts * 8) + 152 * 16 + 4 * (B + P)
    got = stof.stof_prefix_attn_workspace_bytes(B, P, H, Hkv, T, d)
    assert got == want
    if megabytes is not None:
        assert round(got / 1e6, 1) == megabytes
