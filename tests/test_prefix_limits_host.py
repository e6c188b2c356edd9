"""The most rows that stof_prefix_attn_fwd takes (no GPU, no launch)."""
from sparse_mask_transformer_gb300 import stof
from tests.test_prefix_host import _call, lib  # noqa: F401 (fixture)


def test_the_most_rows(lib):  # noqa: F811
    most = 2147480000 - 1
    one = dict(B=1, P=1, H=1, Hkv=1, T=1, d=64, ws_bytes=0)
    assert _call(lib, **one, pcap=most - 64, cap=64) == stof.STOF_ERR_WORKSPACE      # the sizes are in order
    assert _call(lib, **one, pcap=most - 63, cap=64) == stof.STOF_ERR_SHAPE
    alone = dict(one, k=None, v=None, lens=None, cap=0)
    assert _call(lib, **alone, pcap=most - 1) == stof.STOF_ERR_WORKSPACE
    assert _call(lib, **alone, pcap=most) == stof.STOF_ERR_SHAPE
