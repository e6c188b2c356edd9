"""Refusals of stof_prefix_attn_fwd and its workspace sizes (no GPU, no launch)."""
import ctypes

import pytest
import torch

from sparse_mask_transformer_gb300 import build as stof_build
from sparse_mask_transformer_gb300 import stof

FAKE = 1 << 20  # never dereferenced


@pytest.fixture(scope="module")
def lib():
    stof_build.build()
    return stof.load_library()


def _call(lib, q=FAKE, kp=FAKE, vp=FAKE, k=FAKE, v=FAKE, o=FAKE, dt=1, B=4, P=2, H=8, Hkv=2, T=4, d=128, pcap=256, cap=64,
          plens=FAKE, lens=FAKE, counts=None, tree=None, positions=None, scale=0.1, score=None, ws=FAKE, ws_bytes=1 << 40,
          err=None):
    return lib.stof_prefix_attn_fwd(q, kp, vp, k, v, dt, B, P, H, Hkv, T, d, pcap, cap, plens, lens, counts, tree, positions,
                                    scale, None if score is None else ctypes.byref(score), o, ws, ws_bytes, err, None)


def test_bad_calls_are_refused(lib):
    S = stof.stof_score
    for kw in (dict(q=None), dict(kp=None), dict(vp=None), dict(o=None), dict(plens=None), dict(ws=None), dict(k=None),
               dict(v=None), dict(lens=None), dict(k=None, v=None), dict(k=None, lens=None), dict(v=None, lens=None)):
        assert _call(lib, **kw) == stof.STOF_ERR_INVALID_ARG, kw
    assert _call(lib, dt=2) == stof.STOF_ERR_DTYPE
    for kw in (dict(B=0), dict(P=0), dict(H=0), dict(Hkv=0), dict(T=0), dict(cap=0), dict(pcap=0), dict(scale=float("nan"))):
        assert _call(lib, **kw) == stof.STOF_ERR_INVALID_ARG, kw
    for d in (32, 96, 256):
        assert _call(lib, d=d) == stof.STOF_ERR_UNSUPPORTED
    assert _call(lib, Hkv=3) == stof.STOF_ERR_SHAPE
    assert _call(lib, P=3) == stof.STOF_ERR_SHAPE
    assert _call(lib, P=8) == stof.STOF_ERR_SHAPE
    assert _call(lib, T=1025) == stof.STOF_ERR_SHAPE
    assert _call(lib, B=1 << 20, H=1 << 10, T=4) == stof.STOF_ERR_SHAPE
    assert _call(lib, pcap=2 ** 31 - 1, cap=2 ** 31 - 1) == stof.STOF_ERR_SHAPE
    assert _call(lib, B=1 << 16, P=1 << 16, pcap=1 << 22) == stof.STOF_ERR_SHAPE   # more tiles than 32 bits count
    assert _call(lib, score=S(-2.0, None, 0)) == stof.STOF_ERR_INVALID_ARG
    for name in ("q", "kp", "vp", "k", "v", "o", "ws"):
        assert _call(lib, **{name: FAKE + 8}) == stof.STOF_ERR_ALIGNMENT, name
    for name in ("plens", "lens", "counts", "tree", "positions"):
        assert _call(lib, **{name: FAKE + 2}) == stof.STOF_ERR_ALIGNMENT, name
    assert _call(lib, err=FAKE + 4) == stof.STOF_ERR_ALIGNMENT
    need = stof.stof_prefix_attn_workspace_bytes(4, 2, 8, 2, 4, 128)
    assert _call(lib, ws_bytes=need - 1) == stof.STOF_ERR_WORKSPACE


def test_without_own_caches(lib):
    alone = dict(k=None, v=None, lens=None, cap=0)
    need = stof.stof_prefix_attn_workspace_bytes(4, 2, 8, 2, 4, 128)
    assert _call(lib, **alone, ws_bytes=need - 1) == stof.STOF_ERR_WORKSPACE       # everything before it is in order
    assert _call(lib, **alone, tree=FAKE) == stof.STOF_ERR_INVALID_ARG
    assert _call(lib, **alone, positions=FAKE) == stof.STOF_ERR_INVALID_ARG
    assert _call(lib, **alone, score=stof.stof_score(0.0, FAKE, 0)) == stof.STOF_ERR_UNSUPPORTED


def test_workspace_sizes(lib):
    ws = stof.stof_prefix_attn_workspace_bytes
    assert ws(4, 2, 8, 2, 1, 64) > 0
    for bad in ((0, 1, 8, 2, 1, 64), (4, 0, 8, 2, 1, 64), (4, 3, 8, 2, 1, 64), (4, 2, 8, 3, 1, 64), (4, 2, 8, 2, 0, 64),
                (4, 2, 8, 2, 1025, 64), (4, 2, 8, 2, 1, 96), (1 << 20, 1, 1 << 10, 1, 4, 64)):
        assert ws(*bad) == 0, bad


def test_binding_refuses_host_tensors_and_half_of_a_cache(lib):
    q = torch.zeros(2, 4, 2, 64, dtype=torch.float16)
    k = torch.zeros(1, 2, 16, 64, dtype=torch.float16)
    n = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(stof.StofError) as e:
        stof.stof_prefix_attn_fwd(q, k, k, n, None, None, None, 0.1, q.clone(), torch.zeros(16, dtype=torch.uint8))
    assert e.value.status == stof.STOF_ERR_INVALID_ARG
