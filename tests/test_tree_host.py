"""Refusals of stof_tree_attn_fwd and its workspace sizes (no GPU, no launch)."""
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


def _call(lib, q=FAKE, k=FAKE, o=FAKE, dt=1, B=2, H=8, Hkv=2, T=4, d=128, cap=256, lens=FAKE, counts=None, tree=None,
          positions=None, scale=0.1, score=None, ws=FAKE, ws_bytes=1 << 40, err=None):
    return lib.stof_tree_attn_fwd(q, k, FAKE, dt, B, H, Hkv, T, d, cap, lens, counts, tree, positions, scale,
                                  None if score is None else ctypes.byref(score), o, ws, ws_bytes, err, None)


def test_bad_calls_are_refused(lib):
    S = stof.stof_score
    assert _call(lib, q=None) == stof.STOF_ERR_INVALID_ARG
    assert _call(lib, lens=None) == stof.STOF_ERR_INVALID_ARG
    assert _call(lib, ws=None) == stof.STOF_ERR_INVALID_ARG
    assert _call(lib, dt=2) == stof.STOF_ERR_DTYPE
    for kw in (dict(B=0), dict(H=0), dict(Hkv=0), dict(T=0), dict(cap=0), dict(scale=float("inf"))):
        assert _call(lib, **kw) == stof.STOF_ERR_INVALID_ARG, kw
    assert _call(lib, d=32) == stof.STOF_ERR_UNSUPPORTED
    assert _call(lib, d=256) == stof.STOF_ERR_UNSUPPORTED
    assert _call(lib, Hkv=3) == stof.STOF_ERR_SHAPE
    assert _call(lib, T=1025) == stof.STOF_ERR_SHAPE
    assert _call(lib, B=1 << 20, H=1 << 10, T=4) == stof.STOF_ERR_SHAPE
    assert _call(lib, score=S(-2.0, None, 0)) == stof.STOF_ERR_INVALID_ARG
    assert _call(lib, q=FAKE + 8) == stof.STOF_ERR_ALIGNMENT
    assert _call(lib, ws=FAKE + 8) == stof.STOF_ERR_ALIGNMENT
    assert _call(lib, tree=FAKE + 2) == stof.STOF_ERR_ALIGNMENT
    assert _call(lib, positions=FAKE + 1) == stof.STOF_ERR_ALIGNMENT
    assert _call(lib, err=FAKE + 4) == stof.STOF_ERR_ALIGNMENT
    need = stof.stof_tree_attn_workspace_bytes(2, 8, 2, 4, 128)
    assert _call(lib, ws_bytes=need - 1) == stof.STOF_ERR_WORKSPACE


def test_workspace_sizes(lib):
    ws = stof.stof_tree_attn_workspace_bytes
    assert ws(1, 8, 2, 1, 64) > 0
    assert ws(0, 8, 2, 1, 64) == 0 and ws(1, 8, 3, 1, 64) == 0 and ws(1, 8, 2, 0, 64) == 0
    assert ws(1, 8, 2, 1025, 64) == 0 and ws(1, 8, 2, 1, 96) == 0


def test_binding_refuses_host_tensors(lib):
    q = torch.zeros(1, 4, 2, 64, dtype=torch.float16)
    k = torch.zeros(1, 2, 16, 64, dtype=torch.float16)
    n = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(stof.StofError) as e:
        stof.stof_tree_attn_fwd(q, k, k, n, 0.1, q.clone(), torch.zeros(16, dtype=torch.uint8))
    assert e.value.status == stof.STOF_ERR_INVALID_ARG
