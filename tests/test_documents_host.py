"""Refusals of stof_encode_documents and stof_mha_fwd_score, before any
launch (no GPU)."""
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


def _encode(lib, q_doc=FAKE, k_doc=FAKE, q_order=FAKE, k_order=FAKE, n=1, lq=256, lk=256, bm=128, bn=128, ws=FAKE,
            ws_bytes=1 << 30):
    fmt = stof.stof_format()
    return lib.stof_encode_documents(q_doc, k_doc, q_order, k_order, n, lq, lk, bm, bn, ws, ws_bytes, ctypes.byref(fmt),
                                     None)


def test_encode_documents_refuses(lib):
    assert _encode(lib, q_doc=None) == stof.STOF_ERR_INVALID_ARG
    assert _encode(lib, k_doc=None) == stof.STOF_ERR_INVALID_ARG
    assert _encode(lib, q_order=None) == stof.STOF_ERR_INVALID_ARG  # one order without the other
    assert _encode(lib, k_order=None) == stof.STOF_ERR_INVALID_ARG
    assert _encode(lib, q_doc=FAKE + 2) == stof.STOF_ERR_ALIGNMENT
    assert _encode(lib, k_order=FAKE + 1) == stof.STOF_ERR_ALIGNMENT
    assert _encode(lib, n=0) == stof.STOF_ERR_INVALID_ARG
    assert _encode(lib, lk=0) == stof.STOF_ERR_INVALID_ARG
    assert _encode(lib, bm=12) == stof.STOF_ERR_SHAPE
    assert _encode(lib, bn=512) == stof.STOF_ERR_SHAPE
    assert _encode(lib, ws=FAKE + 128) == stof.STOF_ERR_ALIGNMENT
    assert _encode(lib, ws_bytes=100) == stof.STOF_ERR_WORKSPACE


def _fmt(L=256, bm=128, bn=128, synced=1):
    f = stof.stof_format()
    f.n_masks, f.lq, f.lk, f.bm, f.bn = 1, L, L, bm, bn
    f.n_tr = f.n_tc = -(-L // bm)
    for name in ("full_row_ptr", "full_col_idx", "part_row_ptr", "part_col_idx", "bitmaps", "counts_dev", "scratch"):
        setattr(f, name, FAKE)
    f.synced = synced
    return f


def _score(lib, score=None, H=4, Hkv=2, L=256, d=64, dt=1, scale=0.125, which=stof.STOF_KERNEL_ROWWISE, fmt=None, sb=0,
           q=FAKE, o=FAKE):
    fmt = _fmt(L) if fmt is None else fmt
    return lib.stof_mha_fwd_score(q, FAKE, FAKE, dt, 2, H, Hkv, L, L, d, scale, None if score is None else ctypes.byref(score),
                                  ctypes.byref(fmt), sb, 0, which, o, None)


def test_scored_attention_refuses(lib):
    S = stof.stof_score
    assert _score(lib, q=None) == stof.STOF_ERR_INVALID_ARG
    assert _score(lib, q=FAKE + 8) == stof.STOF_ERR_ALIGNMENT
    assert _score(lib, dt=5) == stof.STOF_ERR_DTYPE
    assert _score(lib, Hkv=0) == stof.STOF_ERR_INVALID_ARG
    assert _score(lib, H=4, Hkv=3) == stof.STOF_ERR_SHAPE
    assert _score(lib, d=48) == stof.STOF_ERR_UNSUPPORTED
    assert _score(lib, scale=float("nan")) == stof.STOF_ERR_INVALID_ARG
    assert _score(lib, sb=1) == stof.STOF_ERR_SHAPE  # a mask past the format's
    assert _score(lib, which=3) == stof.STOF_ERR_INVALID_ARG
    assert _score(lib, score=S(-1.0, None, 0)) == stof.STOF_ERR_INVALID_ARG
    assert _score(lib, score=S(float("inf"), None, 0)) == stof.STOF_ERR_INVALID_ARG
    assert _score(lib, score=S(1e-38, None, 0), scale=1e10) == stof.STOF_ERR_INVALID_ARG
    assert _score(lib, score=S(0.0, FAKE + 2, 0)) == stof.STOF_ERR_ALIGNMENT
    assert _score(lib, score=S(0.0, FAKE, (1 << 30) + 1)) == stof.STOF_ERR_SHAPE
    assert _score(lib, d=32, which=stof.STOF_KERNEL_BLOCKWISE) == stof.STOF_ERR_UNSUPPORTED
    assert _score(lib, fmt=_fmt(256, 64, 64), which=stof.STOF_KERNEL_BLOCKWISE) == stof.STOF_ERR_UNSUPPORTED
    # 128 x 64 OTs: block-wise only for plain scores with a K/V head each
    half = _fmt(256, 128, 128)
    half.bn, half.n_tc = 64, 4
    assert _score(lib, fmt=half, which=stof.STOF_KERNEL_BLOCKWISE) == stof.STOF_ERR_UNSUPPORTED
    assert _score(lib, fmt=half, H=4, Hkv=4, score=S(30.0, None, 0), which=stof.STOF_KERNEL_BLOCKWISE) == \
        stof.STOF_ERR_UNSUPPORTED


def test_bindings_refuse_host_tensors(lib):
    q = torch.zeros(1, 4, 128, 64, dtype=torch.bfloat16)
    with pytest.raises(stof.StofError) as e:
        stof.stof_mha_fwd_score(q, q, q, stof.stof_format(), 0.1, None, 0, 0, stof.STOF_KERNEL_AUTO, q.clone())
    assert e.value.status == stof.STOF_ERR_INVALID_ARG
    d = torch.zeros(1, 128, dtype=torch.int32)
    with pytest.raises(stof.StofError) as e:
        stof.stof_encode_documents(d, d, None, None, 128, 128, torch.zeros(16, dtype=torch.uint8))
    assert e.value.status == stof.STOF_ERR_INVALID_ARG
