"""Refusals of stof_cache_keep and stof_cache_fork (no GPU, no launch)."""
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


def caches(data=(FAKE, 2 * FAKE), n=None, slots=4, heads=2, rows=64, d=64):
    a = (ctypes.c_void_p * len(data))(*data)
    c = stof.stof_caches(ctypes.cast(a, ctypes.c_void_p), len(data) if n is None else n, slots, heads, rows, d)
    c._keep = a
    return c


BAD_CACHES = [(dict(n=0), stof.STOF_ERR_INVALID_ARG), (dict(slots=0), stof.STOF_ERR_INVALID_ARG),
              (dict(heads=0), stof.STOF_ERR_INVALID_ARG), (dict(rows=0), stof.STOF_ERR_INVALID_ARG),
              (dict(d=0), stof.STOF_ERR_INVALID_ARG), (dict(d=60), stof.STOF_ERR_UNSUPPORTED),
              (dict(d=1032), stof.STOF_ERR_UNSUPPORTED), (dict(data=(FAKE, 0)), stof.STOF_ERR_INVALID_ARG),
              (dict(data=(FAKE, FAKE + 8)), stof.STOF_ERR_ALIGNMENT), (dict(data=(FAKE,) * 257), stof.STOF_ERR_UNSUPPORTED),
              (dict(heads=1 << 28, d=64), stof.STOF_ERR_SHAPE)]


@pytest.mark.parametrize("kw,status", BAD_CACHES)
def test_bad_caches_are_refused(lib, kw, status):
    c = caches(**kw)
    assert lib.stof_cache_keep(c, 4, FAKE, FAKE, FAKE, None, None, None) == status
    assert lib.stof_cache_fork(c, caches(), FAKE, FAKE, None, None, None) == status
    assert lib.stof_cache_fork(caches(), c, FAKE, FAKE, None, None, None) == status


def test_bad_keeps_are_refused(lib):
    def call(c=None, T=4, lens=FAKE, path=2 * FAKE, kept=3 * FAKE, new=None, err=None):
        return lib.stof_cache_keep(caches() if c is None else c, T, lens, path, kept, new, err, None)
    assert lib.stof_cache_keep(None, 4, FAKE, FAKE, FAKE, None, None, None) == stof.STOF_ERR_INVALID_ARG
    for kw in (dict(lens=None), dict(path=None), dict(kept=None), dict(T=0), dict(new=FAKE), dict(new=3 * FAKE)):
        assert call(**kw) == stof.STOF_ERR_INVALID_ARG, kw
    assert call(T=1025) == stof.STOF_ERR_SHAPE
    assert call(c=caches(slots=65536)) == stof.STOF_ERR_SHAPE
    for kw in (dict(lens=FAKE + 2), dict(path=FAKE + 1), dict(kept=FAKE + 3), dict(new=FAKE + 6), dict(err=FAKE + 4)):
        assert call(**kw) == stof.STOF_ERR_ALIGNMENT, kw


def test_bad_forks_are_refused(lib):
    far = (8 * FAKE, 9 * FAKE)

    def call(a=None, b=None, src=FAKE, lens=2 * FAKE, new=None, err=None):
        return lib.stof_cache_fork(caches() if a is None else a, caches(far) if b is None else b, src, lens, new, err, None)
    for kw in (dict(src=None), dict(lens=None), dict(new=FAKE), dict(new=2 * FAKE)):
        assert call(**kw) == stof.STOF_ERR_INVALID_ARG, kw
    assert call(b=caches((8 * FAKE,))) == stof.STOF_ERR_SHAPE
    assert call(b=caches(far, heads=4)) == stof.STOF_ERR_SHAPE
    assert call(b=caches(far, d=128)) == stof.STOF_ERR_SHAPE
    # partly the same caches, or the same with other sizes
    assert call(b=caches((FAKE, 9 * FAKE))) == stof.STOF_ERR_INVALID_ARG
    assert call(b=caches(rows=32)) == stof.STOF_ERR_INVALID_ARG
    assert call(b=caches(slots=3)) == stof.STOF_ERR_INVALID_ARG
    for kw in (dict(src=FAKE + 2), dict(lens=FAKE + 1), dict(new=FAKE + 6), dict(err=FAKE + 4)):
        assert call(**kw) == stof.STOF_ERR_ALIGNMENT, kw


def test_forks_between_overlapping_caches_are_refused(lib):
    size = 4 * 2 * 64 * 64 * 2  # bytes of a cache
    a = caches()
    for data in ((2 * FAKE, FAKE), (8 * FAKE, FAKE + size - 16), (2 * FAKE - size + 16, 8 * FAKE)):
        assert lib.stof_cache_fork(a, caches(data), FAKE, 2 * FAKE, None, None, None) == stof.STOF_ERR_INVALID_ARG, data
    # a smaller set that begins inside one of the larger
    assert lib.stof_cache_fork(a, caches((8 * FAKE, 2 * FAKE + size // 2), rows=32), FAKE, 2 * FAKE, None, None,
                               None) == stof.STOF_ERR_INVALID_ARG
    # side by side is no overlap: the next check answers
    for data in ((FAKE + size, 2 * FAKE + size), (FAKE - size, 2 * FAKE - size)):
        assert lib.stof_cache_fork(a, caches(data), FAKE + 2, 2 * FAKE, None, None, None) == stof.STOF_ERR_ALIGNMENT, data
    # sizes whose product passes 64 bits
    wide = dict(slots=(1 << 31) - 1, rows=(1 << 31) - 1)
    assert lib.stof_cache_fork(caches(**wide), caches((8 * FAKE, 9 * FAKE), **wide), FAKE, 2 * FAKE, None, None,
                               None) == stof.STOF_ERR_INVALID_ARG


def test_binding_refuses_host_tensors(lib):
    with pytest.raises(stof.StofError) as e:
        stof.Caches([torch.zeros(2, 2, 8, 64, dtype=torch.float16)])
    assert e.value.status == stof.STOF_ERR_INVALID_ARG
    with pytest.raises(stof.StofError):
        stof.Caches([])
