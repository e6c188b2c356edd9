"""Which sets of caches stof_cache_fork and stof_cache_keep take for
overlapping, against all pairs; and the time that takes (no GPU, no launch: a
call that passes is refused by the check of alignment behind it)."""
import random
import time

import pytest

from sparse_mask_transformer_gb300 import stof
from tests.test_cache_rows_host import FAKE, caches, lib  # noqa: F401 (fixture)

SIZES = dict(slots=2, heads=2, rows=16, d=64)  # 8192 bytes a cache
BYTES = 8192


def fork(lib, a, b):
    return lib.stof_cache_fork(a, b, FAKE + 2, 2 * FAKE, None, None, None)  # src is misaligned


def apart(rng, n, size):
    """Addresses of caches of `size` bytes that do not overlap one another, in any order."""
    at, out = FAKE, []
    for _ in range(n):
        at += 16 * rng.choice([0, 0, 1, 200, 511, 513, 3000])
        out.append(at)
        at += size
    rng.shuffle(out)
    return out


@pytest.mark.parametrize("seed", range(60))
def test_overlap_of_two_sets_is_that_of_some_pair(lib, seed):  # noqa: F811
    rng = random.Random(seed)
    n, more = rng.choice([1, 2, 3, 17, 256]), rng.choice([1, 1, 2])
    a, b = apart(rng, n, BYTES), apart(rng, n, BYTES * more)
    if seed % 3:  # in the gaps of the first, or behind it
        b = [x + max(a) + BYTES - FAKE + 16 * rng.choice([-1, 0, 1]) * (seed % 3 - 1) for x in b]
    x, y = caches(a, **SIZES), caches(b, **dict(SIZES, rows=16 * more))
    some = any(p < q + BYTES * more and q < p + BYTES for p in a for q in b)
    same = any(p == q for p, q in zip(a, b))  # equal sets of other sizes are refused too
    if a == b and more == 1:  # the very same caches, which a fork takes
        some = same = False
    # a set that overlaps itself (the shifted ones may)
    some |= any(p != q and p < q + BYTES * more and q < p + BYTES * more for p in b for q in b)
    want = stof.STOF_ERR_INVALID_ARG if some or same else stof.STOF_ERR_ALIGNMENT
    assert fork(lib, x, y) == want and fork(lib, y, x) == want


@pytest.mark.parametrize("shuffled", [False, True])
def test_the_check_does_not_take_all_pairs(lib, shuffled):  # noqa: F811
    """A fork of 256 caches into as many others, beside one in the same caches, which has nothing to compare: all pairs
    took some 50 times as long."""
    addresses = [FAKE * (i + 1) for i in range(512)]
    if shuffled:
        random.Random(1).shuffle(addresses)
    a, b = caches(addresses[:256], **SIZES), caches(addresses[256:], **SIZES)
    assert fork(lib, a, b) == fork(lib, a, a) == stof.STOF_ERR_ALIGNMENT
    best = [float("inf")] * 2
    for _ in range(40):
        for i, to in enumerate((a, b)):
            begin = time.perf_counter()
            for _ in range(50):
                fork(lib, a, to)
            best[i] = min(best[i], time.perf_counter() - begin)
    assert best[1] < 15 * best[0], best


@pytest.mark.parametrize("n", [2, 3, 24, 256])
@pytest.mark.parametrize("by", [0, 16, BYTES - 16, BYTES])
def test_caches_of_one_set_that_overlap_are_refused(lib, n, by):  # noqa: F811
    """One given twice, or two that share bytes: in the set that is kept, copied from, copied to, or both."""
    rng = random.Random(n + by)
    bad, far = [FAKE + 3 * BYTES * i for i in range(n - 1)], [1 << 30, *(2 * FAKE + FAKE * (i + 600) for i in range(n - 1))]
    bad.append(rng.choice(bad) + by)
    rng.shuffle(bad)
    x, y = caches(bad, **SIZES), caches(far, **SIZES)

    want = stof.STOF_ERR_ALIGNMENT if by == BYTES else stof.STOF_ERR_INVALID_ARG
    for a, b in ((x, y), (y, x), (x, x)):
        assert fork(lib, a, b) == want
    assert lib.stof_cache_keep(x, 4, FAKE + 2, 2 * FAKE, 3 * FAKE, None, None, None) == want  # lens is misaligned
