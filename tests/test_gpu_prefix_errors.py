"""Error bits of stof_prefix_attn_fwd where the bad length is that of a request
or a prefix behind the first warp's (32), or behind the block's threads (384):
in the workspace's first 8 bytes, with and without an error word."""
import numpy as np
import pytest
import torch

from sparse_mask_transformer_gb300 import stof
from tests.test_gpu_prefix_attention import Case, i32

pytestmark = pytest.mark.gpu


def word(a):
    return a["ws"][:8].view(torch.int64).item()


@pytest.mark.parametrize("name,NP,n,bad", [("lens", 2, 40, 32), ("lens", 2, 40, 40), ("lens", 1, 80, 79), ("counts", 1, 80, 40),
                                           ("plens", 48, 1, 32), ("plens", 48, 2, 47), ("lens", 3, 140, 383), ("lens", 3, 140, 384),
                                           ("counts", 3, 140, 410), ("plens", 420, 1, 400)])
@pytest.mark.parametrize("value", [-1, 2 ** 31 - 1])
def test_a_bad_length_behind_the_first_warp_is_reported(gpu_lib, name, NP, n, bad, value):
    rng = np.random.default_rng(bad)
    c = Case(n, 2, 1, 1, 64, rng.integers(1, 60, NP), rng.integers(0, 20, NP * n), sees="chain", seed=bad)
    a = c.args()
    good = torch.full(c.q.shape, 5.0, dtype=c.dtype, device="cuda")
    c.call(a, good)
    assert word(a) == 0
    c.check(good)
    lengths = {"lens": c.lens, "counts": c.counts, "plens": c.plens}[name].copy()
    lengths[bad] = value
    skipped = range(bad * n, (bad + 1) * n) if name == "plens" else (bad,)
    words, outs = [], []
    for k in range(20):  # what one call leaves in shared memory is not what the next one reports
        b = dict(c.args(), ws=a["ws"])
        if k % 2 == 0:
            b[name] = i32(lengths)
        outs.append(torch.full_like(good, 5.0))
        err = torch.zeros(1, dtype=torch.int64, device="cuda") if k % 4 < 2 else None
        c.call(b, outs[-1], err)
        words.append(b["ws"][:8].view(torch.int64).clone())
        if err is not None:
            assert err.item() == (0 if k % 2 else stof.STOF_DEVERR_BAD_LENGTH)
    assert [int(w) for w in words] == [stof.STOF_DEVERR_BAD_LENGTH, 0] * 10
    for k, o in enumerate(outs):
        assert torch.equal(o, outs[k % 2])
    for got, left in ((outs[0].cpu(), skipped), (outs[1].cpu(), ())):
        for b in left:
            assert torch.all(got[b] == 5.0)
            got[b] = good[b].cpu()
        c.check(got)
