"""stof_prefix_attn_fwd with groups of unequal size, the smaller ones filled up
with requests of no tokens, and with thousands of requests or prefixes."""
import numpy as np
import pytest
import torch

from tests.scored_reference import head_slopes
from tests.test_gpu_prefix_attention import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d,H,Hkv,T,softcap,slopes", [(64, 4, 4, 1, 0.0, False), (64, 12, 12, 1, 30.0, True), (128, 8, 2, 1, 0.0, False),
                                                      (128, 8, 2, 5, 20.0, False), (64, 6, 1, 9, 0.0, True)])
@pytest.mark.parametrize("own", [True, False])
def test_groups_of_unequal_size(gpu_lib, d, H, Hkv, T, softcap, slopes, own):
    sizes, n = [5, 1, 0, 16, 3], 16
    rng = np.random.default_rng(d + H + T)
    counts = np.concatenate([np.where(np.arange(n) < m, rng.integers(1, T + 1, n), 0) for m in sizes])
    lens = rng.integers(0, 150, n * len(sizes)) if own else None
    Case(n, H, Hkv, T, d, [700, 90, 300, 1, 257], lens, counts=counts, softcap=softcap, seed=d,
         slopes=head_slopes(H) if slopes and own else None).run()


@pytest.mark.parametrize("NP,n", [(1, 5000), (3000, 1), (1000, 3)])
@pytest.mark.parametrize("d", [64, 128])
def test_thousands_of_requests_and_prefixes(gpu_lib, NP, n, d):
    """Many rounds of the block's threads over the lengths; shares that begin within any of them."""
    rng = np.random.default_rng(NP)
    B = NP * n
    c = Case(n, 1, 1, 1, d, rng.integers(0, 90, NP), rng.integers(0, 40, B), torch.float16, counts=rng.integers(0, 2, B),
             sees="chain", seed=NP)
    c.run()
