"""Rotary positions of a step without tokens: nothing to do, whatever the caches
the tokens would have gone to."""
import ctypes
import struct

import pytest
import torch

from sparse_mask_transformer_gb300 import build as stof_build
from sparse_mask_transformer_gb300 import stof

FAKE = 1 << 20  # never dereferenced: nothing is launched


@pytest.mark.parametrize("B,T", [(2, 0), (0, 4), (0, 0)])
def test_no_tokens_beside_caches(B, T):
    stof_build.build()
    lib, plan = stof.load_library(), stof.stof_rope_plan_init(64)
    row = lambda data: (data, 4096, 512, 64)  # noqa: E731
    x = struct.pack("24q", *row(0), *row(0), *row(0), *row(0), *row(FAKE), *row(FAKE))
    assert lib.stof_rope_fwd(ctypes.byref(plan), x, 0, B, 4, 2, T, 64, None, None, None, 8, None, None) == stof.STOF_OK
    assert lib.stof_rope_fwd(ctypes.byref(plan), x, 0, 1, 4, 2, 1, 64, None, None, None, 8, None, None) == \
        stof.STOF_ERR_INVALID_ARG


@pytest.mark.gpu
def test_an_empty_step_from_the_binding(gpu_lib):
    cache = torch.full((2, 2, 16, 64), 7.0, dtype=torch.float16, device="cuda")
    q, k, v = (torch.empty(2, h, 0, 64, dtype=torch.float16, device="cuda") for h in (4, 2, 2))
    rows = torch.tensor([3, 5], dtype=torch.int32, device="cuda")
    out = cache.clone(), cache.clone()
    stof.stof_rope_fwd(stof.stof_rope_plan_init(64), q, k, v, q.clone(), *out, rows=rows)
    assert torch.equal(out[0], cache) and torch.equal(out[1], cache)
