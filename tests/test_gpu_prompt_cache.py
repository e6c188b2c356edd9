"""The documented calls of a decoder's prompt and its next tokens, one after the
other on the K/V caches themselves (zeros before, as documented, and longer
than the prompt; ragged requests, one of them empty), with no copy of the
caches in between: rotate into the cache, encode the documents with k_doc = -1
behind each prompt, attend over the caches; then drafted tokens.  Against the
definition in 64 bits (tests/scored_reference.py derives the tolerance)."""
import os
import re

import numpy as np
import pytest
import torch

from sparse_mask_transformer_gb300 import stof
from tests.conftest import ROOT
from tests.scored_reference import attend, default_scale, f64, head_slopes

pytestmark = pytest.mark.gpu
OPTIONS = {"cap": (30.0, False), "slopes": (0.0, True), "both": (20.0, True), "plain": (0.0, False)}


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("option", list(OPTIONS))
@pytest.mark.parametrize("d,Hkv", [(32, 2), (64, 2), (64, 4), (128, 2), (128, 4), (256, 2)])
def test_the_documented_sequence(gpu_lib, d, Hkv, option, dtype):
    B, H, L, T, cap = 3, 4, 300, 2, 417
    softcap, sl = OPTIONS[option]
    slopes = head_slopes(H) if sl else None
    lens = np.array([300, 217, 0])
    g = torch.Generator().manual_seed(d)
    packed = torch.randn(B, L, H + 2 * Hkv, d, generator=g).to(dtype).cuda()
    draft = torch.randn(B, T, H + 2 * Hkv, d, generator=g).to(dtype).cuda()
    q, k, v = (t.transpose(1, 2) for t in packed.split([H, Hkv, Hkv], dim=2))
    counts = torch.tensor(lens, dtype=torch.int32, device="cuda")
    for b, n in enumerate(lens):
        packed[b, n:] = float("nan")                    # padding of the projection: neither read nor written
    k_cache, v_cache = (torch.zeros(B, Hkv, cap, d, dtype=dtype, device="cuda") for _ in range(2))
    k_cache[1, :, 350:] = float("nan")                  # K rows of masked keys may hold anything
    q_rot = torch.zeros(B, H, L, d, dtype=dtype, device="cuda")
    plan = stof.stof_rope_plan_init(d)
    stof.stof_rope_fwd(plan, q, k, v, q_rot, k_cache, v_cache, counts=counts)
    at, keys = torch.arange(L, device="cuda"), torch.arange(cap, device="cuda")
    doc = torch.where(at[None] < counts[:, None], 0, -1).to(torch.int32)
    k_doc = torch.where(keys[None] < counts[:, None], 0, -1).to(torch.int32)
    order, k_order = at.to(torch.int32).repeat(B, 1), keys.to(torch.int32).repeat(B, 1)
    ws = torch.empty(stof.stof_encode_workspace_bytes(B, L, cap, 128, 128), dtype=torch.uint8, device="cuda")
    fmt = stof.stof_encode_documents(doc, k_doc, order, k_order, 128, 128, ws)
    o = torch.full_like(q_rot, 5.0)
    score = stof.Score(softcap, None if slopes is None else torch.tensor(slopes, dtype=torch.float32, device="cuda"))
    scale = default_scale(d)
    stof.stof_mha_fwd_score(q_rot, k_cache, v_cache, fmt, scale, None if option == "plain" else score, 1, 0,
                            stof.STOF_KERNEL_AUTO, o)
    stof.stof_format_sync(fmt)
    assert fmt.device_error == 0

    def check(got, query, b, n, valid, rows):
        dist = np.abs(rows[:, None] - np.arange(n)[None, :]).astype(np.float64)
        for h in range(H):
            kv = h // (H // Hkv)
            want, tol = attend(f64(query[b, h]), f64(k_cache[b, kv, :n]), f64(v_cache[b, kv, :n]), valid, dist, scale, softcap,
                               0.0 if slopes is None else slopes[h], dtype)
            assert np.all(np.abs(f64(got[b, h]) - want) <= tol)

    for b, n in enumerate(lens):
        assert torch.all(o[b, :, n:] == 0)
        if n:
            check(o[:, :, :n], q_rot[:, :, :n], b, n, np.tril(np.ones((n, n), dtype=bool)), np.arange(n))
    if d not in (64, 128):
        return
    dq, dk, dv = (t.transpose(1, 2) for t in draft.split([H, Hkv, Hkv], dim=2))
    t_rot = torch.empty(B, H, T, d, dtype=dtype, device="cuda")
    stof.stof_rope_fwd(plan, dq, dk, dv, t_rot, k_cache, v_cache, rows=counts)
    tws = torch.empty(stof.stof_tree_attn_workspace_bytes(B, H, Hkv, T, d), dtype=torch.uint8, device="cuda")
    to = torch.full_like(t_rot, 5.0)
    stof.stof_tree_attn_fwd(t_rot, k_cache, v_cache, counts, scale, to, tws, score=score)
    for b, n in enumerate(lens):
        check(to, t_rot, b, n + T, np.arange(n + T)[None, :] <= n + np.arange(T)[:, None], n + np.arange(T))


def test_the_readmes_block_runs(gpu_lib):
    """The decoder's block of README.md as it stands, with only the caller's own tensors given; the allocator's memory is
    full of NaN beforehand."""
    text = open(os.path.join(ROOT, "README.md")).read()
    block, = [b for b in re.findall(r"```python\n(.*?)```", text, re.S) if "stof_rope_plan_init" in b]
    B, H, Hkv, L, T, cap, d = 2, 4, 2, 200, 3, 333, 64
    g = torch.Generator().manual_seed(5)

    def views(n):
        x = torch.randn(B, n, H + 2 * Hkv, d, generator=g).to(torch.bfloat16).cuda()
        return (t.transpose(1, 2) for t in x.split([H, Hkv, Hkv], dim=2))

    def i32(x):
        return x.to(torch.int32).cuda().contiguous()

    at, keys = torch.arange(L).repeat(B, 1), torch.arange(cap).repeat(B, 1)
    env = dict(stof=stof, torch=torch, B=B, Hkv=Hkv, cap=cap, d=d, scale=default_scale(d), doc=i32(at * 0),
               k_doc=i32(torch.where(keys < L, 0, -1)), order=i32(at), k_order=i32(keys), lens=i32(torch.tensor([L, L])),
               bits=i32(torch.tensor([1, 3, 5]).repeat(B, 1)[..., None]), pos=i32(L + torch.tensor([0, 1, 1]).repeat(B, 1)),
               ws=torch.empty(stof.stof_encode_workspace_bytes(B, L, cap, 128, 128), dtype=torch.uint8, device="cuda"),
               ws1=torch.empty(stof.stof_tree_attn_workspace_bytes(B, H, Hkv, T, d), dtype=torch.uint8, device="cuda"))
    env["q"], env["k"], env["v"] = views(L)
    env["q1"], env["k1"], env["v1"] = views(T)
    for name, n in (("q_rot", L), ("o", L), ("q1_rot", T), ("o1", T)):
        env[name] = torch.empty(B, H, n, d, dtype=torch.bfloat16, device="cuda")
    junk = [torch.full((B, Hkv, cap, d), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(4)]
    torch.cuda.synchronize()
    del junk
    exec(block, env)
    torch.cuda.synchronize()
    assert torch.isfinite(env["o"].float()).all() and torch.isfinite(env["o1"].float()).all()
