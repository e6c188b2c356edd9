"""The language-model operators in one run, as a decoder uses them: the prompt's
packed projection is turned (stof_rope_fwd) into the attention's layout and
into the K/V cache, attended under a document mask with capped and lowered
scores (stof_encode_documents, stof_mha_fwd_score), projected
(stof_oproj_fwd); then drafted tokens are turned and appended at each
request's length and attended over the cache (stof_tree_attn_fwd).  Against
the whole computation in 64 bits, and the two attentions against each other."""
import math

import numpy as np
import pytest
import torch

import oracle
from sparse_mask_transformer_gb300 import stof
from tests.scored_reference import HALF, attend, f64, head_slopes

pytestmark = pytest.mark.gpu


def turned(x, pos, w):
    """x [B, H, T, d] in 64 bits, halves layout."""
    h = x.shape[-1] // 2
    ang = pos[:, None, :, None] * w
    c, s = np.cos(ang), np.sin(ang)
    return np.concatenate([x[..., :h] * c - x[..., h:] * s, x[..., h:] * c + x[..., :h] * s], axis=-1)


@pytest.mark.parametrize("d,H,Hkv,dtype", [(128, 8, 2, torch.bfloat16), (64, 4, 4, torch.float16)])
def test_prompt_then_drafted_tokens(gpu_lib, d, H, Hkv, dtype):
    B, L, T, cap, N = 2, 300, 6, 400, 256
    g = torch.Generator().manual_seed(d)
    packed = torch.randn(B, L, H + 2 * Hkv, d, generator=g).to(dtype).cuda()
    draft = torch.randn(B, T, H + 2 * Hkv, d, generator=g).to(dtype).cuda()
    wo = (torch.randn(N, H * d, generator=g) / math.sqrt(H * d)).to(dtype).cuda()
    lens = np.array([300, 217])                      # request 1 is padded behind its 217 tokens
    plan = stof.stof_rope_plan_init(d, theta=10000.0, scaling=stof.STOF_ROPE_LINEAR, factor=2.0)
    w = np.array([10000.0 ** (-2 * p / d) / 2.0 for p in range(d // 2)])
    slopes, softcap, scale = head_slopes(H), 30.0, 1 / math.sqrt(d)
    score = stof.Score(softcap, torch.tensor(slopes, dtype=torch.float32, device="cuda"))
    dlens = torch.tensor(lens, dtype=torch.int32, device="cuda")
    err = torch.zeros(1, dtype=torch.int64, device="cuda")

    # the prompt: Q to the attention's layout, K and V straight into the cache's rows 0 .. len
    split = [H, Hkv, Hkv]
    q, k, v = (t.transpose(1, 2) for t in packed.split(split, dim=2))
    qo = torch.zeros(B, H, L, d, dtype=dtype, device="cuda")
    kc, vc = (torch.full((B, Hkv, cap, d), float("nan"), dtype=dtype, device="cuda") for _ in range(2))
    zero = torch.zeros(B, dtype=torch.int32, device="cuda")
    stof.stof_rope_fwd(plan, q, k, v, qo, kc, vc, counts=dlens, rows=zero, device_error=err)
    # attention over the prompt (K, V of the padding are 0, not the cache's untouched rows)
    kp, vp = (torch.nan_to_num(t[:, :, :L], nan=0.0).contiguous() for t in (kc, vc))
    at = torch.arange(L, device="cuda")
    doc = torch.where(at[None] < dlens[:, None], 0, -1).to(torch.int32)
    order = at.to(torch.int32).repeat(B, 1)
    ws = torch.empty(stof.stof_encode_workspace_bytes(B, L, L, 128, 128), dtype=torch.uint8, device="cuda")
    fmt = stof.stof_encode_documents(doc, doc, order, order, 128, 128, ws)
    o = torch.empty_like(qo)
    stof.stof_mha_fwd_score(qo, kp, vp, fmt, scale, score, 1, 0, stof.STOF_KERNEL_AUTO, o)
    y = torch.empty(B, L, N, dtype=dtype, device="cuda")
    stof.stof_oproj_fwd(o, wo, None, None, y)
    # drafted tokens: a tree of T, K and V appended at each request's length
    parents = [-1, 0, 0, 1, 1, 2]
    sees = np.zeros((T, T), dtype=bool)
    depth = np.zeros(T, dtype=np.int64)
    for t, p in enumerate(parents):
        sees[t, t] = True
        if p >= 0:
            sees[t] |= sees[p]
            depth[t] = depth[p] + 1
    bits = torch.tensor([[sum(1 << u for u in range(T) if sees[t, u])] for t in range(T)], dtype=torch.int32,
                        device="cuda").repeat(B, 1, 1)
    positions = torch.tensor(lens[:, None] + depth, dtype=torch.int32, device="cuda")
    dq, dk, dv = (t.transpose(1, 2) for t in draft.split(split, dim=2))
    tq = torch.empty(B, H, T, d, dtype=dtype, device="cuda")
    stof.stof_rope_fwd(plan, dq, dk, dv, tq, kc, vc, positions=positions, rows=dlens, device_error=err)
    tws = torch.empty(stof.stof_tree_attn_workspace_bytes(B, H, Hkv, T, d), dtype=torch.uint8, device="cuda")
    to = torch.empty_like(tq)
    stof.stof_tree_attn_fwd(tq, kc, vc, dlens, scale, to, tws, tree=bits, positions=positions, score=score, device_error=err)
    stof.stof_format_sync(fmt)
    assert err.item() == 0 and fmt.device_error == 0

    # 64 bits: rotations from the packed inputs (checked against the kernels' within one rounding and their fp32 angles),
    # then each attention from the rotated values the kernels stored, as every step rounds its outputs
    pos = np.tile(np.arange(L, dtype=np.float64), (B, 1))
    u = HALF[dtype]
    for got, want in ((qo, turned(f64(q), pos, w)), (kc[:, :, :L], turned(f64(k), pos, w))):
        for b in range(B):
            n = lens[b]
            e = np.abs(f64(got[b, :, :n]) - want[b, :, :n])
            assert np.all(e <= u * np.abs(want[b, :, :n]) * 1.02 + 2.0 ** -17)
    dist = np.abs(np.arange(L)[:, None] - np.arange(L)[None, :]).astype(np.float64)
    causal = np.tril(np.ones((L, L), dtype=bool))
    for b in range(B):
        n = int(lens[b])
        for h in range(H):
            kv = h // (H // Hkv)
            want, tol = attend(f64(qo[b, h]), f64(kp[b, kv]), f64(vp[b, kv]), causal & (np.arange(L) < n), dist, scale,
                               softcap, slopes[h], dtype)
            want[n:] = 0.0
            assert np.all(np.abs(f64(o[b, h]) - want) <= tol)
            valid = np.concatenate([np.ones((T, n), dtype=bool), sees], axis=1)
            where = np.concatenate([np.arange(n), n + depth])
            want, tol = attend(f64(tq[b, h]), f64(kc[b, kv, :n + T]), f64(vc[b, kv, :n + T]), valid,
                               np.abs((n + depth)[:, None] - where[None]).astype(np.float64), scale, softcap, slopes[h], dtype)
            assert np.all(np.abs(f64(to[b, h]) - want) <= tol)
    want = oracle.oproj(f64(o), f64(wo), None, None)
    assert np.all(np.abs(f64(y) - want) <= u * (np.abs(want) + 1))


def test_decoding_repeats_the_prompts_rows(gpu_lib):
    """One token at a time over the cache gives the rows of the prompt's causal attention (two kernels, two roundings
    of P: both within the tolerance of the same 64-bit values)."""
    B, H, Hkv, L, d, dtype = 1, 4, 2, 140, 128, torch.bfloat16
    g = torch.Generator().manual_seed(3)
    q = (torch.randn(B, H, L, d, generator=g) * 2).to(dtype).cuda()
    k, v = (torch.randn(B, Hkv, L, d, generator=g).to(dtype).cuda() for _ in range(2))
    order = torch.arange(L, dtype=torch.int32, device="cuda")[None].contiguous()
    doc = torch.zeros_like(order)
    ws = torch.empty(stof.stof_encode_workspace_bytes(1, L, L, 128, 128), dtype=torch.uint8, device="cuda")
    fmt = stof.stof_encode_documents(doc, doc, order, order, 128, 128, ws)
    o = torch.empty_like(q)
    scale, score = 1 / math.sqrt(d), stof.Score(50.0)
    stof.stof_mha_fwd_score(q, k, v, fmt, scale, score, 0, 0, stof.STOF_KERNEL_AUTO, o)
    tws = torch.empty(stof.stof_tree_attn_workspace_bytes(B, H, Hkv, 1, d), dtype=torch.uint8, device="cuda")
    dist = np.zeros((1, L))
    for t in (0, 1, 63, 64, 127, 128, 139):
        one = q[:, :, t:t + 1].contiguous()
        got = torch.empty_like(one)
        stof.stof_tree_attn_fwd(one, k, v, torch.tensor([t], dtype=torch.int32, device="cuda"), scale, got, tws, score=score)
        for h in range(H):
            want, tol = attend(f64(one[0, h]), f64(k[0, h // 2]), f64(v[0, h // 2]), np.arange(L)[None] <= t, dist, scale, 50.0,
                               0.0, dtype)
            assert np.all(np.abs(f64(got[0, h]) - want) <= tol)
            assert np.all(np.abs(f64(o[0, h, t:t + 1]) - want) <= tol)
