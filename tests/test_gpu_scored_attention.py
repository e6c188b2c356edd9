"""stof_mha_fwd_score: capped and distance-lowered scores, shared K/V heads,
against the definition in 64 bits (tests/scored_reference.py, which derives
the tolerance), on every kernel."""
import numpy as np
import pytest
import torch

from sparse_mask_transformer_gb300 import stof
from tests.conftest import gpu_encode
from tests.scored_reference import attend_heads, default_scale, f64, head_slopes

pytestmark = pytest.mark.gpu
ROW, BLOCK, AUTO = stof.STOF_KERNEL_ROWWISE, stof.STOF_KERNEL_BLOCKWISE, stof.STOF_KERNEL_AUTO
OPTIONS = {"cap": (30.0, False), "slopes": (0.0, True), "both": (20.0, True), "plain": (0.0, False)}


def tensors(B, H, Hkv, Lq, Lk, d, dtype, seed, gain=2.0):
    g = torch.Generator().manual_seed(seed)
    return [(torch.randn(B, h, L, d, generator=g) * s).to(dtype) for h, L, s in ((H, Lq, gain), (Hkv, Lk, 1.0), (Hkv, Lk, 1.0))]


def run(q, k, v, masks, stride_b, stride_h, which, softcap, slopes, bm=128, bn=128, q_start=0, scale=None, sync=True):
    """Encode, attend; o is followed by a guard."""
    fmt, ws, _ = gpu_encode(torch.from_numpy(masks).cuda(), bm, bn)
    if not sync:
        fmt.synced = 0
    n = q.numel()
    buf = torch.full((n + 4096,), float("nan"), dtype=q.dtype, device="cuda")
    o = buf[:n].view(q.shape)
    s = torch.tensor(slopes, dtype=torch.float32, device="cuda") if slopes is not None else None
    scale = default_scale(q.shape[3]) if scale is None else scale
    stof.stof_mha_fwd_score(q.cuda(), k.cuda(), v.cuda(), fmt, scale, stof.Score(softcap, s, q_start), stride_b, stride_h,
                            which, o)
    stof.stof_format_sync(fmt)
    assert fmt.device_error == 0
    assert torch.isnan(buf[n:]).all()
    return o


def check(o, q, k, v, masks, stride_b, stride_h, softcap, slopes, q_start=0, scale=None):
    scale = default_scale(q.shape[3]) if scale is None else scale
    Lq, Lk = q.shape[2], k.shape[2]
    dist = np.abs(np.arange(Lq)[:, None] + q_start - np.arange(Lk)[None, :]).astype(np.float64)
    want, tol = attend_heads(f64(q), f64(k), f64(v), lambda b, h: masks[b * stride_b + h * stride_h] != 0, dist, scale,
                             softcap, slopes, q.dtype)
    err = np.abs(f64(o) - want)
    assert np.all(err <= tol), (float((err / np.maximum(tol, 1e-30)).max()), np.argwhere(err > tol)[:3])


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("option", list(OPTIONS))
@pytest.mark.parametrize("d,which", [(32, ROW), (64, ROW), (128, ROW), (256, ROW), (64, BLOCK), (128, BLOCK)])
def test_options_types_and_head_sizes(gpu_lib, dtype, option, d, which):
    B, H, Hkv, L = 2, 4, 2, 300
    softcap, sl = OPTIONS[option]
    slopes = head_slopes(H) if sl else None
    rng = np.random.default_rng(d)
    masks = (rng.random((B, L, L)) < 0.3).astype(np.uint8)
    masks[0, :, :128] = 1        # full tiles next to partial ones
    masks[1, 5] = 0              # a row without keys
    masks[1, 150:290, 128:] = 0
    q, k, v = tensors(B, H, Hkv, L, L, d, dtype, 1)
    o = run(q, k, v, masks, 1, 0, which, softcap, slopes)
    check(o, q, k, v, masks, 1, 0, softcap, slopes)
    assert torch.all(o[1, :, 5] == 0)


@pytest.mark.parametrize("which", [ROW, BLOCK, AUTO])
@pytest.mark.parametrize("L", [1, 2, 9, 77, 128, 129, 1000])
@pytest.mark.parametrize("d", [64, 128])
def test_lengths(gpu_lib, which, L, d):
    B, H, Hkv = 1, 6, 2
    masks = np.tril(np.ones((1, L, L), dtype=np.uint8))
    q, k, v = tensors(B, H, Hkv, L, L, d, torch.bfloat16, L)
    o = run(q, k, v, masks, 0, 0, which, 25.0, head_slopes(H))
    check(o, q, k, v, masks, 0, 0, 25.0, head_slopes(H))


@pytest.mark.parametrize("which", [ROW, BLOCK, AUTO])
@pytest.mark.parametrize("Lq,Lk", [(1, 700), (37, 500), (200, 130), (130, 200)])
def test_two_lengths_and_a_query_start(gpu_lib, which, Lq, Lk):
    B, H, Hkv, d = 2, 8, 1, 64
    start = Lk - Lq
    masks = (np.arange(Lk)[None, :] <= np.arange(Lq)[:, None] + start).astype(np.uint8)[None]
    q, k, v = tensors(B, H, Hkv, Lq, Lk, d, torch.float16, Lq)
    o = run(q, k, v, masks, 0, 0, which, 0.0, head_slopes(H), q_start=start)
    check(o, q, k, v, masks, 0, 0, 0.0, head_slopes(H), q_start=start)


@pytest.mark.parametrize("group", [1, 2, 8])
@pytest.mark.parametrize("which", [ROW, BLOCK])
def test_groups_and_mask_strides(gpu_lib, group, which):
    B, Hkv, L, d = 2, 2, 260, 128
    H = Hkv * group
    rng = np.random.default_rng(group)
    masks = (rng.random((B * H, L, L)) < 0.2).astype(np.uint8)
    q, k, v = tensors(B, H, Hkv, L, L, d, torch.bfloat16, group)
    o = run(q, k, v, masks, H, 1, which, 30.0, None)
    check(o, q, k, v, masks, H, 1, 30.0, None)


@pytest.mark.parametrize("bm,bn", [(64, 64), (128, 64), (16, 32)])
def test_other_tile_sizes(gpu_lib, bm, bn):
    B, H, Hkv, L, d = 1, 4, 4, 190, 64
    masks = (np.random.default_rng(bm).random((1, L, L)) < 0.4).astype(np.uint8)
    q, k, v = tensors(B, H, Hkv, L, L, d, torch.bfloat16, bn)
    for sync in (True, False):
        o = run(q, k, v, masks, 0, 0, AUTO, 30.0, head_slopes(H), bm, bn, sync=sync)
        check(o, q, k, v, masks, 0, 0, 30.0, head_slopes(H))


@pytest.mark.parametrize("which", [ROW, BLOCK])
@pytest.mark.parametrize("scale,softcap,gain", [(-0.125, 5.0, 2.0), (0.0, 5.0, 2.0), (0.125, 0.5, 2.0), (1.0, 30.0, 8.0),
                                                (1.0, 50.0, 40.0), (-0.125, 0.0, 2.0)])
def test_scales_and_saturated_caps(gpu_lib, which, scale, softcap, gain):
    """Scores far past the cap on both sides, a scale of either sign and none."""
    B, H, L, d = 1, 2, 200, 64
    masks = (np.random.default_rng(5).random((1, L, L)) < 0.6).astype(np.uint8)
    q, k, v = tensors(B, H, H, L, L, d, torch.bfloat16, 3, gain)
    slopes = [0.5, -0.01]
    o = run(q, k, v, masks, 0, 0, which, softcap, slopes, scale=scale)
    check(o, q, k, v, masks, 0, 0, softcap, slopes, scale=scale)


def test_plain_scores_are_the_usual_call(gpu_lib):
    """Without options and with a K/V head each, the call is stof_mha_fwd_cross, bit for bit."""
    B, H, L, d = 1, 2, 300, 64
    masks = (np.random.default_rng(6).random((1, L, L)) < 0.3).astype(np.uint8)
    q, k, v = (t.cuda() for t in tensors(B, H, H, L, L, d, torch.bfloat16, 6))
    fmt, ws, _ = gpu_encode(torch.from_numpy(masks).cuda(), 128, 128)
    for which in (ROW, BLOCK):
        a, b = torch.empty_like(q), torch.empty_like(q)
        stof.stof_mha_fwd_cross(q, k, v, fmt, 0.125, 0, 0, which, a)
        stof.stof_mha_fwd_score(q, k, v, fmt, 0.125, None, 0, 0, which, b)
        assert torch.equal(a, b)


@pytest.mark.parametrize("which", [ROW, BLOCK])
def test_masked_keys_take_no_part_whatever_their_scores(gpu_lib, which):
    """K rows of masked keys hold NaN and infinities (V finite, as documented)."""
    B, H, L, d = 1, 2, 260, 64
    masks = np.tril(np.ones((1, L, L), dtype=np.uint8))
    dead = np.arange(3, L, 7)
    masks[:, :, dead] = 0
    q, k, v = tensors(B, H, H, L, L, d, torch.bfloat16, 8)
    clean = k.clone()
    k[:, :, dead[0::3]] = float("nan")
    k[:, :, dead[1::3]] = float("inf")
    k[:, :, dead[2::3]] = -float("inf")
    for cap, sl in ((30.0, None), (0.0, head_slopes(H)), (30.0, head_slopes(H))):
        o = run(q, k, v, masks, 0, 0, which, cap, sl)
        check(o, q, clean, v, masks, 0, 0, cap, sl)


def test_documents_then_attention_without_a_host_round_trip(gpu_lib):
    """As a prompt's pass calls it: encode the packed documents, attend (AUTO on the unsynced format), captured into
    a graph and replayed on other documents."""
    B, H, Hkv, L, d = 2, 4, 2, 600, 128
    q, k, v = tensors(B, H, Hkv, L, L, d, torch.bfloat16, 9)
    qd, kd, vd = q.cuda(), k.cuda(), v.cuda()
    ids = torch.zeros(B, L, dtype=torch.int32, device="cuda")
    order = torch.arange(L, dtype=torch.int32, device="cuda").repeat(B, 1)
    ws = torch.empty(stof.stof_encode_workspace_bytes(B, L, L, 128, 128), dtype=torch.uint8, device="cuda")
    slopes = torch.tensor(head_slopes(H), dtype=torch.float32, device="cuda")
    o = torch.empty_like(qd)

    def step():
        fmt = stof.stof_encode_documents(ids, ids, order, order, 128, 128, ws)
        stof.stof_mha_fwd_score(qd, kd, vd, fmt, default_scale(d), stof.Score(40.0, slopes), 1, 0, AUTO, o)
        return fmt

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fmt = step()
    for cut in (100, 333):
        doc = np.zeros((B, L), dtype=np.int64)
        doc[0, cut:] = 1
        doc[1, cut + 50:] = 3
        doc[1, 580:] = -1
        ids.copy_(torch.tensor(doc, dtype=torch.int32))
        o.fill_(float("nan"))
        graph.replay()
        stof.stof_format_sync(fmt)
        masks = ((doc[:, :, None] == doc[:, None, :]) & (doc[:, :, None] >= 0) & np.tril(np.ones((L, L), dtype=bool))).astype(np.uint8)
        check(o, q, k, v, masks, 1, 0, 40.0, head_slopes(H))
        assert torch.all(o[1, :, 580:] == 0)


@pytest.mark.parametrize("which", [ROW, BLOCK])
def test_calls_that_share_a_format_may_overlap(gpu_lib, which):
    """Two streams, one format, calls queued behind one another on both; every result as alone."""
    B, H, Hkv, L, d = 1, 8, 2, 1500, 64
    masks = np.tril(np.ones((1, L, L), dtype=np.uint8))
    fmt, ws, _ = gpu_encode(torch.from_numpy(masks).cuda(), 128, 128)
    slopes = torch.tensor(head_slopes(H), dtype=torch.float32, device="cuda")
    sets = [[t.cuda() for t in tensors(B, H, Hkv, L, L, d, torch.bfloat16, seed)] for seed in (20, 21)]
    scores = [stof.Score(30.0), stof.Score(0.0, slopes)]
    want, got = ([torch.full_like(s[0], float("nan")) for s in sets] for _ in range(2))
    for (q, k, v), sc, o in zip(sets, scores, want):
        stof.stof_mha_fwd_score(q, k, v, fmt, 0.125, sc, 0, 0, which, o)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(6):
        for (q, k, v), sc, o, s in zip(sets, scores, got, streams):
            stof.stof_mha_fwd_score(q, k, v, fmt, 0.125, sc, 0, 0, which, o, stream=s)
    torch.cuda.synchronize()
    stof.stof_format_sync(fmt)
    assert fmt.device_error == 0
    for a, b in zip(want, got):
        assert torch.equal(a, b) and torch.isfinite(a.float()).all()


@pytest.mark.parametrize("option", list(OPTIONS))
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("H,L,Lk", [(1, 130, 4500), (1, 1100, 1100), (2, 1500, 1300), (5, 1024, 700), (160, 300, 300)])
def test_few_query_tiles_share_out_their_keys(gpu_lib, option, d, H, L, Lk):
    """Few query tiles: several workers take parts of one tile's keys and merge them; many: none does.  Rows that see
    nothing, parts without tiles (the mask's lower rows list few), tiles past the last row."""
    softcap, sl = OPTIONS[option]
    slopes = head_slopes(H) if sl else None
    rng = np.random.default_rng(H + L)
    masks = (rng.random((1, L, Lk)) < 0.4).astype(np.uint8)
    masks[0, :, 256:512] = 1
    masks[0, 5] = 0
    masks[0, :128, 640:] = 0
    q, k, v = tensors(1, H, 1, L, Lk, d, torch.bfloat16, 31)
    o = run(q, k, v, masks, 0, 0, BLOCK, softcap, slopes, q_start=Lk - L)
    heads = sorted({0, H // 2, H - 1})
    check(o[:, heads], q[:, heads], k, v, masks, 0, 0, softcap, None if slopes is None else [slopes[h] for h in heads],
          q_start=Lk - L)
    assert torch.all(o[0, :, 5] == 0)
    again = run(q, k, v, masks, 0, 0, BLOCK, softcap, slopes, q_start=Lk - L)
    assert torch.equal(o, again)


def test_shared_out_keys_in_a_graph_beside_another_stream(gpu_lib):
    """Calls that share out their keys among several workers, captured, replayed on two streams at once."""
    H, L, d = 1, 1500, 128
    masks = np.tril(np.ones((1, L, L), dtype=np.uint8))
    fmt, ws, _ = gpu_encode(torch.from_numpy(masks).cuda(), 128, 128)
    sets = [[t.cuda() for t in tensors(1, H, 1, L, L, d, torch.bfloat16, seed)] for seed in (40, 41)]
    outs = [torch.full_like(s[0], float("nan")) for s in sets]
    graphs = []
    for (q, k, v), o in zip(sets, outs):
        stof.stof_mha_fwd_score(q, k, v, fmt, 0.1, stof.Score(30.0), 0, 0, BLOCK, o)
        torch.cuda.synchronize()
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            for _ in range(4):
                stof.stof_mha_fwd_score(q, k, v, fmt, 0.1, stof.Score(30.0), 0, 0, BLOCK, o)
        o.fill_(float("nan"))
    streams = [torch.cuda.Stream() for _ in graphs]
    torch.cuda.synchronize()
    for _ in range(3):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for (q, k, v), o in zip(sets, outs):
        check(o, q.cpu(), k.cpu(), v.cpu(), masks, 0, 0, 30.0, None, scale=0.1)
