"""stof_encode_documents against the oracle's brute-force encoding of the
mask its arrays define, bit for bit: packed documents, padding, prefixes,
chunks, two lengths, sides that are not whole tiles, and tile sizes."""
import numpy as np
import pytest
import torch

import oracle
from sparse_mask_transformer_gb300 import stof
from tests.conftest import assert_format_equal

pytestmark = pytest.mark.gpu


def dense(qd, kd, qo, ko):
    m = (qd[:, :, None] == kd[:, None, :]) & (qd[:, :, None] >= 0)
    if qo is not None:
        m &= ko[:, None, :] <= qo[:, :, None]
    return m.astype(np.uint8)


def dev(x):
    return None if x is None else torch.tensor(x, dtype=torch.int32, device="cuda")


def check(qd, kd, qo, ko, bm=128, bn=128):
    (n, lq), lk = qd.shape, kd.shape[1]
    ws = torch.full((stof.stof_encode_workspace_bytes(n, lq, lk, bm, bn),), 0xAB, dtype=torch.uint8, device="cuda")
    fmt = stof.stof_encode_documents(dev(qd), dev(kd), dev(qo), dev(ko), bm, bn, ws)
    stof.stof_format_sync(fmt)
    arrs = {k: v.cpu().numpy() for k, v in stof.format_arrays(fmt, ws).items()}
    arrs["bitmaps"] = arrs["bitmaps"].view("uint64")
    assert_format_equal(fmt, arrs, oracle.encode(dense(qd, kd, qo, ko), bm, bn))


def packed(rng, n, L, docs, pad):
    out = np.full((n, L), -1)
    for m in range(n):
        cuts = np.sort(rng.choice(np.arange(1, max(2, L - pad)), min(docs - 1, max(0, L - pad - 1)), replace=False)) if docs > 1 else []
        for i, (a, e) in enumerate(zip([0, *cuts], [*cuts, L - pad])):
            out[m, a:e] = i * 7
    return out


@pytest.mark.parametrize("L", [1, 7, 8, 100, 128, 333, 1024, 1500])
@pytest.mark.parametrize("bm,bn", [(128, 128), (128, 64), (64, 256), (8, 8), (256, 24)])
def test_causal_documents(gpu_lib, L, bm, bn):
    rng = np.random.default_rng(L + bm)
    d = packed(rng, 2, L, 3 if L > 8 else 1, L // 9)
    order = np.tile(np.arange(L), (2, 1))
    check(d, d, order, order, bm, bn)


@pytest.mark.parametrize("L", [77, 640])
def test_bidirectional_documents_and_no_order(gpu_lib, L):
    d = packed(np.random.default_rng(L), 3, L, 4, 5)
    check(d, d, None, None)
    z = np.zeros_like(d)
    check(d, d, z, z)


def test_prefix_sees_and_is_seen(gpu_lib):
    L = 500
    d = packed(np.random.default_rng(1), 2, L, 2, 0)
    order = np.tile(np.arange(L), (2, 1))
    ko = order.copy()
    ko[0, :130] = -2 ** 31
    ko[1, 20:300] = -1
    check(d, d, order, ko)


def test_last_queries_of_a_longer_sequence(gpu_lib):
    lq, lk = 200, 900
    kd = packed(np.random.default_rng(2), 1, lk, 2, 3)
    check(kd[:, lk - lq:], kd, np.arange(lk - lq, lk)[None], np.arange(lk)[None])


def test_any_numbers(gpu_lib):
    """Shuffled documents (no runs), extreme numbers and orders, all padding, chunked order."""
    rng = np.random.default_rng(3)
    lq, lk = 150, 260
    big = np.array([0, 1, 2 ** 31 - 1, -1, -2, -3, -2 ** 31])
    check(rng.choice(big, (2, lq)), rng.choice(big, (2, lk)), rng.choice(big, (2, lq)), rng.choice(big, (2, lk)))
    none = np.full((1, 300), -1)
    check(none, none, None, None)
    d, chunk = np.zeros((1, 512), dtype=int), (np.arange(512) // 48)[None]
    check(d, d, chunk, chunk)


def test_a_reused_workspace_and_graph_replay(gpu_lib):
    """The encoder clears what it needs: replayed on changed arrays it gives the new format."""
    L = 700
    rng = np.random.default_rng(4)
    ids = dev(packed(rng, 2, L, 3, 10))
    order = dev(np.tile(np.arange(L), (2, 1)))
    ws = torch.empty(stof.stof_encode_workspace_bytes(2, L, L, 128, 128), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fmt = stof.stof_encode_documents(ids, ids, order, order, 128, 128, ws)
    for docs in (2, 6):
        d = packed(rng, 2, L, docs, 0)
        ids.copy_(dev(d))
        graph.replay()
        stof.stof_format_sync(fmt)
        arrs = {k: v.cpu().numpy() for k, v in stof.format_arrays(fmt, ws).items()}
        arrs["bitmaps"] = arrs["bitmaps"].view("uint64")
        o = np.tile(np.arange(L), (2, 1))
        assert_format_equal(fmt, arrs, oracle.encode(dense(d, d, o, o), 128, 128))


@pytest.mark.parametrize("n,L,bm,bn", [(18, 1032, 8, 8), (520, 130, 16, 128)])
def test_more_chunks_than_two_kernels_take(gpu_lib, n, L, bm, bn):
    """Over 4096 chunks: the single-pass encoder."""
    d = packed(np.random.default_rng(n), n, L, 3, 4)
    order = np.tile(np.arange(L), (n, 1))
    check(d, d, order, order, bm, bn)


@pytest.mark.parametrize("bm,bn", [(256, 256), (256, 24), (128, 128), (8, 8)])
def test_chunks_in_which_no_group_settles_a_word(gpu_lib, bm, bn):
    rng = np.random.default_rng(bm + bn)
    lq, lk = 300, 1100
    check(rng.integers(0, 3, (2, lq)), rng.integers(0, 3, (2, lk)), rng.integers(0, 9, (2, lq)), rng.integers(0, 9, (2, lk)), bm, bn)
