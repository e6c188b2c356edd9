"""stof_cache_keep and stof_cache_fork against row by row copies, bit for bit:
types, sizes and layers, paths that overlap the rows they move to, bad
requests and slots, rows that stay, streams and graphs."""
import numpy as np
import pytest
import torch

from sparse_mask_transformer_gb300 import stof

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def make(n, slots, heads, rows, d, dtype=torch.bfloat16, seed=0):
    """Any 16-bit patterns, NaN among them, compared as integers; with a guard behind each."""
    g = torch.Generator().manual_seed(seed)
    size = slots * heads * rows * d
    raw = [torch.randint(-2 ** 15, 2 ** 15, (size + 512,), generator=g, dtype=torch.int16).cuda() for _ in range(n)]
    return raw, [r[:size].view(slots, heads, rows, d).view(dtype) for r in raw]


def bits(t):
    return t.view(torch.int16).cpu()


def random_paths(rng, slots, T, gaps=True):
    paths = []
    for _ in range(slots):
        k = int(rng.integers(0, T + 1))
        paths.append(sorted(rng.choice(T, k, replace=False).tolist()) if gaps else list(range(k)))
    return paths


def padded(paths, T):
    return i32([p + [-5] * (T - len(p)) for p in paths])  # what is behind the kept ones is not used


@pytest.mark.parametrize("d", [8, 64, 72, 128, 256, 1024])
@pytest.mark.parametrize("T", [1, 2, 9, 64, 200])
def test_keep(gpu_lib, d, T):
    n, slots, heads, rows = 3, 5, 2, T + 60
    rng = np.random.default_rng(T * d)
    raw, c = make(n, slots, heads, rows, d, seed=T)
    want = [bits(r).clone() for r in raw]
    lens = rng.integers(0, rows - T + 1, slots)
    lens[0], lens[1] = 0, rows - T
    paths = random_paths(rng, slots, T)
    paths[2], paths[3] = list(range(T)), [T - 1]          # all of them (already in place); the last alone
    new = i32([-9] * slots)
    err = torch.zeros(1, dtype=torch.int64, device="cuda")
    stof.stof_cache_keep(stof.Caches(c), i32(lens), padded(paths, T), i32([len(p) for p in paths]), new, err)
    for w in want:
        v = w[:slots * heads * rows * d].view(slots, heads, rows, d)
        before = v.clone()
        for b, p in enumerate(paths):
            for i, u in enumerate(p):
                v[b, :, lens[b] + i] = before[b, :, lens[b] + u]
    assert err.item() == 0
    assert new.tolist() == [int(a) + len(p) for a, p in zip(lens, paths)]
    for r, w in zip(raw, want):
        assert torch.equal(bits(r), w)


def test_keep_the_longest_path(gpu_lib):
    T, heads, rows, d = stof.STOF_TREE_MAX_TOKENS, 1, 1100, 16
    raw, c = make(1, 1, heads, rows, d, seed=3)
    path = sorted(np.random.default_rng(3).choice(T, 700, replace=False).tolist())
    before = bits(c[0]).clone()
    stof.stof_cache_keep(stof.Caches(c), i32([76]), padded([path], T), i32([700]))
    want = before.clone()
    want[0, :, 76:776] = before[0, :, [76 + u for u in path]]
    assert torch.equal(bits(c[0]), want)


def test_keep_skips_bad_requests(gpu_lib):
    T, slots, heads, rows, d = 6, 9, 2, 40, 64
    raw, c = make(2, slots, heads, rows, d, torch.float16, seed=4)
    before = [bits(t).clone() for t in c]
    lens = [10, -1, 41, 36, 2 ** 31 - 1, 10, 10, 10, 34]
    paths = [[1, 3], [1], [], [1, 4], [0], [3, 3], [4, 2], [-1, 5], [2, 5]]
    kept = [2, 1, 0, 2, 1, 2, 2, 2, 2]
    new = i32([-9] * slots)
    err = torch.zeros(1, dtype=torch.int64, device="cuda")
    stof.stof_cache_keep(stof.Caches(c), i32(lens), padded(paths, T), i32(kept), new, err)
    assert err.item() == stof.STOF_DEVERR_BAD_LENGTH
    assert new.tolist() == [12, -9, -9, -9, -9, -9, -9, -9, 36]
    for t, w in zip(c, before):
        v = w.clone()
        v[0, :, 10], v[0, :, 11] = w[0, :, 11], w[0, :, 13]
        v[8, :, 34], v[8, :, 35] = w[8, :, 36], w[8, :, 39]
        assert torch.equal(bits(t), v)
    for bad in (-1, T + 1, 2 ** 31 - 1, -2 ** 31):       # kept out of range; and no error word to tell
        stof.stof_cache_keep(stof.Caches(c), i32([10] * slots), padded([[1]] * slots, T), i32([bad] * slots), new)
    err.zero_()
    stof.stof_cache_keep(stof.Caches(c), i32([10] * slots), i32([[T, 0, 0, 0, 0, 0]] * slots), i32([1] * slots), None, err)
    assert err.item() == stof.STOF_DEVERR_BAD_LENGTH


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("n,slots,heads,rows,d", [(1, 1, 1, 1, 8), (2, 7, 3, 33, 64), (5, 12, 4, 130, 128), (2, 3, 2, 2000, 72),
                                                 (40, 2, 2, 50, 256)])
def test_fork_into_other_caches(gpu_lib, dtype, n, slots, heads, rows, d):
    rng = np.random.default_rng(rows)
    _, a = make(n, slots, heads, rows, d, dtype, seed=5)
    to_slots, to_rows = slots + 2, rows + 3
    raw, b = make(n, to_slots, heads, to_rows, d, dtype, seed=6)
    lens = rng.integers(0, rows + 1, slots)
    lens[0] = rows
    src = rng.integers(-1, slots, to_slots)
    src[-1], src[0] = -2 ** 31, 0
    new, err = i32([-9] * to_slots), torch.zeros(1, dtype=torch.int64, device="cuda")
    want = [bits(r).clone() for r in raw]
    from_before = [bits(t).clone() for t in a]
    stof.stof_cache_fork(stof.Caches(a), stof.Caches(b), i32(src), i32(lens), new, err)
    assert err.item() == 0
    assert new.tolist() == [int(lens[s]) if s >= 0 else -9 for s in src]
    for w, f in zip(want, from_before):
        v = w[:to_slots * heads * to_rows * d].view(to_slots, heads, to_rows, d)
        for slot, s in enumerate(src):
            if s >= 0:
                v[slot, :, :lens[s]] = f[s, :, :lens[s]]
    for r, w in zip(raw, want):
        assert torch.equal(bits(r), w)
    for t, f in zip(a, from_before):
        assert torch.equal(bits(t), f)


def test_fork_inside_the_same_caches(gpu_lib):
    slots, heads, rows, d = 6, 3, 700, 128
    raw, c = make(4, slots, heads, rows, d, seed=7)
    want = [bits(r).clone() for r in raw]
    lens = i32([650, 3, 77, 0, 5, 700])
    src = [0, 0, 5, -1, 3, 5]                            # 0 and 5 stay and are copied from; 3 has no rows
    stof.stof_cache_fork(stof.Caches(c), stof.Caches(c), i32(src), lens, lens)
    assert lens.tolist() == [650, 650, 700, 0, 0, 700]
    for r, w in zip(raw, want):
        v = w[:slots * heads * rows * d].view(slots, heads, rows, d)
        v[1, :, :650], v[2] = v[0, :, :650], v[5]
        assert torch.equal(bits(r), w)


def test_fork_skips_bad_slots(gpu_lib):
    slots, heads, rows, d = 6, 2, 50, 64
    _, a = make(2, slots, heads, rows, d, seed=8)
    _, b = make(2, 4, heads, 40, d, seed=9)
    before = [bits(t).clone() for t in b]
    err, new = torch.zeros(1, dtype=torch.int64, device="cuda"), i32([-9] * 4)
    # a slot that is not there, a length below 0, one above the source's rows and one above the destination's
    for src, lens, good in (([6, 1, 2 ** 31 - 1, 1], [9, 8, 7, 6, 5, 4], (1, 3)), ([0, 1, 0, 2], [-1, 8, 7, 6, 5, 4], (1, 3)),
                            ([0, 1, 0, 2], [51, 8, 7, 6, 5, 4], (1, 3)), ([0, 1, 0, 2], [41, 8, 40, 6, 5, 4], (1, 3))):
        err.zero_()
        new.fill_(-9)
        stof.stof_cache_fork(stof.Caches(a), stof.Caches(b), i32(src), i32(lens), new, err)
        assert err.item() == stof.STOF_DEVERR_BAD_LENGTH
        assert new.tolist() == [lens[s] if slot in good else -9 for slot, s in enumerate(src)]
        for t, f, w in zip(b, a, before):
            for slot in range(4):
                if slot in good:
                    w[slot, :, :lens[src[slot]]] = bits(f)[src[slot], :, :lens[src[slot]]]
            assert torch.equal(bits(t), w)
    # in the same caches: a chain 0 -> 1 -> 2, a swap of 3 and 4; 5 <- 0 is fine
    before = [bits(t).clone() for t in a]
    err.zero_()
    lens = i32([50, 49, 48, 47, 46, 45])
    stof.stof_cache_fork(stof.Caches(a), stof.Caches(a), i32([-1, 0, 1, 4, 3, 0]), lens, lens, err)
    assert err.item() == stof.STOF_DEVERR_BAD_LENGTH
    assert lens.tolist() == [50, 49, 49, 47, 46, 50]
    for t, w in zip(a, before):
        w[2, :, :49], w[5] = w[1, :, :49], w[0]
        assert torch.equal(bits(t), w)


def test_rows_past_32_bit_offsets(gpu_lib):
    """2^31 elements and more in front of the rows that move."""
    slots, heads, d = 3, 2, 128
    rows = (1 << 31) // (heads * d) // 2 + 1000
    c = torch.zeros(slots, heads, rows, d, dtype=torch.bfloat16, device="cuda")
    c[2, :, rows - 8:] = torch.arange(8, device="cuda", dtype=torch.bfloat16)[None, :, None]
    stof.stof_cache_keep(stof.Caches([c]), i32([0, 0, rows - 8]), i32([[0] * 8, [0] * 8, [1, 3, 6, 7, 0, 0, 0, 0]]), i32([0, 0, 4]))
    assert c[2, :, rows - 8:, 5].tolist() == [[1, 3, 6, 7, 4, 5, 6, 7]] * heads
    small = torch.full((2, heads, rows, d), 9.0, dtype=torch.bfloat16, device="cuda")
    stof.stof_cache_fork(stof.Caches([c]), stof.Caches([small]), i32([-1, 2]), i32([0, 0, rows]))
    assert torch.equal(small[1], c[2]) and small[0].min().item() == 9.0


def test_capture_and_streams(gpu_lib):
    slots, heads, rows, d, T = 4, 2, 90, 64, 8
    _, a = make(3, slots, heads, rows, d, seed=10)
    _, b = make(3, slots, heads, rows, d, seed=11)
    ca, cb = stof.Caches(a), stof.Caches(b)
    lens, path, kept = i32([3, 50, 7, 80]), i32([[1, 2, 5, 7, 0, 0, 0, 0]] * 4), i32([4, 3, 0, 2])
    new, src, out = i32([0] * 4), i32([1, 1, 3, 0]), i32([0] * 4)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    stof.stof_cache_keep(ca, lens, path, kept, new, stream=side)
    stof.stof_cache_fork(ca, cb, src, new, out, stream=side)
    torch.cuda.synchronize()
    assert out.tolist() == [53, 53, 82, 7]
    for x, y in zip(a, b):
        assert torch.equal(bits(y)[0, :, :53], bits(x)[1, :, :53])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        stof.stof_cache_keep(ca, lens, path, kept, new)
        stof.stof_cache_fork(ca, cb, src, new, out)
    lens.copy_(i32([10, 20, 30, 40]))
    want = [bits(x).clone() for x in a]
    graph.replay()
    torch.cuda.synchronize()
    assert out.tolist() == [23, 23, 42, 14]
    for x, y, w in zip(a, b, want):
        before = w.clone()
        for s, n in enumerate((10, 20, 30, 40)):
            for i in range(int(kept[s])):
                w[s, :, n + i] = before[s, :, n + int(path[s, i])]
        assert torch.equal(bits(x), w)
        assert torch.equal(bits(y)[2, :, :42], w[3, :, :42])


def test_caches_of_different_shapes_are_refused(gpu_lib):
    x = torch.zeros(2, 2, 8, 64, dtype=torch.float16, device="cuda")
    for other in (torch.zeros_like(x, dtype=torch.bfloat16), torch.zeros(2, 2, 9, 64, dtype=torch.float16, device="cuda"),
                  x.transpose(1, 2)[:, :, :2]):
        with pytest.raises(stof.StofError) as e:
            stof.Caches([x, other])
        assert e.value.status == stof.STOF_ERR_SHAPE
    with pytest.raises(stof.StofError):
        stof.Caches([x.float()])
    with pytest.raises(stof.StofError) as e:
        stof.Caches([x, x])
    assert e.value.status == stof.STOF_ERR_INVALID_ARG
    c = stof.Caches([x])
    with pytest.raises(stof.StofError) as e:
        stof.stof_cache_keep(c, i32([0, 0, 0]), i32([[0], [0]]), i32([0, 0]))
    assert e.value.status == stof.STOF_ERR_SHAPE


def test_overlapping_caches_are_refused(gpu_lib):
    c = torch.zeros(6, 2, 8, 64, dtype=torch.float16, device="cuda")
    d = torch.zeros_like(c)
    with pytest.raises(stof.StofError) as e:
        stof.Caches([c[:4], c[2:]])
    assert e.value.status == stof.STOF_ERR_INVALID_ARG
    stof.Caches([c[3:], c[:3]])  # side by side
    src, lens = torch.zeros(6, dtype=torch.int32, device="cuda"), torch.ones(6, dtype=torch.int32, device="cuda")
    with pytest.raises(stof.StofError) as e:
        stof.stof_cache_fork(stof.Caches([c, d]), stof.Caches([d, c]), src, lens)
    assert e.value.status == stof.STOF_ERR_INVALID_ARG
