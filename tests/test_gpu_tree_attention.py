"""stof_tree_attn_fwd against the definition in 64 bits
(tests/scored_reference.py derives the tolerance): decoding, trees, ragged
requests, long and empty caches, unused rows that hold NaN, score options,
bad lengths, graphs and streams."""
import numpy as np
import pytest
import torch

from sparse_mask_transformer_gb300 import stof
from tests.scored_reference import attend, default_scale, f64, head_slopes

pytestmark = pytest.mark.gpu


def random_trees(rng, B, T, reach=5):
    """Ancestor matrices [B, T, T] (self included) and depths [B, T]."""
    sees, depth = np.zeros((B, T, T), dtype=bool), np.zeros((B, T), dtype=np.int64)
    for t in range(T):
        if t:
            parent = rng.integers(max(0, t - reach), t, B)
            sees[:, t] = sees[np.arange(B), parent]
            depth[:, t] = depth[np.arange(B), parent] + 1
        sees[:, t, t] = True
    return sees, depth


def bits_of(sees):
    B, T, _ = sees.shape
    wide = np.zeros((B, T, -(-T // 32) * 32), dtype=bool)
    wide[..., :T] = sees
    return torch.tensor(np.packbits(wide, axis=-1, bitorder="little").view("<i4").copy(), device="cuda")


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


class Case:
    def __init__(self, B, H, Hkv, T, d, lens, dtype=torch.bfloat16, counts=None, sees="tree", softcap=0.0, slopes=None,
                 seed=0, slack=37, scale=None):
        rng = np.random.default_rng(seed)
        self.B, self.H, self.Hkv, self.T, self.d, self.dtype = B, H, Hkv, T, d, dtype
        self.lens = [int(n) for n in lens]
        self.counts = [T] * B if counts is None else [int(n) for n in counts]
        self.cap = max(self.lens) + T + slack
        self.scale = default_scale(d) if scale is None else scale
        self.softcap, self.slopes = softcap, slopes
        tree, dep = random_trees(rng, B, T)
        if isinstance(sees, np.ndarray):
            tree = sees
        self.chain = isinstance(sees, str) and sees == "chain"
        self.sees = np.tile(np.tril(np.ones((T, T), dtype=bool)), (B, 1, 1)) if self.chain else tree
        self.positions = np.array(self.lens)[:, None] + (np.arange(T)[None, :] if self.chain else dep)
        g = torch.Generator().manual_seed(seed)
        self.q = (torch.randn(B, H, T, d, generator=g) * 2).to(dtype)
        self.k, self.v = (torch.randn(B, Hkv, self.cap, d, generator=g).to(dtype) for _ in range(2))
        for b in range(B):  # rows that no token has written yet
            end = self.lens[b] + self.counts[b]
            self.k[b, :, end:] = float("nan")
            self.v[b, :, end:] = float("inf") if b % 2 else float("nan")
            self.q[b, :, self.counts[b]:] = float("nan")

    def args(self):
        return dict(q=self.q.cuda(), k=self.k.cuda(), v=self.v.cuda(), lens=i32(self.lens), counts=i32(self.counts),
                    tree=None if self.chain else bits_of(self.sees), positions=None if self.chain else i32(self.positions),
                    slopes=None if self.slopes is None else torch.tensor(self.slopes, dtype=torch.float32, device="cuda"),
                    ws=torch.full((stof.stof_tree_attn_workspace_bytes(self.B, self.H, self.Hkv, self.T, self.d),), 0xCD,
                                  dtype=torch.uint8, device="cuda"))

    def call(self, a, o, err=None, stream=None):
        stof.stof_tree_attn_fwd(a["q"], a["k"], a["v"], a["lens"], self.scale, o, a["ws"], tree=a["tree"], counts=a["counts"],
                                positions=a["positions"], score=stof.Score(self.softcap, a["slopes"]), device_error=err,
                                stream=stream)

    def check(self, o, planes=None):
        for b in range(self.B):
            n, c = self.lens[b], self.counts[b]
            assert torch.all(o[b, :, c:] == 5.0), "rows past the request's tokens were written"
            valid = np.concatenate([np.ones((c, n), dtype=bool), self.sees[b, :c, :c]], axis=1)
            at = np.concatenate([np.arange(n), self.positions[b, :c]])
            dist = np.abs(self.positions[b, :c, None] - at[None, :]).astype(np.float64)
            k, v = f64(self.k[b, :, :n + c]), f64(self.v[b, :, :n + c])
            for h in range(self.H):
                if planes is not None and (b, h) not in planes or c == 0:
                    continue
                g = h // (self.H // self.Hkv)
                want, tol = attend(f64(self.q[b, h, :c]), k[g], v[g], valid, dist, self.scale, self.softcap,
                                   0.0 if self.slopes is None else self.slopes[h], self.dtype)
                err = np.abs(f64(o[b, h, :c]) - want)
                assert np.all(err <= tol), (b, h, float((err / np.maximum(tol, 1e-30)).max()))

    def run(self, planes=None):
        a = self.args()
        n = self.q.numel()
        buf = torch.full((n + 4096,), 5.0, dtype=self.dtype, device="cuda")
        o, err = buf[:n].view(self.q.shape), torch.zeros(1, dtype=torch.int64, device="cuda")
        self.call(a, o, err)
        torch.cuda.synchronize()
        assert err.item() == 0 and torch.all(buf[n:] == 5.0)
        self.check(o, planes)
        return a, o


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("length", [0, 1, 127, 128, 129, 1000])
def test_one_token(gpu_lib, dtype, d, length):
    Case(1, 8, 2, 1, d, [length], dtype, sees="chain", seed=length).run()


@pytest.mark.parametrize("T,H,Hkv", [(1, 4, 4), (3, 6, 1), (16, 8, 2), (31, 8, 1), (33, 4, 1), (64, 16, 2), (100, 5, 5), (257, 2, 2),
                                     (8, 4, 1), (16, 2, 1), (33, 1, 1), (130, 9, 1)])
@pytest.mark.parametrize("d", [64, 128])
def test_trees_and_groups(gpu_lib, T, H, Hkv, d):
    """Rows of a group that fill part of a tile, one tile and several; bitsets of one and several words."""
    Case(3, H, Hkv, T, d, [0, 200, 511], seed=T).run()


@pytest.mark.parametrize("softcap,sl", [(30.0, False), (0.0, True), (20.0, True)])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("sees", ["tree", "chain"])
def test_score_options(gpu_lib, softcap, sl, d, sees):
    Case(2, 8, 4, 9, d, [300, 77], torch.float16, softcap=softcap, slopes=head_slopes(8) if sl else None, seed=1,
         sees=sees).run()


def test_ragged_batch(gpu_lib):
    lens = [0, 5, 1023, 128, 700, 0, 64, 2000, 1]
    counts = [1, 7, 3, 0, 7, 2, 7, 1, 6]
    Case(9, 6, 2, 7, 64, lens, counts=counts, softcap=25.0, slopes=head_slopes(6), seed=2).run()
    Case(9, 6, 2, 7, 128, lens, counts=counts, seed=3).run()


def test_many_requests(gpu_lib):
    """More (request, head) pairs than there are SMs, lengths far apart."""
    rng = np.random.default_rng(4)
    lens = rng.integers(0, 900, 450)
    lens[7] = 6000
    Case(450, 2, 2, 2, 64, lens, counts=rng.integers(0, 3, 450), seed=4).run()


def test_more_row_tiles_than_go_together(gpu_lib):
    """Nine and more row tiles per K/V head: two groups, the last one smaller; several shares and requests."""
    Case(2, 10, 1, 116, 64, [0, 700], seed=21).run(planes={(0, 0), (0, 9), (1, 3), (1, 9)})
    Case(1, 19, 1, 128, 128, [3000], seed=22).run(planes={(0, 0), (0, 7), (0, 8), (0, 18)})


def test_a_long_cache(gpu_lib):
    Case(1, 8, 1, 16, 128, [70001], seed=5).run(planes={(0, 0), (0, 7)})


def test_a_cache_past_32_bit_offsets(gpu_lib):
    """2^31 elements and more in front of the last request's rows."""
    B, Hkv, d, T = 3, 2, 128, 2
    cap = (1 << 31) // (Hkv * d) // 2 + 1000  # two requests: over 2^31 elements
    k = torch.zeros(B, Hkv, cap, d, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    small = Case(1, 4, Hkv, T, d, [300], seed=6)
    n = 300 + T
    k[2, :, :n], v[2, :, :n] = small.k[0, :, :n].cuda(), small.v[0, :, :n].cuda()
    a = small.args()
    q = torch.zeros(B, 4, T, d, dtype=torch.bfloat16, device="cuda")
    q[2] = a["q"][0]
    o = torch.full_like(q, 5.0)
    ws = torch.empty(stof.stof_tree_attn_workspace_bytes(B, 4, Hkv, T, d), dtype=torch.uint8, device="cuda")
    stof.stof_tree_attn_fwd(q, k, v, i32([0, 1, 300]), small.scale, o, ws, tree=a["tree"].repeat(B, 1, 1))
    small.check(o[2:])
    assert torch.all(o[:2] == 0)


def test_rows_that_see_nothing_and_bits_past_the_count(gpu_lib):
    T = 40
    sees = np.zeros((2, T, T), dtype=bool)
    sees[1] = True                      # every bit, those past the request's tokens included
    c = Case(2, 4, 2, T, 64, [0, 90], counts=[T, 11], sees=sees, seed=7)
    a, o = c.run()
    assert torch.all(o[0] == 0)


@pytest.mark.parametrize("scale,softcap", [(-0.1, 0.0), (0.0, 0.0), (-0.1, 10.0), (2.0, 10.0)])
def test_scales(gpu_lib, scale, softcap):
    Case(1, 4, 2, 5, 64, [200], torch.float16, scale=scale, softcap=softcap, seed=8).run()


def test_bad_lengths_are_skipped_and_reported(gpu_lib):
    c = Case(5, 4, 2, 3, 64, [10, 20, 30, 40, 50], seed=9)
    for name, bad in (("lens", [-1, 20, c.cap - 2, 2 ** 31 - 1, 50]), ("counts", [4, 3, -1, 2 ** 31 - 1, 3])):
        a = c.args()
        a[name] = i32(bad)
        o = torch.full(c.q.shape, 5.0, dtype=c.dtype, device="cuda")
        err = torch.zeros(1, dtype=torch.int64, device="cuda")
        c.call(a, o, err)
        assert err.item() == stof.STOF_DEVERR_BAD_LENGTH
        for b in (0, 2, 3):
            assert torch.all(o[b] == 5.0)
        good = torch.full_like(o, 5.0)
        c.call(c.args(), good)
        assert torch.equal(o[1], good[1]) and torch.equal(o[4], good[4])
        c.call(a, o)  # without an error word


def test_graph_replay_follows_the_lengths_and_repeats_bit_for_bit(gpu_lib):
    c = Case(3, 8, 2, 6, 128, [400, 900, 20], seed=10)
    a = c.args()
    a["k"][torch.isnan(a["k"])] = 0.0
    a["v"][~torch.isfinite(a["v"])] = 0.0
    o = torch.full(c.q.shape, 5.0, dtype=c.dtype, device="cuda")
    c.call(a, o)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.call(a, o)
    for lens in ([400, 900, 20], [0, 130, 920], [128, 128, 128]):
        a["lens"].copy_(i32(lens))
        a["ws"].fill_(0xEE)  # nothing is kept in the workspace
        o.fill_(float("nan"))
        graph.replay()
        want = torch.full_like(o, 5.0)
        c.call(a, want)
        torch.cuda.synchronize()
        assert torch.equal(o, want) and torch.isfinite(o.float()).all()


def test_two_streams_with_their_own_workspaces(gpu_lib):
    cs = [Case(2, 8, 2, 4, 128, [3000, 100], seed=s) for s in (11, 12)]
    aa = [c.args() for c in cs]
    oo = [torch.full(c.q.shape, 5.0, dtype=c.dtype, device="cuda") for c in cs]
    streams = [torch.cuda.Stream() for _ in cs]
    torch.cuda.synchronize()
    for _ in range(5):
        for c, a, o, s in zip(cs, aa, oo, streams):
            c.call(a, o, stream=s)
    torch.cuda.synchronize()
    for c, o in zip(cs, oo):
        c.check(o)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("H", [2, 40])
def test_far_positions_are_subtracted_exactly(gpu_lib, d, H):
    """Drafted tokens at positions near 2^31, whose neighbours fp32 cannot tell apart; and at the two ends of 32 bits."""
    T = 12
    c = Case(2, H, 1, T, d, [0, 0], torch.float16, slopes=head_slopes(H), seed=13)
    c.positions = 2_000_000_000 + np.arange(T)[None, :] + np.array([[0], [77]])
    c.run()
    c = Case(1, H, 1, T, d, [0], torch.float16, slopes=[2.0 ** -31] * H, seed=14)
    c.positions = np.where(np.arange(T) % 3 == 0, -2 ** 31, 2 ** 31 - 1 - np.arange(T))[None, :]
    c.run()


def test_the_most_drafted_tokens(gpu_lib):
    T = stof.STOF_TREE_MAX_TOKENS
    Case(1, 2, 1, T, 64, [100], seed=15, counts=[T - 1]).run()
    Case(1, 1, 1, T, 128, [33], seed=16, sees="chain").run()


def test_two_graphs_that_share_a_workspace_in_turn(gpu_lib):
    cs = [Case(2, 8, 2, 4, 64, [1000, 100], seed=17), Case(2, 8, 2, 4, 64, [3, 2500], seed=18)]
    aa = [c.args() for c in cs]
    oo = [torch.full(c.q.shape, 5.0, dtype=c.dtype, device="cuda") for c in cs]
    graphs = []
    for c, a, o in zip(cs, aa, oo):
        a["ws"] = aa[0]["ws"]
        c.call(a, o)
        torch.cuda.synchronize()
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            c.call(a, o)
    for o in oo:
        o.fill_(5.0)
    for _ in range(3):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    for c, o in zip(cs, oo):
        c.check(o)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("softcap,sl", [(0.0, False), (0.0, True), (200.0, False)])
def test_scores_that_rise_far_above_the_first_tiles(gpu_lib, dtype, softcap, sl):
    """The tiles go from the last key to the first: keys ever earlier have scores ever higher (by 15 nats a tile of 64 keys,
    a step of 60 among them), so that a reference taken from the tiles before is passed by more than P can hold."""
    T, H, n = 3, 2, 700
    c = Case(1, H, 1, T, 128, [n], dtype, softcap=softcap, slopes=head_slopes(H) if sl else None, seed=19, scale=1.0)
    level = torch.zeros(n + T)
    for at in range(0, n, 64):
        level[at:at + 64] = 15.0 * ((n - at) // 64) + (60.0 if at < 256 else 0.0)
    c.q[:] = 0.0
    c.q[..., 0] = 1.0                                      # score = K's first element, exact in both types
    c.k[0, 0, :n + T, 0] = level.to(dtype)
    c.k[0, 0, :n + T, 1:] = 0.0
    c.run()
