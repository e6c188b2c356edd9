"""stof_prefix_attn_fwd against the definition in 64 bits
(tests/scored_reference.py derives the tolerance; merging a row's parts adds
fp32 operations of the kind its last term counts): groups of requests, tiles of
several requests and requests of several tiles, empty prefixes, prefixes alone
(cross attention), trees, score options, unused rows that hold NaN, bad
lengths, graphs and streams."""
import numpy as np
import pytest
import torch

from sparse_mask_transformer_gb300 import stof
from tests.scored_reference import attend, default_scale, f64, head_slopes
from tests.test_gpu_tree_attention import bits_of, i32, random_trees

pytestmark = pytest.mark.gpu


class Case:
    def __init__(self, n, H, Hkv, T, d, plens, lens, dtype=torch.bfloat16, counts=None, sees="tree", softcap=0.0, slopes=None,
                 seed=0, slack=37, scale=None):
        """n requests of each prefix; lens None: the prefixes alone."""
        rng = np.random.default_rng(seed)
        self.NP, self.n, self.H, self.Hkv, self.T, self.d, self.dtype = len(plens), n, H, Hkv, T, d, dtype
        B = self.B = self.NP * n
        self.plens, self.cross = [int(x) for x in plens], lens is None
        self.lens = [0] * B if lens is None else [int(x) for x in lens]
        self.counts = [T] * B if counts is None else [int(x) for x in counts]
        self.pcap, self.cap = max(1, max(self.plens) + slack), max(self.lens) + T + slack
        self.scale = default_scale(d) if scale is None else scale
        self.softcap, self.slopes = softcap, slopes
        tree, depth = random_trees(rng, B, T)
        if isinstance(sees, np.ndarray):
            tree = sees
        self.chain = isinstance(sees, str) and sees == "chain"
        self.sees = np.tile(np.tril(np.ones((T, T), dtype=bool)), (B, 1, 1)) if self.chain else tree
        start = np.repeat(self.plens, n) + np.array(self.lens)
        self.positions = start[:, None] + (np.arange(T)[None, :] if self.chain else depth)
        g = torch.Generator().manual_seed(seed)
        self.q = (torch.randn(B, H, T, d, generator=g) * 2).to(dtype)
        self.kp, self.vp = (torch.randn(self.NP, Hkv, self.pcap, d, generator=g).to(dtype) for _ in range(2))
        self.k, self.v = (torch.randn(B, Hkv, self.cap, d, generator=g).to(dtype) for _ in range(2))
        for p, m in enumerate(self.plens):  # rows that nothing has written yet
            self.kp[p, :, m:] = float("nan")
            self.vp[p, :, m:] = float("nan") if p % 2 else float("inf")
        for b in range(B):
            end = self.lens[b] + self.counts[b]
            self.k[b, :, end:] = float("nan")
            self.v[b, :, end:] = float("inf") if b % 2 else float("nan")
            self.q[b, :, self.counts[b]:] = float("nan")

    def args(self):
        own = not self.cross
        given = own and not self.chain
        return dict(q=self.q.cuda(), kp=self.kp.cuda(), vp=self.vp.cuda(), plens=i32(self.plens),
                    k=self.k.cuda() if own else None, v=self.v.cuda() if own else None, lens=i32(self.lens) if own else None,
                    counts=i32(self.counts), tree=bits_of(self.sees) if given else None,
                    positions=i32(self.positions) if given else None,
                    slopes=None if self.slopes is None else torch.tensor(self.slopes, dtype=torch.float32, device="cuda"),
                    ws=torch.full((stof.stof_prefix_attn_workspace_bytes(self.B, self.NP, self.H, self.Hkv, self.T, self.d),),
                                  0xCD, dtype=torch.uint8, device="cuda"))

    def call(self, a, o, err=None, stream=None):
        stof.stof_prefix_attn_fwd(a["q"], a["kp"], a["vp"], a["plens"], a["k"], a["v"], a["lens"], self.scale, o, a["ws"],
                                  tree=a["tree"], counts=a["counts"], positions=a["positions"],
                                  score=stof.Score(self.softcap, a["slopes"]), device_error=err, stream=stream)

    def check(self, o, planes=None):
        o = o.cpu()
        for b in range(self.B):
            p, n, c = b // self.n, self.lens[b], self.counts[b]
            m = self.plens[p]
            assert torch.all(o[b, :, c:] == 5.0), "rows past the request's tokens were written"
            k, v = f64(self.kp[p, :, :m]), f64(self.vp[p, :, :m])
            valid = np.ones((c, m), dtype=bool)
            dist = np.zeros((c, m))
            if not self.cross:
                k = np.concatenate([k, f64(self.k[b, :, :n + c])], axis=1)
                v = np.concatenate([v, f64(self.v[b, :, :n + c])], axis=1)
                valid = np.concatenate([np.ones((c, m + n), dtype=bool), self.sees[b, :c, :c]], axis=1)
                at = np.concatenate([np.arange(m + n), self.positions[b, :c]])
                dist = np.abs(self.positions[b, :c, None] - at[None, :]).astype(np.float64)
            for h in range(self.H):
                if planes is not None and (b, h) not in planes or c == 0:
                    continue
                if k.shape[1] == 0:
                    assert torch.all(o[b, h, :c] == 0)
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
        assert err.item() == 0 and a["ws"][:8].view(torch.int64).item() == 0 and torch.all(buf[n:] == 5.0)
        self.check(o, planes)
        return a, o


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("length", [0, 1, 63, 64, 65, 127, 128, 129, 1000])
def test_one_token_of_two_requests(gpu_lib, dtype, d, length):
    Case(2, 8, 2, 1, d, [length], [0, 200], dtype, sees="chain", seed=length).run()
    Case(2, 8, 2, 1, d, [300], [0, length], dtype, sees="chain", seed=length).run()


@pytest.mark.parametrize("n,T,H,Hkv", [(1, 1, 4, 4), (40, 1, 4, 2), (33, 1, 8, 2), (5, 3, 6, 1), (3, 16, 8, 2), (130, 1, 1, 1),
                                       (2, 33, 4, 1), (3, 31, 2, 1), (2, 100, 5, 5), (1, 130, 2, 1), (2, 257, 2, 2), (9, 7, 3, 1),
                                       (17, 1, 8, 1)])
@pytest.mark.parametrize("d", [64, 128])
def test_groups_and_row_tiles(gpu_lib, n, T, H, Hkv, d):
    """Tiles of several requests, the last one part empty; requests of several tiles; one prefix and two."""
    rng = np.random.default_rng(n)
    B = 2 * n
    Case(n, H, Hkv, T, d, [200, 517], rng.integers(0, 300, B), counts=rng.integers(1, T + 1, B), seed=T).run(
        planes={(b, h) for b in (0, 1, n - 1, n, B - 2, B - 1) for h in (0, H - 1)})


@pytest.mark.parametrize("softcap,sl", [(30.0, False), (0.0, True), (20.0, True), (100.0, False)])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("sees", ["tree", "chain"])
def test_score_options(gpu_lib, softcap, sl, dtype, d, sees):
    Case(3, 8, 4, 9, d, [300, 77], [0, 130, 5, 200, 64, 1], dtype, softcap=softcap, slopes=head_slopes(8) if sl else None,
         seed=1, sees=sees).run()


@pytest.mark.parametrize("d", [64, 128])
def test_slopes_of_either_sign(gpu_lib, d):
    Case(2, 4, 2, 5, d, [900, 40], [0, 300, 77, 2], torch.float16, slopes=[0.5, -0.25, 2.0 ** -6, -1.0], seed=2).run()


def test_ragged_batch(gpu_lib):
    plens = [0, 1000, 1]
    lens = [0, 5, 1023, 128, 700, 0, 64, 2000, 1]
    counts = [1, 7, 3, 0, 7, 2, 7, 1, 6]
    Case(3, 6, 2, 7, 64, plens, lens, counts=counts, softcap=25.0, slopes=head_slopes(6), seed=3).run()
    Case(3, 6, 2, 7, 128, plens, lens, counts=counts, seed=4).run()


@pytest.mark.parametrize("d", [64, 128])
def test_prefixes_alone(gpu_lib, d):
    """Cross attention: a source each, or one for four beams; one of them empty; capped; one token and many."""
    Case(1, 4, 2, 1, d, [37, 0, 700, 1, 64], None, seed=5).run()
    Case(4, 6, 6, 1, d, [500, 33, 0], None, torch.float16, softcap=30.0, seed=6).run()
    Case(2, 4, 1, 50, d, [300, 128], None, counts=[50, 0, 7, 50], seed=7).run()
    Case(1, 3, 3, 200, d, [90], None, seed=8).run()


def test_many_prefixes_and_requests(gpu_lib):
    """More (prefix, head) and (request, head) pairs than there are SMs, lengths far apart: runs that lie in one share."""
    rng = np.random.default_rng(9)
    lens = rng.integers(0, 300, 900)
    lens[7] = 5000
    plens = rng.integers(0, 400, 450)
    plens[3], plens[100] = 6000, 0
    Case(2, 2, 2, 2, 64, plens, lens, counts=rng.integers(0, 3, 900), seed=9).run(
        planes={(b, b % 2) for b in list(range(0, 30)) + list(range(190, 210)) + list(range(890, 900))})
    Case(2, 2, 2, 1, 64, plens, None, seed=10).run(planes={(b, b % 2) for b in list(range(0, 30)) + list(range(190, 210))})


@pytest.mark.parametrize("d", [64, 128])
def test_more_row_tiles_than_go_together(gpu_lib, d):
    """Nine and more row tiles per K/V head, of the prefix (300 requests) and of a request (1160 rows)."""
    rng = np.random.default_rng(11)
    Case(300, 4, 1, 1, d, [1500], rng.integers(0, 50, 300), seed=11).run(
        planes={(b, h) for b in (0, 31, 32, 255, 256, 287, 288, 299) for h in (0, 3)})
    Case(2, 10, 1, 116, d, [700], [0, 300], seed=12).run(planes={(0, 0), (0, 9), (1, 3), (1, 9)})


def test_a_long_prefix(gpu_lib):
    Case(3, 8, 1, 16, 128, [70001], [100, 0, 3000], seed=13).run(planes={(0, 0), (0, 7), (2, 5)})
    Case(3, 8, 1, 1, 64, [50001], [100, 0, 3000], torch.float16, seed=14).run(planes={(0, 0), (0, 7), (2, 5)})


def test_a_prefix_past_32_bit_offsets(gpu_lib):
    """2^31 elements and more in front of the last prefix's rows."""
    Hkv, d, T = 2, 128, 2
    small = Case(2, 4, Hkv, T, d, [300], [10, 70], seed=15)
    pcap = (1 << 31) // (Hkv * d) // 2 + 1000  # two prefixes: over 2^31 elements
    kp = torch.zeros(3, Hkv, pcap, d, dtype=torch.bfloat16, device="cuda")
    vp = torch.zeros_like(kp)
    kp[2, :, :300], vp[2, :, :300] = small.kp[0, :, :300].cuda(), small.vp[0, :, :300].cuda()
    a = small.args()
    six = [t.repeat(3, *[1] * (t.dim() - 1)) for t in (a["q"], a["k"], a["v"], a["lens"], a["tree"])]
    o = torch.full_like(six[0], 5.0)
    ws = torch.empty(stof.stof_prefix_attn_workspace_bytes(6, 3, 4, Hkv, T, d), dtype=torch.uint8, device="cuda")
    stof.stof_prefix_attn_fwd(six[0], kp, vp, i32([0, 1, 300]), six[1], six[2], six[3], small.scale, o, ws, tree=six[4])
    small.check(o[4:])


def test_rows_that_see_nothing(gpu_lib):
    T = 40
    sees = np.zeros((4, T, T), dtype=bool)
    sees[1] = True                      # every bit, those past the request's tokens included
    c = Case(2, 4, 2, T, 64, [0, 50], [0, 90, 0, 3], counts=[T, 11, T, 1], sees=sees, seed=16)
    a, o = c.run()
    assert torch.all(o[0] == 0)


@pytest.mark.parametrize("d", [64, 128])
def test_against_the_call_without_a_prefix(gpu_lib, d):
    """A prefix and own rows are one cache of both in stof_tree_attn_fwd: the two calls meet the same definition."""
    n, H, Hkv, T = 3, 4, 2, 5
    c = Case(n, H, Hkv, T, d, [333], [0, 200, 77], seed=17)
    a = c.args()
    o = torch.full(c.q.shape, 5.0, dtype=c.dtype, device="cuda")
    c.call(a, o)
    cap = 333 + c.cap
    k, v = (torch.zeros(n, Hkv, cap, d, dtype=c.dtype, device="cuda") for _ in range(2))
    for x, pre, own in ((k, a["kp"], a["k"]), (v, a["vp"], a["v"])):
        x[:, :, :333] = pre[:, :, :333]
        x[:, :, 333:] = torch.nan_to_num(own, nan=0.0, posinf=0.0)
    want = torch.full_like(o, 5.0)
    ws = torch.empty(stof.stof_tree_attn_workspace_bytes(n, H, Hkv, T, d), dtype=torch.uint8, device="cuda")
    stof.stof_tree_attn_fwd(a["q"], k, v, a["lens"] + 333, c.scale, want, ws, tree=a["tree"], counts=a["counts"])
    c.check(o)
    c.check(want)


@pytest.mark.parametrize("scale,softcap", [(-0.1, 0.0), (0.0, 0.0), (-0.1, 10.0), (2.0, 10.0)])
def test_scales(gpu_lib, scale, softcap):
    Case(2, 4, 2, 5, 64, [200, 90], [3, 70, 0, 11], torch.float16, scale=scale, softcap=softcap, seed=18).run()


def test_bad_lengths_are_skipped_and_reported(gpu_lib):
    c = Case(2, 4, 2, 3, 64, [100, 200, 300], [10, 20, 30, 40, 50, 60], seed=19)
    good = torch.full(c.q.shape, 5.0, dtype=c.dtype, device="cuda")
    c.call(c.args(), good)
    for name, bad, skipped in (("lens", [-1, 20, c.cap - 2, 2 ** 31 - 1, 50, 60], (0, 2, 3)),
                               ("counts", [4, 3, -1, 2 ** 31 - 1, 3, 3], (0, 2, 3)),
                               ("plens", [100, -1, 300], (2, 3)), ("plens", [100, 200, c.pcap + 1], (4, 5)),
                               ("plens", [-2 ** 31, 200, 300], (0, 1))):
        a = c.args()
        a[name] = i32(bad)
        o = torch.full_like(good, 5.0)
        err = torch.zeros(1, dtype=torch.int64, device="cuda")
        c.call(a, o, err)
        assert err.item() == stof.STOF_DEVERR_BAD_LENGTH == a["ws"][:8].view(torch.int64).item()
        for b in range(c.B):
            if b in skipped:
                assert torch.all(o[b] == 5.0)
        c.call(a, o)  # without an error word
        got = o.cpu()
        for b in range(c.B):  # the others' values: by the definition, as the shares have changed
            if b in skipped:
                got[b] = good[b].cpu()
        c.check(got)


def test_graph_replay_follows_the_lengths_and_repeats_bit_for_bit(gpu_lib):
    c = Case(2, 8, 2, 6, 128, [700, 300], [400, 900, 20, 5], seed=20)
    a = c.args()
    for name in ("kp", "vp", "k", "v"):
        a[name][~torch.isfinite(a[name])] = 0.0
    o = torch.full(c.q.shape, 5.0, dtype=c.dtype, device="cuda")
    c.call(a, o)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.call(a, o)
    for plens, lens in (([700, 300], [400, 900, 20, 5]), ([0, 337], [0, 130, 920, 9]), ([128, 128], [128] * 4)):
        a["plens"].copy_(i32(plens))
        a["lens"].copy_(i32(lens))
        a["ws"].fill_(0xEE)  # nothing is kept in the workspace
        o.fill_(float("nan"))
        graph.replay()
        want = torch.full_like(o, 5.0)
        c.call(a, want)
        torch.cuda.synchronize()
        assert torch.equal(o, want) and torch.isfinite(o.float()).all()


def test_values_do_not_depend_on_what_was_in_shared_memory(gpu_lib):
    """Rows of a tile that no request fills: after a call that leaves infinities there the bits are the same."""
    c = Case(3, 4, 2, 1, 64, [700], [5, 60, 0], softcap=30.0, seed=21)
    a = c.args()
    first = torch.full(c.q.shape, 5.0, dtype=c.dtype, device="cuda")
    c.call(a, first)
    wild = Case(40, 4, 1, 2, 64, [500], [64] * 40, softcap=30.0, seed=22)
    w = wild.args()
    w["q"].fill_(float("inf"))
    wild.call(w, torch.empty_like(w["q"]))
    again = torch.full_like(first, 5.0)
    c.call(a, again)
    assert torch.equal(first, again)


def test_two_streams_with_their_own_workspaces(gpu_lib):
    cs = [Case(2, 8, 2, 4, 128, [1500], [800, 100], seed=s) for s in (23, 24)]
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


def test_two_graphs_that_share_a_workspace_in_turn(gpu_lib):
    cs = [Case(2, 8, 2, 4, 64, [1000, 10], [100, 50, 0, 900], seed=25), Case(2, 8, 2, 4, 64, [3, 600], [2500, 0, 1, 77], seed=26)]
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


@pytest.mark.parametrize("d", [64, 128])
def test_far_positions_are_subtracted_exactly(gpu_lib, d):
    """Drafted tokens at positions near 2^31, whose neighbours fp32 cannot tell apart; and at the two ends of 32 bits."""
    T = 12
    c = Case(2, 4, 1, T, d, [0, 0], [0] * 4, torch.float16, slopes=head_slopes(4), seed=27)
    c.positions = 2_000_000_000 + np.arange(T)[None, :] + np.array([[0], [77], [1], [5]])
    c.run()
    c = Case(1, 4, 1, T, d, [40], [30], torch.float16, slopes=[2.0 ** -31] * 4, seed=28)
    c.positions = np.where(np.arange(T) % 3 == 0, -2 ** 31, 2 ** 31 - 1 - np.arange(T))[None, :]
    c.run()


def test_the_most_drafted_tokens(gpu_lib):
    T = stof.STOF_TREE_MAX_TOKENS
    Case(1, 2, 1, T, 64, [100], [100], seed=29, counts=[T - 1]).run(planes={(0, 1)})
    Case(1, 1, 1, T, 128, [33], [0], seed=30, sees="chain").run()


def test_calls_in_a_row_that_share_a_workspace(gpu_lib):
    """Each call is set up while the one before it and the copies between them still run: what is written just before a
    call is what it reads, and what is overwritten just after it is not."""
    cs = [Case(3, 8, 2, 2, 64, [700, 90], [30, 0, 5, 200, 1, 64], seed=31),
          Case(2, 16, 8, 1, 128, [1200], [100, 3], seed=32)]
    size = max(stof.stof_prefix_attn_workspace_bytes(c.B, c.NP, c.H, c.Hkv, c.T, c.d) for c in cs)
    ws = torch.full((size,), 0xCD, dtype=torch.uint8, device="cuda")
    want, aa, kept = [], [], []
    for c in cs:
        a = c.args()
        o = torch.full(c.q.shape, 5.0, dtype=c.dtype, device="cuda")
        c.call(a, o)
        c.check(o)
        a["ws"] = ws
        want.append(o)
        aa.append(a)
        kept.append({n: a[n].clone() for n in ("q", "kp", "vp", "k", "v")})
    got = []
    for i in range(24):
        c, a, keep = cs[i % 2], aa[i % 2], kept[i % 2]
        for n in ("q", "kp", "vp", "k", "v"):
            a[n].copy_(keep[n])
        got.append(torch.full(c.q.shape, 5.0, dtype=c.dtype, device="cuda"))
        c.call(a, got[-1])
        for n in ("q", "kp", "vp", "k", "v"):
            a[n].fill_(float("nan"))
        if i % 3 == 0:  # and straight after one another
            for n in ("q", "kp", "vp", "k", "v"):
                a[n].copy_(keep[n])
            got.append(torch.full_like(got[-1], 5.0))
            c.call(a, got[-1])
            c.call(a, got[-1])
    torch.cuda.synchronize()
    for o in got:
        assert torch.equal(o, want[0] if o.shape == want[0].shape else want[1])


def random_case(seed):
    rng = np.random.default_rng(seed)
    pick = lambda *xs: xs[rng.integers(len(xs))]
    Hkv = pick(1, 1, 2, 3)
    H = Hkv * pick(1, 2, 3, 5, 8)
    T = int(np.exp(rng.uniform(0, np.log(150))))
    n = int(np.exp(rng.uniform(0, np.log(60))))
    NP = int(np.exp(rng.uniform(0, np.log(12))))
    while NP * n * H * T > 6000:                     # rows of the definition in 64 bits
        n, NP = (n + 1) // 2, (NP + 1) // 2
        T = max(1, T - T // 3)
    cross = rng.random() < 0.25
    most = int(np.exp(rng.uniform(0, np.log(1500))))
    plens = rng.integers(0, most + 1, NP)
    lens = None if cross else rng.integers(0, int(np.exp(rng.uniform(0, np.log(400)))) + 1, NP * n)
    softcap = pick(0.0, 0.0, 25.0, 80.0)
    slopes = None
    if not cross and rng.random() < 0.4:
        slopes = (np.array(head_slopes(H)) * pick(1.0, 1.0, -0.05)).tolist()
    counts = rng.integers(0, T + 1, NP * n) if rng.random() < 0.5 else None
    return Case(n, H, Hkv, T, pick(64, 128), plens, lens, pick(torch.float16, torch.bfloat16), counts=counts,
                sees=pick("tree", "chain"), softcap=softcap, slopes=slopes, seed=seed, slack=int(rng.integers(0, 200)))


@pytest.mark.parametrize("seed", range(40))
def test_random_cases(gpu_lib, seed):
    random_case(seed).run()


def test_copies_from_the_host_and_events_come_before_a_call(gpu_lib):
    """What a copy from pinned memory, or another stream behind an event, writes just before a call is what it reads."""
    c = Case(2, 8, 2, 2, 128, [700, 90], [30, 0, 5, 200], seed=33)
    a = c.args()
    for name in ("kp", "vp", "k", "v", "q"):
        a[name][~torch.isfinite(a[name])] = 0.0
    settings = [([700, 90], [30, 0, 5, 200]), ([3, 120], [100, 7, 230, 0]), ([0, 1], [0, 0, 64, 65])]
    want, pinned = [], []
    for plens, lens in settings:
        a["plens"].copy_(i32(plens))
        a["lens"].copy_(i32(lens))
        o = torch.full(c.q.shape, 5.0, dtype=c.dtype, device="cuda")
        c.call(a, o)
        want.append(o)
        pinned.append([torch.tensor(x, dtype=torch.int32).pin_memory() for x in (plens, lens)])
    q_host, side = a["q"].cpu().pin_memory(), torch.cuda.Stream()
    big = torch.zeros(1 << 26, device="cuda")
    torch.cuda.synchronize()
    got = []
    for i in range(60):
        n = i % 3
        o = torch.full(c.q.shape, 5.0, dtype=c.dtype, device="cuda")
        if i % 2:
            a["q"].zero_()
            a["q"].copy_(q_host, non_blocking=True)
            for name, x in zip(("plens", "lens"), pinned[n]):
                a[name].copy_(x, non_blocking=True)
        else:
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                a["q"].zero_()
                big.add_(1.0)                            # some 80 us
                a["q"].copy_(q_host, non_blocking=True)
                for name, x in zip(("plens", "lens"), pinned[n]):
                    a[name].copy_(x, non_blocking=True)
                done = side.record_event()
            torch.cuda.current_stream().wait_event(done)
        c.call(a, o)
        got.append((n, o))
    torch.cuda.synchronize()
    for n, o in got:
        assert torch.equal(o, want[n])


def test_captured_calls_between_copies_and_joined_streams(gpu_lib):
    """In a graph: a copy node, or a copy and kernels of a joined stream, before the call; behind it a copy of its output
    and then kernels that overwrite its inputs."""
    c = Case(2, 8, 2, 2, 128, [700, 90], [30, 0, 5, 200], seed=34)
    a = c.args()
    for name in ("kp", "vp", "k", "v", "q"):
        a[name][~torch.isfinite(a[name])] = 0.0
    settings = [([700, 90], [30, 0, 5, 200]), ([3, 120], [100, 7, 230, 0]), ([0, 1], [0, 0, 64, 65])]
    want = []
    for plens, lens in settings:
        a["plens"].copy_(i32(plens))
        a["lens"].copy_(i32(lens))
        want.append(torch.full(c.q.shape, 5.0, dtype=c.dtype, device="cuda"))
        c.call(a, want[-1])
    staged = [a["plens"].clone(), a["lens"].clone(), a["q"].clone()]
    names = ("plens", "lens", "q")
    big = torch.zeros(1 << 24, device="cuda")
    o = torch.full(c.q.shape, 5.0, dtype=c.dtype, device="cuda")
    out = torch.empty_like(o)
    graphs = []
    for joined in (False, True):
        torch.cuda.synchronize()
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            o.fill_(5.0)
            if joined:
                here, side = torch.cuda.current_stream(), torch.cuda.Stream()
                side.wait_stream(here)
                with torch.cuda.stream(side):
                    big.add_(1.0)
                    for name, x in zip(names, staged):
                        a[name].copy_(x)
                big.neg()  # beside it
                here.wait_stream(side)
            else:
                for name, x in zip(names, staged):
                    a[name].copy_(x)
            c.call(a, o)
            out.copy_(o)
            for name in names:  # (after the call has read them)
                a[name].fill_(-7)
    for i in range(60):
        n = i % 3
        for x, y in zip(staged, settings[n]):
            x.copy_(i32(y))
        graphs[i // 3 % 2].replay()
        assert torch.equal(out, want[n]), i
