"""Many requests of one video prompt, as a decoder runs them: the prompt's packed
projection is turned by its tokens' times, heights and widths into a shared
prefix (stof_rope_axes_fwd); each request's drafted tokens are turned and
appended to its own cache, and attend over the prefix and their own rows
(stof_prefix_attn_fwd); the accepted ones are kept (stof_cache_keep), one
request's rows replace another's (stof_cache_fork), and the next tokens attend
over what is left.  Each step in 64 bits from what the step before it stored,
the moved rows bit for bit; in eager calls and as one captured graph."""
import math
import os
import re

import numpy as np
import pytest
import torch

from sparse_mask_transformer_gb300 import stof
from tests.scored_reference import HALF, attend, f64
from tests.test_gpu_rope_axes import turned
from tests.test_gpu_tree_attention import bits_of, i32

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


class Layer:
    """The projections' outputs of one layer, its caches, and the same in 64 bits."""

    def __init__(self, g, B, H, Hkv, d, P, T, cap, dtype, axes, axis, w):
        self.B, self.H, self.Hkv, self.d, self.T, self.dtype = B, H, Hkv, d, T, dtype
        self.axes, self.axis, self.w = axes, axis, w
        self.prompt = torch.randn(1, P, H + 2 * Hkv, d, generator=g).to(dtype).cuda()
        self.steps = [torch.randn(B, T, H + 2 * Hkv, d, generator=g).to(dtype).cuda() for _ in range(2)]
        self.kp, self.vp = (torch.full((1, Hkv, P + 9, d), float("nan"), dtype=dtype, device="cuda") for _ in range(2))
        self.k, self.v = (torch.full((B, Hkv, cap, d), float("nan"), dtype=dtype, device="cuda") for _ in range(2))
        self.ws = torch.empty(stof.stof_prefix_attn_workspace_bytes(B, 1, H, Hkv, T, d), dtype=torch.uint8, device="cuda")
        self.q = [torch.empty(B, H, T, d, dtype=dtype, device="cuda") for _ in range(2)]
        self.seen = [[torch.empty_like(self.k) for _ in range(2)] for _ in range(2)]  # the caches as a step's attention has them
        self.o = [torch.full((B, H, T, d), 5.0, dtype=dtype, device="cuda") for _ in range(2)]

    def split(self, packed):
        return [t.transpose(1, 2) for t in packed.split([self.H, self.Hkv, self.Hkv], dim=2)]

    def fill(self, positions):
        q, k, v = self.split(self.prompt)
        stof.stof_rope_axes_fwd(self.axes, None, k, v, None, self.kp, self.vp, positions)

    def step(self, n, positions, lens, plen, tree, scale, score, err):
        q, k, v = self.split(self.steps[n])
        stof.stof_rope_axes_fwd(self.axes, q, k, v, self.q[n], self.k, self.v, positions, rows=lens, device_error=err)
        for to, cache in zip(self.seen[n], (self.k, self.v)):
            to.copy_(cache)
        stof.stof_prefix_attn_fwd(self.q[n], self.kp, self.vp, plen, self.k, self.v, lens, scale, self.o[n], self.ws, tree=tree,
                                  score=score, device_error=err)


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("d,H,Hkv,dtype", [(128, 8, 2, torch.bfloat16), (64, 6, 6, torch.float16)])
def test_samples_of_a_video_prompt(gpu_lib, d, H, Hkv, dtype, captured):
    B, P, T, cap, layers = 5, 450, 6, 64, 2
    g = torch.Generator().manual_seed(d)
    axis = [p % 3 for p in range(d // 2)]
    plan = stof.stof_rope_plan_init(d, theta=1000.0)
    w = np.array([1000.0 ** (-2 * p / d) for p in range(d // 2)])
    axes = stof.stof_rope_axes_init(plan, 3, axis)
    ls = [Layer(g, B, H, Hkv, d, P, T, cap, dtype, axes, axis, w) for _ in range(layers)]
    caches = stof.Caches([t for l in ls for t in (l.k, l.v)])
    softcap, scale = 30.0, 1 / math.sqrt(d)
    score, err = stof.Score(softcap), torch.zeros(1, dtype=torch.int64, device="cuda")
    # frames of 6 x 5 patches; text goes on behind the largest position of the prompt
    t = np.arange(P)
    grid = np.stack([t // 30, t // 5 % 6, t % 5])[:, None]
    text = int(grid.max()) + 1
    parents = [-1, 0, 0, 1, 1, 2]
    sees = np.eye(T, dtype=bool)
    depth = np.zeros(T, dtype=np.int64)
    for u, p in enumerate(parents):
        if p >= 0:
            sees[u] |= sees[p]
            depth[u] = depth[p] + 1
    tree = bits_of(np.tile(sees, (B, 1, 1)))
    lens0 = np.array([0, 3, 17, 9, 40])
    paths = [[0, 2, 5], [0, 1, 4], [0], [], [0, 1, 3]]       # branches of the tree; request 3 keeps nothing
    kept = np.array([len(p) for p in paths])
    src = np.array([-1, -1, 4, 0, -1])                       # request 4's rows go to 2, 0's to 3
    lens1 = lens0 + kept
    lens2 = np.where(src < 0, lens1, lens1[src])
    at = [np.broadcast_to((text + lens[:, None] + depth)[None], (3, B, T)) for lens in (lens0, lens2)]
    d_lens, d_new = i32(lens0), i32(np.zeros(B))
    d_path, d_kept, d_src = i32([p + [0] * (T - len(p)) for p in paths]), i32(kept), i32(src)
    d_plen, d_grid, d_at = i32([P]), i32(grid), [i32(x) for x in at]
    for l in ls:  # committed rows of earlier steps
        for x in (l.k, l.v):
            for b in range(B):
                x[b, :, :lens0[b]] = torch.randn(Hkv, int(lens0[b]), d, generator=g).to(dtype).cuda()
    start = [[t.clone() for t in (l.k, l.v)] for l in ls]

    def run():
        for l in ls:
            l.fill(d_grid)
            l.step(0, d_at[0], d_lens, d_plen, tree, scale, score, err)
        stof.stof_cache_keep(caches, d_lens, d_path, d_kept, d_new, err)
        stof.stof_cache_fork(caches, caches, d_src, d_new, d_new, err)
        for l in ls:
            l.step(1, d_at[1], d_new, d_plen, tree, scale, score, err)

    run()
    if captured:
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            run()
        for l, s in zip(ls, start):
            l.k.copy_(s[0])
            l.v.copy_(s[1])
            l.kp.fill_(float("nan"))
            for o in l.o:
                o.fill_(5.0)
        d_new.zero_()
        graph.replay()
    torch.cuda.synchronize()
    assert err.item() == 0
    assert d_new.tolist() == lens2.tolist()
    for l, s in zip(ls, start):
        def check_turned(got, packed, pos, heads):
            x = f64(packed[..., heads, :].transpose(1, 2))
            want, size = turned(x, pos, axis, w, False)      # one rounding, and the fp32 angle's and products' error
            assert np.all(np.abs(got - want) <= HALF[dtype] * np.abs(want) * (1 + 2.0 ** -6) + 2.0 ** -20 * size + 2.0 ** -25)
        ks, vs = slice(H, H + Hkv), slice(H + Hkv, H + 2 * Hkv)
        kp, vp = f64(l.kp)[0, :, :P], f64(l.vp)[0, :, :P]
        check_turned(kp[None], l.prompt, grid, ks)
        assert np.array_equal(vp, f64(l.prompt[0, :, vs].transpose(0, 1)))
        rows = [f64(t) for t in s]                           # the committed rows, followed through the steps
        for n, lens in enumerate((lens0, lens2)):
            k, v = (f64(t) for t in l.seen[n])
            q = f64(l.q[n])
            check_turned(q, l.steps[n], at[n], slice(0, H))
            for b in range(B):
                m = int(lens[b])
                for x, committed in zip((k, v), rows):
                    assert np.array_equal(x[b, :, :m], committed[b, :, :m])
                valid = np.concatenate([np.ones((T, P + m), dtype=bool), sees], axis=1)
                for h in range(H):
                    j = h // (H // Hkv)
                    kk, vv = np.concatenate([kp[j], k[b, j, :m + T]]), np.concatenate([vp[j], v[b, j, :m + T]])
                    want, tol = attend(q[b, h], kk, vv, valid, np.zeros(valid.shape), scale, softcap, 0.0, dtype)
                    assert np.all(np.abs(f64(l.o[n][b, h]) - want) <= tol), (n, b, h)
            drafted = np.stack([k[b, :, lens[b]:lens[b] + T] for b in range(B)])
            check_turned(drafted, l.steps[n], at[n], ks)
            assert np.array_equal(np.stack([v[b, :, lens[b]:lens[b] + T] for b in range(B)]), f64(l.steps[n][:, :, vs].transpose(1, 2)))
            rows = [k.copy(), v.copy()]
            if n == 0:                                       # kept rows, then the forked requests
                for x in rows:
                    before = x.copy()
                    for b in range(B):
                        for i, p in enumerate(paths[b]):
                            x[b, :, lens0[b] + i] = before[b, :, lens0[b] + p]
                    before = x.copy()
                    for b in range(B):
                        if src[b] >= 0:
                            x[b, :, :lens1[src[b]]] = before[src[b], :, :lens1[src[b]]]


def test_the_readme_block(gpu_lib):
    """README.md's block as it stands, with only the caller's own tensors given; its attention in 64 bits."""
    text = open(os.path.join(ROOT, "README.md")).read()
    block, = [b for b in re.findall(r"```python\n(.*?)```", text, re.S) if "stof_prefix_attn_fwd" in b]
    B, H, Hkv, P, T, cap, d = 3, 4, 2, 100, 4, 50, 64
    g = torch.Generator().manual_seed(5)

    def views(b, n):
        x = torch.randn(b, n, H + 2 * Hkv, d, generator=g).to(torch.bfloat16).cuda()
        return (t.transpose(1, 2) for t in x.split([H, Hkv, Hkv], dim=2))

    lens = np.array([0, 20, 7])
    own = [torch.randn(B, Hkv, cap, d, generator=g).to(torch.bfloat16).cuda() for _ in range(2)]
    at = np.arange(P)
    env = dict(stof=stof, plan=stof.stof_rope_plan_init(d), axis_of_pair=[p % 3 for p in range(d // 2)], own_caches=own,
               k_own=own[0], v_own=own[1], scale=1 / math.sqrt(d), lens=i32(lens), prefix_lens=i32([P]),
               positions=i32(np.stack([at // 20, at // 5 % 4, at % 5])[:, None]),
               positions1=i32(np.broadcast_to((5 + lens[:, None] + np.arange(T))[None], (3, B, T)).copy()),
               bits=i32([[[1], [3], [5], [13]]] * B), path=i32([[0, 2, 3, 0]] * B), kept=i32([3, 1, 0]),
               src=i32([-1, -1, 1]), new_lens=i32([0] * B), q_rot=torch.empty(1, H, P, d, dtype=torch.bfloat16, device="cuda"),
               ws2=torch.empty(stof.stof_prefix_attn_workspace_bytes(B, 1, H, Hkv, T, d), dtype=torch.uint8, device="cuda"))
    env["k_prefix"], env["v_prefix"] = (torch.full((1, Hkv, P, d), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    env["q"], env["k"], env["v"] = views(1, P)
    env["q1"], env["k1"], env["v1"] = views(B, T)
    for name in ("q1_rot", "o1"):
        env[name] = torch.empty(B, H, T, d, dtype=torch.bfloat16, device="cuda")
    before = [t.clone() for t in own]
    exec(block, env)
    torch.cuda.synchronize()
    assert env["new_lens"].tolist() == [3, 21, 21]
    assert torch.equal(own[0][2, :, :21], own[0][1, :, :21]) and torch.equal(own[0][1, :, :20], before[0][1, :, :20])
    # request 1 keeps its first drafted row where it is: its rows are what the attention saw
    sees = np.array([[1, 0, 0, 0], [1, 1, 0, 0], [1, 0, 1, 0], [1, 0, 1, 1]], dtype=bool)
    valid = np.concatenate([np.ones((T, P + 20), dtype=bool), sees], axis=1)
    for h in range(H):
        k, v = (np.concatenate([f64(env[a][0, h // 2]), f64(x[1, h // 2, :20 + T])])
                for a, x in (("k_prefix", own[0]), ("v_prefix", own[1])))
        want, tol = attend(f64(env["q1_rot"][1, h]), k, v, valid, np.zeros(valid.shape), env["scale"])
        assert np.all(np.abs(f64(env["o1"][1, h]) - want) <= tol)
