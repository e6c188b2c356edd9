"""Operators for many requests of one long prompt as measured cases, next to those of perf/operators.py.

Three operators, each as a decoder's program calls it:

  axes    rotary positions whose pairs follow several axes (a video's time, height and width, an image's rows and
          columns), between the packed [B][T][H + 2 Hkv][d] projection and the head-major [B][H][T][d] layout of the
          attention calls: forward, forward into a K/V cache, and the gradient
  prefix  attention of one token or a tree of drafted ones per request over a prefix that groups of requests share and
          the request's own cache; without own caches: over an encoder's states, a length for each
  rows    rows of the K/V caches of all layers: the accepted ones of the drafted tokens moved together (keep), and a
          request's rows copied to others (fork)

``run`` computes a case in plain torch, or, where ``own`` is true, through the library's calls.
"""
import math
import random

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ---------------------------------------------------------------- cases
def _axes(name, B, T, H, Hkv, d, sections, grid, dtype, direction="fwd", interleaved=False, theta=10000.0,
          frequencies="shared", order="blocks", cap=0, has_v=True):
    """sections: pairs of each axis; grid: height and width of a frame; frequencies: one progression over all pairs
    ("shared") or one for each axis ("own"); order: an axis's pairs together ("blocks") or in turns ("turns")."""
    return dict(name=name, op="axes", B=B, T=T, H=H, Hkv=Hkv, d=d, sections=sections, grid=grid, dtype=dtype,
                direction=direction, interleaved=interleaved, theta=theta, frequencies=frequencies, order=order, cap=cap,
                has_v=has_v)


def _prefix(name, NP, n, H, Hkv, T, d, dtype, plo, phi, lo, hi, softcap=0.0, slopes=False, ragged=False, cross=False):
    """NP prefixes of plo .. phi rows, n requests each, with lo .. hi rows of their own (cross: none)."""
    return dict(name=name, op="prefix", NP=NP, n=n, H=H, Hkv=Hkv, T=T, d=d, dtype=dtype, plo=plo, phi=phi, lo=lo, hi=hi,
                softcap=softcap, slopes=slopes, ragged=ragged, cross=cross)


def _keep(name, caches, B, Hkv, cap, d, T, kept, dtype):
    return dict(name=name, op="keep", caches=caches, B=B, Hkv=Hkv, cap=cap, d=d, T=T, kept=kept, dtype=dtype)


def _fork(name, caches, B, Hkv, cap, d, lo, hi, inplace, dtype):
    """inplace: slot 0 goes to the others; else every slot to any of a second set of caches."""
    return dict(name=name, op="fork", caches=caches, B=B, Hkv=Hkv, cap=cap, d=d, lo=lo, hi=hi, inplace=inplace, dtype=dtype)


def listed():
    return [
        # one new token of each of 16 requests behind prompts with images, rotated and appended to the cache: latency
        _axes("axes_append_16x1", 16, 1, 32, 8, 128, "16 24 24", "24 24", "bf16", theta=1000000.0, cap=2048),
        # a video prompt: 16 frames of 32 x 32 patches out of the packed projection, the axes' pairs in turns
        _axes("axes_video_prompt_16k", 1, 16384, 32, 8, 128, "24 20 20", "32 32", "bf16", theta=500000.0, order="turns"),
        # the gradient of an image encoder's batch: rows and columns with frequencies of their own, an odd grid
        _axes("axes_image_gradient", 5, 37 * 53, 16, 16, 64, "16 16", "37 53", "fp16", direction="bwd",
              frequencies="own"),
        # a few requests of a short shared prompt, one token each: latency
        _prefix("prefix_decode_4", 1, 4, 32, 8, 1, 128, "bf16", 1000, 1000, 20, 200),
        # 64 samples of one long prompt, one token each
        _prefix("prefix_decode_64", 1, 64, 32, 8, 1, 128, "bf16", 16384, 16384, 100, 1500),
        # 8 prompts of different lengths, 16 samples each; head size 64, capped scores lowered with distance
        _prefix("prefix_groups_8x16", 8, 16, 12, 12, 1, 64, "fp16", 300, 6000, 0, 700, softcap=30.0, slopes=True),
        # 16 drafted tokens for each of 16 requests over a very long document, some with fewer
        _prefix("prefix_verify_long", 1, 16, 32, 8, 16, 128, "bf16", 131072, 131072, 500, 4000, ragged=True),
        # the decoder of an encoder-decoder model: 4 beams of each of 24 sources of different lengths
        _prefix("cross_beams_24x4", 24, 4, 16, 16, 1, 64, "bf16", 37, 1500, 0, 0, cross=True),
        # one layer's caches after the verification of 8 requests: latency
        _keep("keep_one_layer", 2, 8, 8, 1024, 128, 16, 6, "bf16"),
        # the caches of 24 layers after the verification of large trees
        _keep("keep_24_layers", 48, 16, 8, 512, 128, 64, 24, "bf16"),
        # one layer's prompt rows copied to 7 samples
        _fork("fork_samples", 2, 8, 8, 1024, 128, 700, 700, True, "bf16"),
        # beams of 12 layers rearranged into a second set of caches, odd lengths
        _fork("fork_beams_12_layers", 24, 12, 12, 1111, 64, 400, 1111, False, "fp16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng: random.Random):
    op = rng.choice(["axes", "prefix", "prefix", "keep", "fork"])
    dtype = rng.choice(["bf16", "fp16"])
    if op == "axes":
        d = rng.choice([32, 64, 80, 128, 256])
        pairs = rng.choice([d, d, d // 2]) // 2
        axes = rng.choice([2, 3, 3, 4])
        cuts = sorted(rng.sample(range(1, pairs), axes - 1))
        sections = " ".join(str(b - a) for a, b in zip([0] + cuts, cuts + [pairs]))
        Hkv = rng.choice([1, 2, 4, 8, 12, 16])
        H = Hkv * rng.choice([1, 1, 2, 4])
        kind = rng.choice(["fwd", "append", "bwd"])
        most = 16384 * 48 * 128 // ((H + 2 * Hkv) * d)          # tokens of the largest listed case's work
        tokens = _log(rng, 1, min(16384, most))
        B = min(tokens, _log(rng, 1, 32))
        T = max(1, tokens // B)
        if kind == "append":
            T = min(T, 64)
        c = _axes("", B, T, H, Hkv, d, sections, f"{rng.randrange(1, 65)} {rng.randrange(1, 65)}", dtype,
                  direction="bwd" if kind == "bwd" else "fwd", interleaved=rng.random() < 0.4,
                  theta=rng.choice([100.0, 10000.0, 1000000.0]), frequencies=rng.choice(["shared", "own"]),
                  order=rng.choice(["blocks", "turns"]), cap=T + rng.randrange(1, 400) if kind == "append" else 0,
                  has_v=kind != "fwd" or rng.random() < 0.7)
    elif op == "prefix":
        d = rng.choice([64, 128])
        Hkv = rng.choice([1, 2, 4, 8])
        H = Hkv * rng.choice([1, 2, 4, 8])
        NP = _log(rng, 1, 16)
        n = _log(rng, 1, 64)
        T = _log(rng, 1, 32)
        cross = rng.random() < 0.25
        rows = NP * n * H * T
        hi = 0 if cross else min(_log(rng, 1, 4096), max(1, 250000 // (NP * n * Hkv)), max(1, 200000000 // rows))
        phi = max(1, min(_log(rng, 16, 65536), 131072 * 6 // (NP * Hkv), 400000000 // rows))
        plo = rng.choice([phi, rng.randrange(0 if not cross else 1, phi + 1)])
        softcap, slopes = rng.choice([(0.0, False), (0.0, False), (30.0, False), (0.0, True), (20.0, True)])
        c = _prefix("", NP, n, H, Hkv, T, d, dtype, plo, phi, rng.randrange(0, hi + 1), hi, softcap=softcap,
                    slopes=slopes and not cross, ragged=T > 1 and rng.random() < 0.4, cross=cross)
    else:
        d = rng.choice([32, 64, 128, 256])
        Hkv = rng.choice([1, 2, 4, 8, 12])
        caches = 2 * _log(rng, 1, 32)
        B = _log(rng, 2, 32)
        if op == "keep":
            T = _log(rng, 1, 64)
            cap = T + _log(rng, 16, 600)
        else:
            T, cap = 0, _log(rng, 16, 2000)
        while caches * B * Hkv * cap * d > 165000000 and caches > 2:
            caches -= 2
        while caches * B * Hkv * cap * d > 165000000 and B > 2:
            B -= 1
        if op == "keep":
            c = _keep("", caches, B, Hkv, cap, d, T, rng.randrange(1, T // 2 + 2), dtype)
        else:
            c = _fork("", caches, B, Hkv, cap, d, rng.randrange(0, cap + 1), cap - rng.randrange(0, cap // 4 + 1),
                      rng.random() < 0.5, dtype)
            c["lo"] = min(c["lo"], c["hi"])
    c.pop("name")
    return c


# ---------------------------------------------------------------- what follows from a case alone
def _lengths(c):
    """Prefix rows of each prefix; own rows and drafted tokens of each request."""
    B = c["NP"] * c["n"]
    r = random.Random(B * 131 + c["hi"] * 7 + c["phi"])
    plens = [r.randint(c["plo"], c["phi"]) for _ in range(c["NP"])]
    plens[0], plens[-1] = c["plo"], c["phi"]
    lens = [r.randint(c["lo"], c["hi"]) for _ in range(B)]
    lens[0], lens[-1] = c["lo"], c["hi"]
    counts = [r.randint(1, c["T"]) if c["ragged"] and b % 3 == 1 else c["T"] for b in range(B)]
    return plens, lens, counts


def _paths(c):
    """Committed rows of each request, and the drafted rows that stay: a chain at first, then with gaps."""
    r = random.Random(c["B"] * 17 + c["T"] * 3 + c["cap"])
    lens = [r.randint(0, c["cap"] - c["T"]) for _ in range(c["B"])]
    paths = []
    for _ in range(c["B"]):
        k = r.randint(0, min(c["kept"], c["T"]))
        chain = r.randint(0, k)                                   # tokens 0, 1, .. of the tree's first branch
        later = range(k, c["T"])                                  # then others, behind the rows that they move to
        rest = sorted(r.sample(later, min(k - chain, len(later))))
        paths.append(list(range(chain)) + rest)
    return lens, paths


def _sources(c):
    """Rows in each slot, and the slot that each slot is copied from (-1: none)."""
    r = random.Random(c["B"] * 29 + c["cap"])
    lens = [r.randint(c["lo"], c["hi"]) for _ in range(c["B"])]
    if c["inplace"]:
        return lens, [-1] + [0] * (c["B"] - 1)
    return lens, [r.randrange(c["B"]) for _ in range(c["B"])]


def work(case):
    c = case
    if c["op"] == "axes":
        heads = c["H"] + c["Hkv"] * (2 if c["has_v"] else 1)
        tokens = c["B"] * c["T"]
        return {"bytes": 4 * tokens * heads * c["d"] + 4 * len(_numbers(c["sections"])) * tokens,
                "flops": 3 * tokens * (c["H"] + c["Hkv"]) * 2 * sum(_numbers(c["sections"]))}
    if c["op"] == "prefix":
        plens, lens, counts = _lengths(c)
        keys = sum(plens)
        pairs = sum(t * plens[b // c["n"]] for b, t in enumerate(counts))
        if not c["cross"]:
            keys += sum(n + t for n, t in zip(lens, counts))
            pairs += sum(t * (n + t / 2) for n, t in zip(lens, counts))
        return {"bytes": 4 * keys * c["Hkv"] * c["d"] + 4 * sum(counts) * c["H"] * c["d"],
                "flops": 4 * c["d"] * c["H"] * pairs}
    row = 4 * c["caches"] * c["Hkv"] * c["d"]                     # bytes of a token's rows, read and written
    if c["op"] == "keep":
        _, paths = _paths(c)
        moved = sum(1 for p in paths for i, u in enumerate(p) if u != i)
        return {"bytes": row * moved + 4 * c["B"] * (3 + c["T"]), "flops": 0}
    lens, src = _sources(c)
    copies = sum(lens[s] for s in src if s >= 0)
    read = sum(lens[s] for s in set(src) if s >= 0)
    return {"bytes": row // 2 * (copies + read) + 12 * c["B"], "flops": 0}


# ---------------------------------------------------------------- inputs
def _numbers(text):
    return [int(x) for x in text.split()]


def _axis_of_pair(c):
    left, out = _numbers(c["sections"]), []
    if c["order"] == "blocks":
        return [a for a, n in enumerate(left) for _ in range(n)]
    while any(left):
        for a in range(len(left)):
            if left[a]:
                out.append(a)
                left[a] -= 1
    return out


def _frequencies(c):
    """The angle of each pair per position of its axis, in radians (64 bits)."""
    axis, sections = _axis_of_pair(c), _numbers(c["sections"])
    n = sum(sections)
    if c["frequencies"] == "shared":
        return c["theta"] ** (-np.arange(n, dtype=np.float64) / n)
    seen, w = [0] * len(sections), np.zeros(n)
    for p, a in enumerate(axis):
        w[p] = c["theta"] ** (-seen[a] / sections[a])
        seen[a] += 1
    return w


def _randn(g, shape, dtype):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def _int32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def _prepare_axes(c, g, rng, dt):
    B, T, H, Hkv, d = c["B"], c["T"], c["H"], c["Hkv"], c["d"]
    heads = (H, Hkv, Hkv) if c["has_v"] else (H, Hkv)
    w = _frequencies(c)
    s = dict(case=c, w=torch.tensor(w, device="cuda"), axis=torch.tensor(_axis_of_pair(c), device="cuda"))
    if c["direction"] == "bwd":       # gradients arrive head-major, as the attention's backward pass leaves them
        s["x"] = [_randn(g, (B, h, T, d), dt) for h in heads]
        s["grad"] = torch.empty(B, T, sum(heads), d, dtype=dt, device="cuda")
        s["out"] = [t.transpose(1, 2) for t in s["grad"].split(heads, dim=2)]
    else:
        packed = _randn(g, (B, T, sum(heads), d), dt)
        s["x"] = [t.transpose(1, 2) for t in packed.split(heads, dim=2)]
        s["out"] = [torch.empty(B, h, T, d, dtype=dt, device="cuda") for h in heads]
    h, wd = _numbers(c["grid"])
    axes = len(_numbers(c["sections"]))
    t = np.arange(T)
    first = rng.integers(0, 5000, B)                              # where the images begin
    if c["cap"]:                                                  # text behind them: all axes alike
        s["rows"] = _int32(rng.integers(0, c["cap"] - T + 1, B))
        s["caches"] = [_randn(g, (B, Hkv, c["cap"], d), dt) for _ in heads[1:]]
        at = [t] * axes
    else:
        frame = [t // (h * wd), t // wd % h, t % wd]
        at = {2: [t // wd, t % wd], 3: frame, 4: [*frame, t]}[axes]
    s["positions"] = _int32(first[None, :, None] + np.stack(at)[:, None, :])
    return s


def _prepare_prefix(c, g, rng, dt):
    H, Hkv, T, d = c["H"], c["Hkv"], c["T"], c["d"]
    B = c["NP"] * c["n"]
    plens, lens, counts = _lengths(c)
    slopes = torch.tensor([2.0 ** (-8.0 * (h + 1) / H) for h in range(H)], dtype=torch.float32, device="cuda")
    s = dict(case=c, slopes=slopes if c["slopes"] else None, scale=1.0 / math.sqrt(d), plens=_int32(plens),
             counts=_int32(counts))
    s["q"] = _randn(g, (B, H, T, d), dt) * 2                      # logits of a few units, as trained heads have
    pcap = c["phi"] + 77
    s["kp"], s["vp"] = (torch.randn(c["NP"], Hkv, pcap, d, generator=g, device="cuda", dtype=dt) for _ in range(2))
    s["o"] = torch.zeros(B, H, T, d, dtype=dt, device="cuda")
    if c["cross"]:
        return s
    cap = c["hi"] + T + 100
    s["k"], s["v"] = (torch.randn(B, Hkv, cap, d, generator=g, device="cuda", dtype=dt) for _ in range(2))
    words = (T + 31) // 32
    sees = np.zeros((B, T, words * 32), dtype=bool)               # a drafted token sees itself and its ancestors
    depth = np.zeros((B, T), dtype=np.int64)
    for t in range(T):
        if t:
            parent = rng.integers(max(0, t - 6), t, B)
            sees[:, t] = sees[np.arange(B), parent]
            depth[:, t] = depth[np.arange(B), parent] + 1
        sees[:, t, t] = True
    s["tree"] = _int32(np.packbits(sees, axis=-1, bitorder="little").view("<i4"))
    s["lens"] = _int32(lens)
    s["positions"] = _int32(np.repeat(plens, c["n"])[:, None] + np.array(lens)[:, None] + depth)
    return s


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda").manual_seed(seed)
    rng = np.random.default_rng(seed)
    dt = DTYPES[c["dtype"]]
    if c["op"] == "axes":
        return _prepare_axes(c, g, rng, dt)
    if c["op"] == "prefix":
        return _prepare_prefix(c, g, rng, dt)
    shape = (c["B"], c["Hkv"], c["cap"], c["d"])
    s = dict(case=c, caches=[_randn(g, shape, dt) for _ in range(c["caches"])])
    if c["op"] == "keep":
        lens, paths = _paths(c)
        s["lens"], s["kept"] = _int32(lens), _int32([len(p) for p in paths])
        s["path"] = _int32([p + [0] * (c["T"] - len(p)) for p in paths])
        s["new_lens"] = torch.empty_like(s["lens"])
        return s
    lens, src = _sources(c)
    s["lens"], s["src"] = _int32(lens), _int32(src)
    s["new_lens"] = _int32(lens)
    s["to"] = s["caches"] if c["inplace"] else [_randn(g, shape, dt) for _ in range(c["caches"])]
    return s


# ---------------------------------------------------------------- the library's calls
def _run_own(s):
    from sparse_mask_transformer_gb300 import stof
    c = s["case"]
    if c["op"] == "axes":
        if "plan" not in s:           # a program makes its plan once
            plan = stof.stof_rope_plan_custom(_frequencies(c).tolist(), interleaved=c["interleaved"])
            s["plan"] = stof.stof_rope_axes_init(plan, len(_numbers(c["sections"])), _axis_of_pair(c))
        x, out = list(s["x"]), list(s["out"])
        if not c["has_v"]:
            x, out = x + [None], out + [None]
        if c["direction"] == "bwd":
            stof.stof_rope_axes_bwd(s["plan"], *x, *out, s["positions"])
            return s["grad"]
        if c["cap"]:
            to = [*s["caches"], None][:2]
            stof.stof_rope_axes_fwd(s["plan"], *x, out[0], *to, s["positions"], rows=s["rows"])
            return [out[0], *s["caches"]]
        stof.stof_rope_axes_fwd(s["plan"], *x, *out, s["positions"])
        return s["out"]
    if c["op"] == "prefix":
        if "ws" not in s:             # a program keeps its workspace
            s["ws"] = torch.empty(stof.stof_prefix_attn_workspace_bytes(c["NP"] * c["n"], c["NP"], c["H"], c["Hkv"], c["T"],
                                                                        c["d"]), dtype=torch.uint8, device="cuda")
        score = stof.Score(softcap=c["softcap"], slopes=s["slopes"])
        if c["cross"]:
            return stof.stof_prefix_attn_fwd(s["q"], s["kp"], s["vp"], s["plens"], None, None, None, s["scale"], s["o"],
                                             s["ws"], counts=s["counts"], score=score)
        return stof.stof_prefix_attn_fwd(s["q"], s["kp"], s["vp"], s["plens"], s["k"], s["v"], s["lens"], s["scale"], s["o"],
                                         s["ws"], tree=s["tree"], counts=s["counts"], positions=s["positions"], score=score)
    if "set" not in s:                # a program makes its list of caches once
        s["set"] = stof.Caches(s["caches"])
        s["to_set"] = s["set"] if c["op"] == "keep" or c["inplace"] else stof.Caches(s["to"])
    if c["op"] == "keep":
        stof.stof_cache_keep(s["set"], s["lens"], s["path"], s["kept"], s["new_lens"])
        return [*s["caches"], s["new_lens"]]
    stof.stof_cache_fork(s["set"], s["to_set"], s["src"], s["lens"], s["new_lens"])
    return [*s["to"], s["new_lens"]]


# ---------------------------------------------------------------- plain forms
def _turn(x, cos, sin, rot, interleaved):
    """x [B, H, T, d] with the first `rot` elements turned by the angles of cos, sin [B, 1, T, rot / 2]."""
    y = x.float().clone()
    if interleaved:
        a, b = y[..., 0:rot:2].clone(), y[..., 1:rot:2].clone()
        y[..., 0:rot:2], y[..., 1:rot:2] = a * cos - b * sin, b * cos + a * sin
    else:
        a, b = y[..., :rot // 2].clone(), y[..., rot // 2:rot].clone()
        y[..., :rot // 2], y[..., rot // 2:rot] = a * cos - b * sin, b * cos + a * sin
    return y.to(x.dtype)


def _run_axes(s):
    c = s["case"]
    rot = 2 * len(s["w"])
    angle = s["positions"].double()[s["axis"]].permute(1, 2, 0)[:, None] * s["w"]      # [B, 1, T, pairs]
    cos, sin = angle.cos().float(), (angle.sin() * (-1.0 if c["direction"] == "bwd" else 1.0)).float()
    got = [_turn(x, cos, sin, rot, c["interleaved"]) for x in s["x"][:2]] + list(s["x"][2:])
    s["out"][0].copy_(got[0])
    if c["cap"]:
        rows = s["rows"].long()[:, None] + torch.arange(c["T"], device="cuda")
        rows = rows[:, None, :, None].expand(c["B"], c["Hkv"], c["T"], c["d"])
        for cache, x in zip(s["caches"], got[1:]):
            cache.scatter_(2, rows, x)
        return [s["out"][0], *s["caches"]]
    for o, x in zip(s["out"][1:], got[1:]):
        o.copy_(x)
    return s["grad"] if c["direction"] == "bwd" else s["out"]


def _scores(s, scores, distance):
    """Scaled products -> capped, lowered by distance (both in 32 bits); scores [.., Hkv, group, rows, keys]."""
    c = s["case"]
    if c["softcap"]:
        scores = scores.mul_(1.0 / c["softcap"]).tanh_().mul_(c["softcap"])
    if s["slopes"] is not None:
        scores.sub_(s["slopes"].view(c["Hkv"], -1, 1, 1) * distance())
    return scores


def _run_prefix(s):
    c = s["case"]
    NP, n, H, Hkv, T, d = c["NP"], c["n"], c["H"], c["Hkv"], c["T"], c["d"]
    B, G, P = NP * n, H // Hkv, c["phi"]
    q = s["q"].float().view(B, Hkv, G, T, d) * s["scale"]
    # every request's rows over their prefix: [NP, n, Hkv, G, T, P]
    j = torch.arange(P, device="cuda")
    qp = q.view(NP, n, Hkv, G * T, d).transpose(1, 2).reshape(NP, Hkv, n * G * T, d)
    x = torch.matmul(qp, s["kp"][:, :, :P].float().transpose(-1, -2))
    x = x.view(NP, Hkv, n, G, T, P).transpose(1, 2).reshape(B, Hkv, G, T, P)
    x = _scores(s, x, lambda: (s["positions"].long()[:, :, None] - j).abs().float()[:, None, None])
    x.masked_fill_((j >= s["plens"].long().repeat_interleave(n)[:, None])[:, None, None, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    if not c["cross"]:                # and over their own rows: [B, Hkv, G, T, m]
        m = c["hi"] + T
        i = torch.arange(m, device="cuda")
        lens, counts = s["lens"].long()[:, None], s["counts"].long()[:, None]
        u = (i[None, :] - lens).clamp(0, T - 1)                   # the drafted token in row i, where there is one
        old = i[None, :] < lens
        y = torch.matmul(q.view(B, Hkv, G * T, d), s["k"][:, :, :m].float().transpose(-1, -2)).view(B, Hkv, G, T, m)

        def distance():
            at = torch.where(old, i + s["plens"].long().repeat_interleave(n)[:, None], s["positions"].long().gather(1, u))
            return (s["positions"].long()[:, :, None] - at[:, None, :]).abs().float()[:, None, None]
        y = _scores(s, y, distance)
        bit = (s["tree"].gather(2, (u // 32)[:, None, :].expand(B, T, m)) >> (u % 32)[:, None, :]) & 1
        valid = old[:, None, :] | ((i[None, :] < lens + counts)[:, None, :] & (bit != 0))
        y.masked_fill_(~valid[:, None, None], -math.inf)
        top = torch.maximum(top, y.amax(-1, keepdim=True))
    ref = torch.where(top == -math.inf, 0.0, top)
    x = x.sub_(ref).exp_()
    total = x.sum(-1, keepdim=True)
    xp = x.reshape(NP, n, Hkv, G * T, P).transpose(1, 2).reshape(NP, Hkv, n * G * T, P)
    o = torch.matmul(xp, s["vp"][:, :, :P].float()).view(NP, Hkv, n, G, T, d).transpose(1, 2).reshape(B, Hkv, G, T, d)
    if not c["cross"]:
        y = y.sub_(ref).exp_()
        total = total + y.sum(-1, keepdim=True)
        o = o + torch.matmul(y.view(B, Hkv, G * T, m), s["v"][:, :, :m].float()).view(B, Hkv, G, T, d)
    o = (o / torch.where(total == 0, 1.0, total)).reshape(B, H, T, d)
    live = (torch.arange(T, device="cuda")[None, :] < s["counts"].long()[:, None])[:, None, :, None]
    return s["o"].copy_(torch.where(live, o.to(s["o"].dtype), s["o"]))


def _run_keep(s):
    c = s["case"]
    i = torch.arange(c["T"], device="cuda")
    stays = i < s["kept"].long()[:, None]
    to = s["lens"].long()[:, None] + i
    frm = s["lens"].long()[:, None] + torch.where(stays, s["path"].long(), i)
    shape = (c["B"], c["Hkv"], c["T"], c["d"])
    to, frm = to[:, None, :, None].expand(shape), frm[:, None, :, None].expand(shape)
    for cache in s["caches"]:
        cache.scatter_(2, to, cache.gather(2, frm))
    torch.add(s["lens"], s["kept"], out=s["new_lens"])
    return [*s["caches"], s["new_lens"]]


def _run_fork(s):
    c = s["case"]
    src = s["src"].long()
    frm = torch.where(src < 0, torch.arange(c["B"], device="cuda"), src)
    lens = torch.where(src < 0, 0, s["lens"].long()[frm])
    copied = (torch.arange(c["cap"], device="cuda") < lens[:, None])[:, None, :, None]
    for a, b in zip(s["caches"], s["to"]):
        b.copy_(torch.where(copied, a[frm], b))
    s["new_lens"].copy_(torch.where(src < 0, s["new_lens"], s["lens"][frm]))
    return [*s["to"], s["new_lens"]]


def run(state):
    if own:
        return _run_own(state)
    return {"axes": _run_axes, "prefix": _run_prefix, "keep": _run_keep, "fork": _run_fork}[state["case"]["op"]](state)


# ---------------------------------------------------------------- the definitions in 64 bits
def _exact_axes(s):
    c = s["case"]
    half = len(s["w"])
    sign = -1 if c["direction"] == "bwd" else 1
    got = []
    for n, x in enumerate(s["x"]):
        y = x.double().clone()
        if n < 2:
            for p in range(half):
                a, b = (2 * p, 2 * p + 1) if c["interleaved"] else (p, p + half)
                phi = (sign * s["positions"][int(s["axis"][p])].double() * float(s["w"][p]))[:, None, :]
                y[..., a] = x[..., a].double() * torch.cos(phi) - x[..., b].double() * torch.sin(phi)
                y[..., b] = x[..., a].double() * torch.sin(phi) + x[..., b].double() * torch.cos(phi)
        got.append(y)
    if c["direction"] == "bwd":
        return torch.cat([y.transpose(1, 2) for y in got], dim=2)
    if c["cap"]:
        for n in range(1, len(got)):
            whole = s["caches"][n - 1].double()
            for b, r in enumerate(s["rows"].tolist()):
                whole[b, :, r:r + c["T"]] = got[n][b]
            got[n] = whole
    return got


def _exact_prefix(s):
    c = s["case"]
    G, out = c["H"] // c["Hkv"], s["o"].double()
    plens, lens, counts = (s[x].tolist() if x in s else None for x in ("plens", "lens", "counts"))
    for b in range(c["NP"] * c["n"]):
        np_, t = b // c["n"], counts[b]
        P, own_rows = plens[np_], 0 if c["cross"] else lens[b] + t
        valid = torch.ones(t, P + own_rows, dtype=torch.bool, device="cuda")
        if not c["cross"]:
            words = s["tree"][b, :t].tolist()
            valid[:, P + lens[b]:] = torch.tensor([[(row[u // 32] >> (u % 32)) & 1 for u in range(t)] for row in words],
                                                  device="cuda").bool()
        if s["slopes"] is not None:
            at = s["positions"][b, :t].long()
            where = torch.cat([torch.arange(P + lens[b], device="cuda"), at])
            distance = (at[:, None] - where[None]).abs().double()
        for kv in range(c["Hkv"]):
            k, v = s["kp"][np_, kv, :P].double(), s["vp"][np_, kv, :P].double()
            if not c["cross"]:
                k = torch.cat([k, s["k"][b, kv, :own_rows].double()])
                v = torch.cat([v, s["v"][b, kv, :own_rows].double()])
            for h in range(kv * G, kv * G + G):
                x = (s["q"][b, h, :t].double() @ k.T) * s["scale"]
                if c["softcap"]:
                    x = c["softcap"] * torch.tanh(x / c["softcap"])
                if s["slopes"] is not None:
                    x = x - float(s["slopes"][h]) * distance
                x = torch.where(valid, x, torch.full_like(x, -math.inf))
                p = torch.where(valid.any(-1, keepdim=True), torch.softmax(x, dim=-1), torch.zeros_like(x))
                out[b, h, :t] = p @ v
    return out


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    if c["op"] == "axes":
        return _exact_axes(s)
    if c["op"] == "prefix":
        return _exact_prefix(s)
    if c["op"] == "keep":
        lens, paths = _paths(c)
        got = []
        for cache in s["caches"]:
            y = cache.double()
            for b, p in enumerate(paths):
                y[b, :, lens[b]:lens[b] + len(p)] = cache[b][:, [lens[b] + u for u in p]].double()
            got.append(y)
        return got + [torch.tensor([n + len(p) for n, p in zip(lens, paths)], dtype=torch.int32, device="cuda")]
    lens, src = _sources(c)
    got = []
    for a, b in zip(s["caches"], s["to"]):
        y = b.double()
        for slot, r in enumerate(src):
            if r >= 0:
                y[slot, :, :lens[r]] = a[r, :, :lens[r]].double()
        got.append(y)
    return got + [torch.tensor([lens[b if r < 0 else r] for b, r in enumerate(src)], dtype=torch.int32, device="cuda")]
