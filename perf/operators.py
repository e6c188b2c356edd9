"""The language-model operators of this library as measured cases.

Three operators, each as a decoder's program calls it:

  rope  rotary positions on Q and K (half and interleaved layouts, part of the head, frequencies scaled for long
        contexts) between the packed [B][T][H + 2 Hkv][d] projection and the head-major [B][H][T][d] layout of the
        attention calls: forward, forward into a K/V cache, and the gradient
  attn  masked attention whose scores are capped by a tanh and / or lowered with the distance of key and query, over
        masks of packed documents (causal, bidirectional, with a prefix), keys and values shared by groups of heads:
        the mask is encoded from the token arrays and the attention run on it
  tree  attention of a tree of drafted tokens (one token: plain decoding) over a cache of keys and values

``run`` computes a case in plain torch, or, where ``own`` is true, through the library's calls.
"""
import math
import random

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ---------------------------------------------------------------- cases
def _rope(name, B, T, H, Hkv, d, rot, dtype, direction="fwd", interleaved=False, theta=10000.0, scaling="none",
          factor=1.0, amplitude=1.0, cap=0, far=0):
    return dict(name=name, op="rope", B=B, T=T, H=H, Hkv=Hkv, d=d, rot=rot, dtype=dtype, direction=direction,
                interleaved=interleaved, theta=theta, scaling=scaling, factor=factor, amplitude=amplitude, cap=cap,
                far=far)


def _attn(name, B, H, Hkv, Lq, Lk, d, dtype, docs, pad=0, causal=True, prefix=0.0, softcap=0.0, slopes=False):
    return dict(name=name, op="attn", B=B, H=H, Hkv=Hkv, Lq=Lq, Lk=Lk, d=d, dtype=dtype, docs=docs, pad=pad,
                causal=causal, prefix=prefix, softcap=softcap, slopes=slopes)


def _tree(name, B, H, Hkv, T, d, dtype, cap, lo, hi, softcap=0.0, slopes=False, ragged=False):
    return dict(name=name, op="tree", B=B, H=H, Hkv=Hkv, T=T, d=d, dtype=dtype, cap=cap, lo=lo, hi=hi,
                softcap=softcap, slopes=slopes, ragged=ragged)


def listed():
    return [
        # one new token of each of 16 requests, rotated and appended to the cache: latency
        _rope("rope_append_16x1", 16, 1, 32, 8, 128, 128, "bf16", cap=2048, scaling="linear", factor=4.0),
        # a 16k-token prompt out of the packed projection, frequencies scaled by their turns over 8192 positions
        _rope("rope_prompt_16k", 1, 16384, 32, 8, 128, 128, "bf16", theta=500000.0, scaling="turns", factor=8.0),
        # interleaved pairs on half of each head, an odd number of tokens
        _rope("rope_partial_interleaved", 3, 1237, 12, 12, 64, 32, "fp16", interleaved=True),
        # the gradient of a training batch, back into the packed projection's gradient
        _rope("rope_gradient", 4, 4096, 16, 16, 64, 64, "bf16", direction="bwd", scaling="index", factor=16.0,
              amplitude=1.25, theta=10000.0, far=30000),
        # five documents packed into 4096 tokens, capped scores, grouped heads
        _attn("attn_documents_cap_4k", 1, 32, 8, 4096, 4096, 128, "bf16", docs=5, softcap=50.0),
        # a batch with a bidirectional prefix and scores lowered by distance
        _attn("attn_prefix_slopes_2k", 8, 12, 12, 2048, 2048, 64, "fp16", docs=1, prefix=0.25, slopes=True),
        # one long causal sequence with capped scores
        _attn("attn_causal_cap_8k", 1, 32, 8, 8192, 8192, 128, "bf16", docs=1, softcap=30.0),
        # short odd sequences with padding behind the last document: rows without any key
        _attn("attn_short_padded", 4, 12, 12, 333, 333, 64, "bf16", docs=3, pad=21, softcap=30.0, slopes=True),
        # one token of one request: latency
        _tree("tree_decode_one", 1, 32, 8, 1, 128, "bf16", 4096, 4000, 4000),
        # 16 drafted tokens for each of 8 requests of different lengths
        _tree("tree_verify_8x16", 8, 32, 8, 16, 128, "bf16", 8192, 500, 8100),
        # large trees over long contexts
        _tree("tree_verify_long", 2, 64, 8, 64, 128, "bf16", 131072, 90000, 131000),
        # many requests with few drafted tokens, some with fewer than others; head size 64, cap and distance
        _tree("tree_many_short", 32, 12, 12, 7, 64, "fp16", 2048, 0, 2000, softcap=30.0, slopes=True, ragged=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng: random.Random):
    op = rng.choice(["rope", "attn", "tree"])
    dtype = rng.choice(["bf16", "fp16"])
    if op == "rope":
        d = rng.choice([32, 64, 128, 256])
        Hkv = rng.choice([1, 2, 4, 8, 12, 16])
        H = Hkv * rng.choice([1, 1, 2, 4])
        kind = rng.choice(["fwd", "append", "bwd"])
        most = 16384 * 48 * 128 // ((H + 2 * Hkv) * d)          # tokens of the largest listed case's work
        tokens = _log(rng, 1, min(16384, most))
        B = min(tokens, _log(rng, 1, 32))
        T = max(1, tokens // B)
        if kind == "append":
            T = min(T, 64)
        scaling = rng.choice(["none", "linear", "index", "turns"])
        c = _rope("", B, T, H, Hkv, d, rng.choice([d, d, d // 2]), dtype,
                  direction="bwd" if kind == "bwd" else "fwd", interleaved=rng.random() < 0.5,
                  theta=rng.choice([10000.0, 500000.0]), scaling=scaling,
                  factor=1.0 if scaling == "none" else rng.choice([2.0, 8.0, 16.0]),
                  amplitude=1.0 if scaling != "index" else 1.25,
                  cap=T + rng.randrange(1, 400) if kind == "append" else 0, far=rng.choice([0, 0, 1000000]))
    elif op == "attn":
        d = rng.choice([64, 128])
        Hkv = rng.choice([1, 2, 4, 8])
        H = Hkv * rng.choice([1, 2, 4])
        L = _log(rng, 1, 4096)
        B = max(1, min(8, 4096 // L, _log(rng, 1, 8)))
        Lq = L if rng.random() < 0.7 else rng.randrange(1, L + 1)
        pad = rng.randrange(0, L // 8 + 1) if Lq == L else 0
        causal = rng.random() < 0.7
        softcap, slopes = rng.choice([(30.0, False), (50.0, False), (0.0, True), (20.0, True), (0.0, False)])
        c = _attn("", B, H, Hkv, Lq, L, d, dtype, docs=1 if Lq != L else rng.randrange(1, max(2, min(9, (L - pad) // 16 + 1))),
                  pad=pad, causal=causal, prefix=rng.choice([0.0, 0.3]) if causal and Lq == L else 0.0,
                  softcap=softcap, slopes=slopes)
    else:
        d = rng.choice([64, 128])
        Hkv = rng.choice([1, 2, 4, 8])
        H = Hkv * rng.choice([1, 2, 4, 8])
        T = _log(rng, 1, 64)
        B = _log(rng, 1, 32)
        hi = min(_log(rng, 16, 32768), 131072 * 16 // (B * Hkv))
        lo = rng.randrange(0, hi + 1)
        softcap, slopes = rng.choice([(0.0, False), (0.0, False), (30.0, False), (0.0, True)])
        c = _tree("", B, H, Hkv, T, d, dtype, hi + T + rng.randrange(0, 130), lo, hi, softcap=softcap, slopes=slopes,
                  ragged=T > 1 and rng.random() < 0.3)
    c.pop("name")
    return c


# ---------------------------------------------------------------- shapes that follow from a case alone
def _documents(c):
    """Per batch element: the cut points of its documents (first token of each, and the end of the last)."""
    r = random.Random(c["docs"] * 7919 + c["Lk"] * 31 + c["B"])
    n = c["Lk"] - c["pad"]
    return [[0] + sorted(r.sample(range(1, n), c["docs"] - 1)) + [n] if c["docs"] > 1 else [0, n] for _ in range(c["B"])]


def _lengths(c):
    """Per request: rows in the cache, and drafted tokens."""
    r = random.Random(c["B"] * 131 + c["hi"])
    lens = [r.randint(c["lo"], c["hi"]) for _ in range(c["B"])]
    lens[0], lens[-1] = c["lo"], c["hi"]
    counts = [r.randint(1, c["T"]) if c["ragged"] and b % 3 == 1 else c["T"] for b in range(c["B"])]
    return lens, counts


def work(case):
    c = case
    if c["op"] == "rope":
        elems = c["B"] * c["T"] * (c["H"] + 2 * c["Hkv"]) * c["d"]
        turned = c["B"] * c["T"] * (c["H"] + c["Hkv"]) * c["rot"]
        return {"bytes": 4 * elems, "flops": 3 * turned}
    if c["op"] == "attn":
        pairs = 0
        for cuts in _documents(c):
            for a, e in zip(cuts, cuts[1:]):
                n = e - a
                if c["Lq"] != c["Lk"]:
                    first = c["Lk"] - c["Lq"]
                    pairs += sum(range(first + 1, c["Lk"] + 1)) if c["causal"] else c["Lq"] * n
                elif c["causal"]:
                    pre = int(c["prefix"] * n)
                    pairs += n * (n + 1) // 2 + pre * (pre - 1) // 2
                else:
                    pairs += n * n
        rows = c["B"] * (2 * c["Lq"] * c["H"] + 2 * c["Lk"] * c["Hkv"])
        return {"bytes": 2 * rows * c["d"] + 8 * c["B"] * (c["Lq"] + c["Lk"]), "flops": 4 * c["d"] * c["H"] * pairs}
    lens, counts = _lengths(c)
    keys = sum(n + t for n, t in zip(lens, counts))
    pairs = sum(t * (n + t / 2) for n, t in zip(lens, counts))
    return {"bytes": 4 * keys * c["Hkv"] * c["d"] + 4 * sum(counts) * c["H"] * c["d"] + 4 * c["B"] * c["T"] * ((c["T"] + 31) // 32),
            "flops": 4 * c["d"] * c["H"] * pairs}


# ---------------------------------------------------------------- inputs
def _frequencies(c):
    """The angle of each pair per position, in radians (64 bits)."""
    n = c["rot"] // 2
    w = c["theta"] ** (-np.arange(n, dtype=np.float64) / n)
    if c["scaling"] == "linear":
        w = w / c["factor"]
    elif c["scaling"] == "index":     # a ramp over the pair's number between two counts of turns in 4096 positions
        at = [c["rot"] * math.log(4096 / (turns * 2 * math.pi)) / (2 * math.log(c["theta"])) for turns in (32.0, 1.0)]
        low, high = max(math.floor(at[0]), 0), min(math.ceil(at[1]), c["rot"] - 1)
        ramp = np.clip((np.arange(n) - low) / max(high - low, 0.001), 0.0, 1.0)
        w = w * (1 - ramp) + w / c["factor"] * ramp
    elif c["scaling"] == "turns":     # a ramp over the pair's turns in 8192 positions
        keep = np.clip((8192 * w / (2 * math.pi) - 1.0) / (4.0 - 1.0), 0.0, 1.0)
        w = w * keep + w / c["factor"] * (1 - keep)
    return w


def _randn(g, shape, dtype):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def _int32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda").manual_seed(seed)
    rng = np.random.default_rng(seed)
    dt = DTYPES[c["dtype"]]
    B, H, Hkv, d = c["B"], c["H"], c["Hkv"], c["d"]
    if c["op"] == "rope":
        T = c["T"]
        s = dict(case=c, w=torch.tensor(_frequencies(c), device="cuda"))
        if c["direction"] == "bwd":   # gradients arrive head-major, as the attention's backward pass leaves them
            s["x"] = [_randn(g, (B, h, T, d), dt) for h in (H, Hkv, Hkv)]
        else:
            s["packed"] = _randn(g, (B, T, H + 2 * Hkv, d), dt)
            s["x"] = [t.transpose(1, 2) for t in s["packed"].split([H, Hkv, Hkv], dim=2)]
        first = rng.integers(0, c["far"] + 1, B) if c["far"] else np.zeros(B, dtype=np.int64)
        if c["cap"]:
            rows = rng.integers(0, c["cap"] - T + 1, B)
            s["rows"] = _int32(rows)
            first = first + rows
            s["caches"] = [_randn(g, (B, Hkv, c["cap"], d), dt) for _ in range(2)]
        s["positions"] = _int32(first[:, None] + np.arange(T)[None, :])
        if c["direction"] == "bwd":
            grad = torch.empty(B, T, H + 2 * Hkv, d, dtype=dt, device="cuda")
            s["grad"], s["out"] = grad, [t.transpose(1, 2) for t in grad.split([H, Hkv, Hkv], dim=2)]
        else:
            s["out"] = [torch.empty(B, h, T, d, dtype=dt, device="cuda") for h in (H, Hkv, Hkv)]
        return s
    slopes = torch.tensor([2.0 ** (-8.0 * (h + 1) / H) for h in range(H)], dtype=torch.float32, device="cuda")
    s = dict(case=c, slopes=slopes if c["slopes"] else None, scale=1.0 / math.sqrt(d))
    if c["op"] == "attn":
        Lq, Lk = c["Lq"], c["Lk"]
        s["q"] = _randn(g, (B, H, Lq, d), dt) * 2                 # logits of a few units, as trained heads have
        s["k"], s["v"] = _randn(g, (B, Hkv, Lk, d), dt), _randn(g, (B, Hkv, Lk, d), dt)
        doc = np.full((B, Lk), -1)
        order = np.tile(np.arange(Lk), (B, 1))
        k_order = order.copy()
        for b, cuts in enumerate(_documents(c)):
            for n, (a, e) in enumerate(zip(cuts, cuts[1:])):
                doc[b, a:e] = n
                k_order[b, a:a + int(c["prefix"] * (e - a))] = -1  # a prefix is seen by its whole document
        if not c["causal"]:
            order, k_order = np.zeros_like(order), np.zeros_like(order)
        s["q_doc"], s["k_doc"] = _int32(doc[:, Lk - Lq:]), _int32(doc)
        s["q_order"], s["k_order"] = _int32(order[:, Lk - Lq:]), _int32(k_order)
        s["o"] = torch.empty(B, H, Lq, d, dtype=dt, device="cuda")
        return s
    T, words = c["T"], (c["T"] + 31) // 32
    lens, counts = _lengths(c)
    s["q"] = _randn(g, (B, H, T, d), dt) * 2
    s["k"], s["v"] = (torch.randn(B, Hkv, c["cap"], d, generator=g, device="cuda", dtype=dt) for _ in range(2))
    sees = np.zeros((B, T, words * 32), dtype=bool)               # a drafted token sees itself and its ancestors
    depth = np.zeros((B, T), dtype=np.int64)
    for t in range(T):
        if t:
            parent = rng.integers(max(0, t - 6), t, B)
            sees[:, t] = sees[np.arange(B), parent]
            depth[:, t] = depth[np.arange(B), parent] + 1
        sees[:, t, t] = True
    bits = np.packbits(sees, axis=-1, bitorder="little").view("<i4")
    s["lens"], s["counts"], s["tree"] = _int32(lens), _int32(counts), _int32(bits)
    s["positions"] = _int32(np.array(lens)[:, None] + depth)
    s["o"] = torch.zeros(B, H, T, d, dtype=dt, device="cuda")
    return s


# ---------------------------------------------------------------- the library's calls
def _run_own(s):
    from sparse_mask_transformer_gb300 import stof
    c = s["case"]
    if c["op"] == "rope":
        if "plan" not in s:           # a program makes its plan once
            s["plan"] = stof.stof_rope_plan_init(
                c["rot"], theta=c["theta"], interleaved=c["interleaved"],
                scaling={"none": stof.STOF_ROPE_PLAIN, "linear": stof.STOF_ROPE_LINEAR, "index": stof.STOF_ROPE_BY_INDEX,
                         "turns": stof.STOF_ROPE_BY_TURNS}[c["scaling"]],
                factor=c["factor"], original_length=4096 if c["scaling"] == "index" else 8192,
                turns_lo=1.0, turns_hi=32.0 if c["scaling"] == "index" else 4.0, amplitude=c["amplitude"])
        q, k, v = s["x"]
        if c["direction"] == "bwd":
            stof.stof_rope_bwd(s["plan"], q, k, v, *s["out"], positions=s["positions"])
            return s["grad"]
        if c["cap"]:
            stof.stof_rope_fwd(s["plan"], q, k, v, s["out"][0], *s["caches"], positions=s["positions"], rows=s["rows"])
            return [s["out"][0], *s["caches"]]
        stof.stof_rope_fwd(s["plan"], q, k, v, *s["out"], positions=s["positions"])
        return s["out"]
    score = stof.Score(softcap=c["softcap"], slopes=s["slopes"], q_start=c["Lk"] - c["Lq"] if c["op"] == "attn" else 0)
    if c["op"] == "attn":
        if "ws" not in s:             # a program keeps its workspace
            s["ws"] = torch.empty(stof.stof_encode_workspace_bytes(c["B"], c["Lq"], c["Lk"], 128, 128), dtype=torch.uint8,
                                  device="cuda")
        fmt = stof.stof_encode_documents(s["q_doc"], s["k_doc"], s["q_order"], s["k_order"], 128, 128, s["ws"])
        return stof.stof_mha_fwd_score(s["q"], s["k"], s["v"], fmt, s["scale"], score, 1, 0, stof.STOF_KERNEL_AUTO, s["o"])
    if "ws" not in s:
        s["ws"] = torch.empty(stof.stof_tree_attn_workspace_bytes(c["B"], c["H"], c["Hkv"], c["T"], c["d"]),
                              dtype=torch.uint8, device="cuda")
    return stof.stof_tree_attn_fwd(s["q"], s["k"], s["v"], s["lens"], s["scale"], s["o"], s["ws"], tree=s["tree"],
                                   counts=s["counts"], positions=s["positions"], score=score)


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


def _scores(s, scores, distance):
    """Scaled products -> capped, lowered by distance (both in 32 bits)."""
    c = s["case"]
    if c["softcap"]:
        scores = scores.mul_(1.0 / c["softcap"]).tanh_().mul_(c["softcap"])
    if s["slopes"] is not None:
        scores.sub_(s["slopes"].view(scores.shape[1], scores.shape[2], 1, 1) * distance)
    return scores


def _attend(scores, valid, v):
    """softmax of the valid scores times v; 0 where nothing is valid."""
    scores = scores.masked_fill_(~valid, -math.inf)
    top = scores.amax(-1, keepdim=True)
    e = scores.sub_(torch.where(top == -math.inf, 0.0, top)).exp_()
    total = e.sum(-1, keepdim=True)
    return torch.matmul(e, v.float()) / torch.where(total == 0, 1.0, total)


def _run_plain(s):
    c = s["case"]
    B, H, Hkv, d = c["B"], c["H"], c["Hkv"], c["d"]
    if c["op"] == "rope":
        angle = s["positions"].double()[:, None, :, None] * s["w"]
        sign = -1.0 if c["direction"] == "bwd" else 1.0
        cos, sin = (c["amplitude"] * angle.cos()).float(), (sign * c["amplitude"] * angle.sin()).float()
        q, k, v = s["x"]
        q, k = _turn(q, cos, sin, c["rot"], c["interleaved"]), _turn(k, cos, sin, c["rot"], c["interleaved"])
        if c["cap"]:
            rows = (s["rows"].long()[:, None] + torch.arange(c["T"], device="cuda"))[:, None, :, None].expand(B, Hkv, c["T"], d)
            s["out"][0].copy_(q)
            s["caches"][0].scatter_(2, rows, k)
            s["caches"][1].scatter_(2, rows, v)
            return [s["out"][0], *s["caches"]]
        s["out"][0].copy_(q)
        s["out"][1].copy_(k)
        s["out"][2].copy_(v)
        return s["grad"] if c["direction"] == "bwd" else s["out"]
    if c["op"] == "attn":
        Lq, Lk = c["Lq"], c["Lk"]
        q = s["q"].float().view(B, Hkv, H // Hkv, Lq, d) * s["scale"]
        scores = torch.matmul(q, s["k"].float()[:, :, None].transpose(-1, -2))
        i, j = torch.arange(Lk - Lq, Lk, device="cuda"), torch.arange(Lk, device="cuda")
        scores = _scores(s, scores, (i[:, None] - j[None, :]).abs().float())
        valid = (s["q_doc"][:, :, None] == s["k_doc"][:, None, :]) & (s["q_doc"][:, :, None] >= 0)
        valid &= s["k_order"][:, None, :] <= s["q_order"][:, :, None]
        o = _attend(scores, valid[:, None, None], s["v"][:, :, None])
        return s["o"].copy_(o.view(B, H, Lq, d))
    T, n = c["T"], c["hi"] + c["T"]
    k, v = s["k"][:, :, :n].float(), s["v"][:, :, :n]
    q = s["q"].float().view(B, Hkv, H // Hkv, T, d) * s["scale"]
    scores = torch.matmul(q, k[:, :, None].transpose(-1, -2))
    j = torch.arange(n, device="cuda")
    lens, counts = s["lens"].long()[:, None], s["counts"].long()[:, None]
    u = (j[None, :] - lens).clamp(0, T - 1)                       # the drafted token in row j, where there is one
    old = j[None, :] < lens
    key_at = torch.where(old, j[None, :], s["positions"].long().gather(1, u))
    scores = _scores(s, scores, (s["positions"].long()[:, :, None] - key_at[:, None, :]).abs().float()[:, None, None])
    bit = (s["tree"].gather(2, (u // 32)[:, None, :].expand(B, T, n)) >> (u % 32)[:, None, :]) & 1
    valid = old[:, None, :] | ((j[None, :] < lens + counts)[:, None, :] & (bit != 0))
    o = _attend(scores, valid[:, None, None], v[:, :, None]).view(B, H, T, d)
    live = (torch.arange(T, device="cuda")[None, :] < counts)[:, None, :, None]
    return s["o"].copy_(torch.where(live, o.to(s["o"].dtype), s["o"]))


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---------------------------------------------------------------- the definitions in 64 bits
def _exact_rope(s):
    c = s["case"]
    half, at = c["rot"] // 2, s["positions"].double()
    got = []
    for n, x in enumerate(s["x"]):
        y = x.double().clone()
        if n < 2:
            for p in range(half):
                a, b = (2 * p, 2 * p + 1) if c["interleaved"] else (p, p + half)
                angle = (at * float(s["w"][p]))[:, None, :] * (-1 if c["direction"] == "bwd" else 1)
                y[..., a] = c["amplitude"] * (x[..., a].double() * torch.cos(angle) - x[..., b].double() * torch.sin(angle))
                y[..., b] = c["amplitude"] * (x[..., a].double() * torch.sin(angle) + x[..., b].double() * torch.cos(angle))
        got.append(y)
    if c["direction"] == "bwd":
        return torch.cat([y.transpose(1, 2) for y in got], dim=2)
    if c["cap"]:
        for n in (1, 2):
            whole = s["caches"][n - 1].double()
            for b, r in enumerate(s["rows"].tolist()):
                whole[b, :, r:r + c["T"]] = got[n][b]
            got[n] = whole
    return got


def _exact_head(c, slope, scale, q, k, v, distance, valid):
    x = (q.double() @ k.double().T) * scale
    if c["softcap"]:
        x = c["softcap"] * torch.tanh(x / c["softcap"])
    if slope is not None:
        x = x - slope * distance
    x = torch.where(valid, x, torch.full_like(x, -math.inf))
    p = torch.softmax(x, dim=-1)
    return torch.where(valid.any(-1, keepdim=True), p, torch.zeros_like(p)) @ v.double()


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    if c["op"] == "rope":
        return _exact_rope(s)
    out = s["o"].double()
    for b in range(c["B"]):
        if c["op"] == "attn":
            rows, keys = slice(0, c["Lq"]), slice(0, c["Lk"])
            distance = (torch.arange(c["Lq"], device="cuda")[:, None] + (c["Lk"] - c["Lq"]) - torch.arange(c["Lk"], device="cuda")).abs().double()
            valid = s["q_doc"][b][:, None].eq(s["k_doc"][b][None]) & s["q_doc"][b][:, None].ge(0) & s["q_order"][b][:, None].ge(s["k_order"][b][None])
        else:
            n, t = int(s["lens"][b]), int(s["counts"][b])
            rows, keys = slice(0, t), slice(0, n + t)
            where = torch.cat([torch.arange(n, device="cuda"), s["positions"][b, :t].long()])
            distance = (s["positions"][b, :t].long()[:, None] - where[None]).abs().double()
            bits = torch.tensor([[(int(row[u // 32]) >> (u % 32)) & 1 for u in range(t)] for row in s["tree"][b, :t].tolist()], device="cuda").bool()
            valid = torch.cat([torch.ones(t, n, dtype=torch.bool, device="cuda"), bits.view(t, t)], dim=1)
        for h in range(c["H"]):
            kv = h // (c["H"] // c["Hkv"])
            slope = None if s["slopes"] is None else float(s["slopes"][h])
            out[b, h, rows] = _exact_head(c, slope, s["scale"], s["q"][b, h, rows], s["k"][b, kv, keys], s["v"][b, kv, keys], distance, valid)
    return out
