"""Attention with capped and distance-lowered scores by its definition in 64
bits, and how far a kernel may be from it, element by element."""
import math

import numpy as np
import torch

HALF = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}  # half a step, relative


def attend(q, k, v, valid, distance, scale, softcap=0.0, slope=0.0, dtype=torch.bfloat16):
    """q [n, d], k, v [m, d] float64, valid [n, m], distance [n, m]: (O, tolerance of every element of O).

    The tolerance counts, with p the softmax, a = sum_j p_j |v_j| and u half a step of the type:
      - the output's rounding: u |O|;
      - P rounded to the type, p_j (1 + e_j) with |e_j| <= u, before both P V and its own sum: O then moves by
        sum p_j e_j (v_j - O) / (1 + sum p_j e_j), at most u (a + |O|) / (1 - u);
      - the scores: an fp32 product is off by at most 2^-20 s, s = scale sum |q| |k| (64 to 256 additions
        of 2^-24 each, and the tensor cores' own accumulation), the cap by 2^-20 softcap, the distance term by
        2^-22 of itself; a score off by e moves p by a factor within 1 +- e of it and O by at most 2 e a;
      - exponentials, sums and the division in fp32: 2^-18 a;
      - fp16's smallest steps: 2^-25 for each key of P (whose sum is at least 1 but for the reference's
        slack of 2^-8) and of O."""
    x = (q @ k.T) * scale
    size = abs(scale) * (np.abs(q) @ np.abs(k).T)
    e = 2.0 ** -20 * size
    if softcap:
        x = softcap * np.tanh(x / softcap)
        e = e + 2.0 ** -20 * softcap
    x = x - slope * distance
    e = e + 2.0 ** -22 * abs(slope) * distance
    x = np.where(valid, x, -np.inf)
    m = x.max(axis=1, keepdims=True)
    p = np.exp(x - np.where(np.isfinite(m), m, 0.0))
    l = p.sum(axis=1, keepdims=True)
    p = p / np.where(l > 0, l, 1.0)
    o, a = p @ v, p @ np.abs(v)
    e = np.where(valid, e, 0.0).max(axis=1, keepdims=True)
    u = HALF[dtype]
    tol = 2 * u * np.abs(o) * (1 + 2.0 ** -6) + (u * (1 + 2.0 ** -6) + 2 * e + 2.0 ** -18) * a
    if dtype == torch.float16:
        tol = tol + 2.0 ** -25 * (1 + np.where(valid, 1.0, 0.0) @ np.abs(v))
    return o, tol


def attend_heads(q, k, v, valid_of, distance, scale, softcap=0.0, slopes=None, dtype=torch.bfloat16):
    """[B, H, n, d] query heads over [B, Hkv, m, d] K/V heads; valid_of(b, h) -> [n, m].  (O, tolerance)."""
    B, H = q.shape[:2]
    group = H // k.shape[1]
    o, tol = np.zeros_like(q), np.zeros_like(q)
    for b in range(B):
        for h in range(H):
            o[b, h], tol[b, h] = attend(q[b, h], k[b, h // group], v[b, h // group], valid_of(b, h), distance, scale, softcap,
                                        0.0 if slopes is None else float(slopes[h]), dtype)
    return o, tol


def head_slopes(H):
    return [2.0 ** (-8.0 * (h + 1) / H) for h in range(H)]


def f64(t):
    return t.double().cpu().numpy()


def default_scale(d):
    return 1.0 / math.sqrt(d)
