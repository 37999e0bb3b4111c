"""Packed prompts in fp64: attention of a prompt's tokens over its keys, and the prologue of every
token (test infrastructure; see ``oracle/__init__``)."""
from __future__ import annotations

import numpy as np

from .attention import to_f64
from .prologue import rms_norm, rope_angles


def attention(q, k, v, scale, causal=True):
    """q [n, Hq, D], k / v [m, Hkv, D] of one request; query i is at key position i + m - n and, when
    causal, sees keys up to its own. Returns (out [n, Hq, D], lse [n, Hq]); a query without keys gets
    zeros and -inf. Masked values are never multiplied."""
    q, k, v = to_f64(q), to_f64(k), to_f64(v)
    n, Hq, D = q.shape
    m, Hkv, _ = k.shape
    out = np.zeros((n, Hq, v.shape[-1]))
    lse = np.full((n, Hq), -np.inf)
    for i in range(n):
        seen = min(m, max(0, i + m - n + 1)) if causal else m
        if seen == 0:
            continue
        for h in range(Hq):
            g = h * Hkv // Hq
            s = k[:seen, g] @ q[i, h] * scale
            top = s.max()
            e = np.exp(s - top)
            out[i, h] = (e / e.sum()) @ v[:seen, g]
            lse[i, h] = top + np.log(e.sum())
    return out, lse


def rotate(x, w, pos, theta, eps):
    """RMSNorm then NeoX RoPE of x [H, D] at one position."""
    x = rms_norm(x, w, eps)
    D = x.shape[-1]
    ang = rope_angles(pos, D, theta)
    a, b = x[..., :D // 2], x[..., D // 2:]
    return np.concatenate([a * np.cos(ang) - b * np.sin(ang), b * np.cos(ang) + a * np.sin(ang)], -1)


def prologue(qkv, cu, seq_lens, q_w, k_w, eps, theta, num_heads, kv_heads, page_size, table):
    """Returns (q [tokens, Hq, D], k [tokens, Hkv, D], v, writes) with writes[i] = (page, slot) of token i."""
    x = to_f64(qkv)
    n, _, D = x.shape
    q, k = np.zeros((n, num_heads, D)), np.zeros((n, kv_heads, D))
    v = x[:, num_heads + kv_heads:]
    writes = {}
    for r in range(len(cu) - 1):
        for i in range(cu[r], cu[r + 1]):
            pos = int(seq_lens[r]) - (cu[r + 1] - i)
            q[i] = rotate(x[i, :num_heads], to_f64(q_w), pos, theta, eps)
            k[i] = rotate(x[i, num_heads:num_heads + kv_heads], to_f64(k_w), pos, theta, eps)
            writes[i] = (int(table[r][pos // page_size]), pos % page_size)
    return q, k, v, writes
