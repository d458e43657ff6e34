"""Rotary positions, and attention of packed prompts (oracle; test only), in float64.

Rotary: pair i of a head at position n turns by ``n * f_i`` radians. Frequencies are
``base^(-2i/d)``, divided by a factor, or by parts: unscaled where the pair turns often within
the original length, divided where it turns seldom, with a ramp between (its slow end may lie
behind the last pair, up to pair d - 1).

Prompts: row i of a sequence of n rows and m keys attends its first ``m - n + 1 + i`` keys
("Context Parallel Guide (PCP & DCP)", prefill context: new tokens behind a context).
"""

from __future__ import annotations

import math

import numpy as np


def frequencies(rot_dim, base, kind=None, factor=1.0, original_len=0.0, beta_fast=32.0, beta_slow=1.0,
                amplitude=0.0):
    """``(radians per position, amplitude)``."""
    n = rot_dim // 2
    f = [base ** (-i / n) for i in range(n)]
    if kind is None:
        return np.array(f), 1.0
    if kind == "linear":
        return np.array(f) / factor, 1.0

    def pair(turns):  # base^(-i/n) * original_len = 2 pi turns
        return n * math.log(original_len / (2 * math.pi * turns), base)

    lo, hi = max(0, math.floor(pair(beta_fast))), min(rot_dim - 1, math.ceil(pair(beta_slow)))
    out = []
    for i, x in enumerate(f):
        stretched = min(1.0, max(0.0, (i - lo) / max(hi - lo, 0.001)))
        out.append(x * (1 - stretched) + x / factor * stretched)
    amp = amplitude if amplitude > 0 else (0.1 * math.log(factor) + 1 if factor > 1 else 1.0)
    return np.array(out), amp


def rotate(x, positions, freq, amplitude, interleaved):
    """``x`` float64 ``[T][H][D]``; the first ``2 len(freq)`` dims of each head are turned."""
    x = np.array(x, dtype=np.float64)
    n = len(freq)
    for i in range(n):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + n)
        angle = np.asarray(positions, dtype=np.float64) * freq[i]
        c, s = amplitude * np.cos(angle)[:, None], amplitude * np.sin(angle)[:, None]
        x[..., a], x[..., b] = x[..., a] * c - x[..., b] * s, x[..., b] * c + x[..., a] * s
    return x


def attend(*, q, k, v, cu_q, cu_k, softmax_scale, causal=True):
    """``q`` ``[T][H][d]``, ``k`` ``[S][Hkv][d]``, ``v`` ``[S][Hkv][dv]``, all float64. Rows of no
    sequence are NaN. ``absv`` and ``abss`` are the sums that a tolerance needs (``gqa.decode``)."""
    T, H, _ = q.shape
    group, dv = H // k.shape[1], v.shape[2]
    out, absv = np.full((T, H, dv), np.nan), np.zeros((T, H, dv))
    lse, abss = np.full((T, H), np.nan), np.zeros((T, H))
    for b in range(len(cu_q) - 1):
        n, m = cu_q[b + 1] - cu_q[b], cu_k[b + 1] - cu_k[b]
        for i in range(n):
            seen = min(m, max(0, m - n + 1 + i)) if causal else m
            row = cu_q[b] + i
            if seen == 0:
                out[row], lse[row] = 0.0, -np.inf
                continue
            of = slice(cu_k[b], cu_k[b] + seen)
            for h in range(H):
                kk, vv = k[of, h // group], v[of, h // group]
                s = softmax_scale * (kk @ q[row, h])
                top = s.max()
                e = np.exp(s - top)
                lse[row, h] = top + np.log(e.sum())
                w = e / e.sum()
                out[row, h] = w @ vv
                absv[row, h] = w @ np.abs(vv)
                abss[row, h] = softmax_scale * (np.abs(kk) @ np.abs(q[row, h])).max()
    return dict(out=out, lse=lse, absv=absv, abss=abss)
