"""Eviction by accumulated attention weight (oracle; test only).

* ``key_weights``: for every token of a sequence, by its global position, the sum over the
  rows that see it of ``exp(softmax_scale * q.k - lse_row)`` in float64, on top of
  ``decay`` times what it had if it is older than the step's qlen tokens.
* ``new_length``: L falls by the smallest multiple of dcp * interleave that brings it
  within the budget.
* ``select``: on a rank, the protected head and tail and the heaviest of the others, by
  plain sorting of (weight, index).
* ``compact``: the kept rows copied out, then written back in order.
"""

from __future__ import annotations

import numpy as np

from . import gqa as _gqa
from . import metadata as _md


def key_weights(*, q, pools, block_table, seq_lens, qlen, dcp, interleave, block_size, kv_dtype,
                kv_scale, softmax_scale, lse, decay, history, causal=True):
    """``q`` float64 ``[R][H][576]``, ``lse`` ``[R][H]``, ``history`` ``[W][B][ML]``. Returns
    ``(w, added, slack)``: the new weights ``[W][B][ML]`` (history where no token is), what
    the step added, and sum over rows of p * softmax_scale * sum |q||k| (for tolerances)."""
    w = np.array(history, dtype=np.float64)
    added, slack = np.zeros_like(w), np.zeros_like(w)
    for b, L in enumerate(int(x) for x in seq_lens):
        if L <= 0:
            continue
        pos = np.arange(L, dtype=np.int64)
        raw, rank, li = _gqa.token_rows(pools, block_table[b], pos, dcp=dcp,
                                        interleave=interleave, block_size=block_size)
        K = _gqa.decode_values(raw, kv_dtype, kv_scale if kv_dtype == "fp8" else 1.0)
        got, loose = np.zeros(L), np.zeros(L)
        for j in range(qlen):
            end = max(L - qlen + 1 + j, 0) if causal else L
            for h in range(q.shape[1]):
                row = b * qlen + j
                if np.isneginf(lse[row, h]):
                    continue
                p = np.exp(softmax_scale * (K[:end] @ q[row, h]) - lse[row, h])
                got[:end] += p
                loose[:end] += p * (softmax_scale * (np.abs(K[:end]) @ np.abs(q[row, h])))
        old = pos < L - qlen
        first = np.where(old, decay * w[rank, b, li], 0.0)
        w[rank, b, li] = got + first
        added[rank, b, li], slack[rank, b, li] = got, loose
    return w, added, slack


def new_length(L, budget, dcp, interleave):
    span = dcp * interleave
    while L > budget:
        L -= span
    return L


def local_count(L, rank, dcp, interleave):
    """Local length by counting the positions a rank owns."""
    pos = np.arange(max(L, 0), dtype=np.int64)
    return int((_md.owner(pos, dcp, interleave) == rank).sum())


def select(*, weights, seq_lens, budget, sink, recent, dcp, interleave):
    """``weights`` ``[W][B][ML]``; returns (kept index lists ``[W][B]``, new lengths)."""
    W, B = weights.shape[:2]
    lens = [new_length(int(L), budget, dcp, interleave) for L in seq_lens]
    kept = [[None] * B for _ in range(W)]
    for r in range(W):
        for b in range(B):
            n = local_count(int(seq_lens[b]), r, dcp, interleave)
            k = local_count(lens[b], r, dcp, interleave)
            if n == k:
                kept[r][b] = list(range(n))
                continue
            ends = set(range(sink)) | set(range(n - recent, n))
            free = [t for t in range(n) if t not in ends]
            value = lambda t: -np.inf if np.isnan(weights[r, b, t]) else float(weights[r, b, t])  # noqa: E731
            free.sort(key=lambda t: (-value(t), t))
            kept[r][b] = sorted(ends | set(free[:k - len(ends)]))
    return kept, lens


def compact(pools, kept, src_table, dst_table, block_size):
    """A copy of ``pools`` ``[W][NB][bs][...]`` with the kept rows written back in order."""
    out = np.array(pools, copy=True)
    for r, row in enumerate(kept):
        rows = [[pools[r, src_table[b][t // block_size], t % block_size].copy() for t in ts]
                for b, ts in enumerate(row)]
        for b, ts in enumerate(rows):
            for i, x in enumerate(ts):
                out[r, dst_table[b][i // block_size], i % block_size] = x
    return out
