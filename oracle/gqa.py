"""Grouped-head decode attention over interleaved K/V pools (oracle; test only).

Every token is looked up by its global position: position p lives on rank
``(p // S) % W`` at the local index that ``metadata`` counts, in block
``block_table[b][li // bs]``, row ``li % bs`` ("Context Parallel Guide (PCP & DCP)", "How
it works" item 1). Query head h reads K/V head ``h // group``; row j of a sequence of L
tokens attends positions ``[0, L - qlen + 1 + j)`` (all L where not causal). Plain softmax
in float64, with the two sums a tolerance needs beside it.
"""

from __future__ import annotations

import numpy as np

from . import fp8 as _fp8
from . import metadata as _md


def decode_values(raw, kv_dtype, scale=1.0):
    """float64 values of E4M3 codes (uint8), BF16 bits (uint16) or values, times the scale."""
    if kv_dtype == "values":  # decoded already (4-bit pools)
        return np.asarray(raw, dtype=np.float64) * float(scale)
    x = _fp8.decode_e4m3(raw) if kv_dtype == "fp8" else _fp8.decode_bf16(raw)
    return x * float(scale)


def token_rows(pools, table_row, positions, *, dcp, interleave, block_size):
    """Raw rows of global positions from pools ``[W][NB][bs][...]``."""
    p = np.asarray(positions, dtype=np.int64)
    rank = _md.owner(p, dcp, interleave)
    li = _md.local_index(p, dcp, interleave)
    return pools[rank, np.asarray(table_row)[li // block_size], li % block_size], rank, li


def decode(*, q, k_pools, v_pools, block_table, seq_lens, qlen, dcp, interleave, block_size,
           kv_dtype, k_scale, v_scale, softmax_scale, causal=True, ranks=None, skip=None):
    """``q`` float64 ``[R][H][D]``; raw pools ``[W][NB][bs][Hkv][D]``. ``ranks``: only these
    ranks' tokens; ``skip(b, li)``: tokens left out. Returns a dict: ``out`` ``[R][H][D]``,
    ``lse`` ``[R][H]`` (-inf for no token), ``absv`` = sum of softmax * |v|, and ``abss`` =
    the largest softmax_scale * sum |q||k| of the row's tokens."""
    R, H, D = q.shape
    hkv = k_pools.shape[3]
    group = H // hkv
    out, absv = np.zeros((R, H, D)), np.zeros((R, H, D))
    lse, abss = np.full((R, H), -np.inf), np.zeros((R, H))
    for b, L in enumerate(int(x) for x in seq_lens):
        pos = np.arange(max(L, 0), dtype=np.int64)
        raw, rank, li = token_rows(k_pools, block_table[b], pos, dcp=dcp, interleave=interleave,
                                   block_size=block_size)
        K = decode_values(raw, kv_dtype, k_scale)
        V = decode_values(token_rows(v_pools, block_table[b], pos, dcp=dcp, interleave=interleave,
                                     block_size=block_size)[0], kv_dtype, v_scale)
        use = np.ones(len(pos), bool) if ranks is None else np.isin(rank, ranks)
        if skip is not None:
            use &= ~np.array([bool(skip(b, int(x))) for x in li], bool)
        for j in range(qlen):
            row = b * qlen + j
            vis = use & (pos < (L - qlen + 1 + j if causal else L))
            if not vis.any():
                continue
            for h in range(H):
                k, v = K[vis, h // group], V[vis, h // group]
                s = softmax_scale * (k @ q[row, h])
                m = s.max()
                e = np.exp(s - m)
                lse[row, h] = m + np.log(e.sum())
                w = e / e.sum()
                out[row, h] = w @ v
                absv[row, h] = w @ np.abs(v)
                abss[row, h] = softmax_scale * (np.abs(k) @ np.abs(q[row, h])).max()
    return dict(out=out, lse=lse, absv=absv, abss=abss)
