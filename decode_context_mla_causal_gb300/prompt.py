"""What stands before and beside a step over the paged rank pools: its pages, rotary positions,
and the attention of packed prompts.

Host-side plumbing around the C entry points, as ``step.VerifyStep`` and ``cache``: buffers are
sized and allocated once, and every call launches kernels on one stream with no host
synchronisation, so a call can be captured in a CUDA graph and replayed with new contents of the
same tensors. Objects hold their own workspace and outputs: calls of one object that overlap on
the GPU race, two objects do not. What sized the buffers cannot be changed afterwards.

A step with prompts: ``PagePlan`` gives blocks, slots, positions and row offsets; ``Rope`` rotates
q and k; ``dcp_kv_write`` or ``dcp_gqa_kv_write`` puts the rows into the pools (dims with
``batch=max_rows, qlen=1``); ``PromptAttention`` attends the new rows, or, with a context that
``dcp_gqa_kv_gather`` has read back, the context and them; ``GqaDecode`` serves the tokens that
follow.
"""

from __future__ import annotations

import torch

from . import binding as B
from .cache import _Sized


class PagePlan(_Sized):
    """Buffers + launch of a step's pages for ranks ``[rank_begin, rank_begin + num_ranks)``;
    ``max_rows`` bounds the new tokens of a step.

    ``slot_mapping`` ``[nr][max_rows]``, ``positions`` ``[max_rows]`` and ``cu_rows`` ``[B + 1]``
    are the last call's."""

    _fixed = frozenset(("_dims", "max_rows", "rank_begin", "num_ranks"))

    def __init__(self, dims: B.Dims, max_rows: int, device=None, rank_begin: int = 0,
                 num_ranks: int | None = None):
        B.dcp_mla_check_dims(dims, rank_begin, num_ranks)
        if max_rows < 1:
            raise ValueError(f"max_rows must be >= 1 (got {max_rows})")
        self._dims = dims = B.Dims.from_buffer_copy(dims)
        self.max_rows = max_rows
        self.rank_begin = rank_begin
        self.num_ranks = dims.dcp - rank_begin if num_ranks is None else num_ranks
        dev = torch.device(device or "cuda")
        i32 = torch.int32
        # as a call without requests, which writes nothing, leaves them
        self.slot_mapping = torch.full((self.num_ranks, max_rows), -1, dtype=i32, device=dev)
        self.positions = torch.zeros(max_rows, dtype=i32, device=dev)
        self.cu_rows = torch.zeros(dims.batch + 1, dtype=i32, device=dev)
        self.new_lens = torch.zeros(dims.batch, dtype=i32, device=dev)
        self.new_count = torch.zeros(1, dtype=i32, device=dev)
        self.workspace = torch.zeros(1, dtype=i32, device=dev)
        self.status = torch.zeros(1, dtype=i32, device=dev)

    def __call__(self, targets, seq_lens, block_table, free_list, free_count, new_lens=None,
                 new_count=None, stream=None):
        """Brings the requests from ``seq_lens`` to ``targets`` as far as blocks and rows go:
        ``seq_lens`` and ``free_count`` are updated in place, unless ``new_lens`` and
        ``new_count`` take their new values. Returns ``(slot_mapping, positions, cu_rows)``."""
        B.dcp_kv_plan(self._dims, targets, seq_lens, seq_lens if new_lens is None else new_lens,
                      block_table, free_list, free_count,
                      free_count if new_count is None else new_count, self.rank_begin,
                      self.num_ranks, self.slot_mapping, self.positions, self.cu_rows,
                      self.workspace, self.status, stream)
        return self.slot_mapping, self.positions, self.cu_rows

    def read_status(self) -> int:
        return int(self.status.item()) & 0xFFFFFFFF


class Rope(_Sized):
    """Rotary positions of the first ``rot_dim`` dims of each head.

    ``scaling``: None; ``dict(kind="linear", factor=..)``; or ``dict(kind="yarn", factor=..,
    original_len=..)`` with ``beta_fast`` (32), ``beta_slow`` (1) and ``amplitude`` (0.1 ln factor
    + 1) where they differ. ``table`` (one number for each pair: radians per position over 2 pi,
    times 2^64) and ``amplitude`` may be given in their place."""

    _fixed = frozenset(("rot_dim", "table"))

    def __init__(self, rot_dim: int, base: float = 10000.0, interleaved: bool = False,
                 scaling: dict | None = None, device=None, table=None, amplitude: float = 1.0):
        if table is None:
            table, amplitude = B.dcp_rope_table(rot_dim, base, self._scaling(scaling))
        elif scaling is not None or len(table) != rot_dim // 2:
            raise ValueError("a table has rot_dim / 2 numbers, and its scaling in them")
        self.rot_dim = rot_dim
        self.interleaved = interleaved
        self.amplitude = amplitude
        signed = [x - (1 << 64) if x >= 1 << 63 else x for x in (int(x) for x in table)]
        self.table = torch.tensor(signed, dtype=torch.int64, device=torch.device(device or "cuda"))

    @staticmethod
    def _scaling(scaling):
        if scaling is None:
            return None
        given = dict(scaling)
        kind = given.pop("kind", None)
        kinds = {"linear": B.ROPE_LINEAR, "yarn": B.ROPE_YARN}
        if kind not in kinds:
            raise ValueError(f"scaling kind must be one of {sorted(kinds)}, got {kind!r}")
        names = ("factor",) if kind == "linear" else ("factor", "original_len", "beta_fast",
                                                      "beta_slow", "amplitude")
        if set(given) - set(names) or not set(names[:2]) <= set(given):
            raise ValueError(f"{kind} scaling takes {names}, got {sorted(given)}")
        return B.RopeScaling(kinds[kind], float(given["factor"]), float(given.get("original_len", 0.0)),
                             float(given.get("beta_fast", 32.0)), float(given.get("beta_slow", 1.0)),
                             float(given.get("amplitude", 0.0)))

    def __call__(self, positions, q, k=None, out_q=None, out_k=None, stream=None):
        """Rotates ``q`` and ``k`` (``[rows][heads][dim]``) by ``positions`` (negative: back), in
        place or into ``out_q`` and ``out_k``; returns the rotated tensors."""
        B.dcp_rope(positions, self.table, self.amplitude, self.rot_dim, self.interleaved, q, k,
                   out_q, out_k, stream)
        return (q if out_q is None else out_q), (k if out_k is None else out_k)


class PromptAttention(_Sized):
    """Buffers + launches of attention over packed prompts, for up to ``max_rows`` rows of q and
    exactly ``max_seqs`` sequences (those that are not there: empty ones)."""

    _fixed = frozenset(("num_heads", "kv_heads", "qk_dim", "v_dim", "max_rows", "max_seqs",
                        "workspace_bytes"))

    def __init__(self, num_heads: int, kv_heads: int, qk_dim: int, v_dim: int, max_rows: int,
                 max_seqs: int, causal: bool = True, device=None):
        self.num_heads = num_heads
        self.kv_heads = kv_heads
        self.qk_dim = qk_dim
        self.v_dim = v_dim
        self.max_rows = max_rows
        self.max_seqs = max_seqs
        self.causal = causal
        dev = torch.device(device or "cuda")
        self.workspace_bytes = B.dcp_prompt_attention_workspace_size(max_rows, max_seqs, num_heads,
                                                                     kv_heads, v_dim)
        self.workspace = torch.empty(self.workspace_bytes, dtype=torch.uint8, device=dev)
        self.out = torch.empty((max_rows, num_heads, v_dim), dtype=torch.bfloat16, device=dev)
        self.lse = torch.empty((max_rows, num_heads), dtype=torch.float32, device=dev)
        self.status = torch.zeros(1, dtype=torch.int32, device=dev)

    def __call__(self, q, k, v, cu_q, cu_k, softmax_scale, stream=None):
        """Returns ``out`` and ``lse`` of q's rows."""
        rows, *heads = q.shape
        if heads != [self.num_heads, self.qk_dim] or rows > self.max_rows:
            raise ValueError(f"q must be [up to {self.max_rows}][{self.num_heads}][{self.qk_dim}], "
                             f"got {list(q.shape)}")
        if v.shape[-1] != self.v_dim or k.shape[1:2] != (self.kv_heads,):
            raise ValueError(f"k and v must be [keys][{self.kv_heads}][{self.qk_dim}] and "
                             f"[..][{self.v_dim}], got {list(k.shape)} and {list(v.shape)}")
        out, lse = self.out, self.lse
        if rows < self.max_rows:
            out, lse = out[:rows], lse[:rows]
        B.dcp_prompt_attention(self.max_seqs, self.causal, cu_q, cu_k, q, k, v, softmax_scale, out,
                               lse, self.workspace, self.status, stream,
                               workspace_bytes=self.workspace_bytes)
        return out, lse

    def read_status(self) -> int:
        return int(self.status.item()) & 0xFFFFFFFF
