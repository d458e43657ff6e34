"""Grouped-head decode attention and eviction over the paged rank pools.

Host-side plumbing around the C entry points, as ``step.VerifyStep``: buffers are sized
and allocated once, and every call launches kernels on one stream with no host
synchronisation, so a call can be captured in a CUDA graph and replayed with new contents
of the same tensors. Objects hold their own workspace and outputs: calls of one object
that overlap on the GPU race, two objects do not. What sized the buffers (``dims``, which
is copied, ranks, heads, type and budget) cannot be changed afterwards.
"""

from __future__ import annotations

import math

import torch

from . import binding as B


class _Sized:
    """An object whose ``_fixed`` attributes sized its buffers: they are set once, and
    ``dims`` hands out copies, so that no call can outgrow a buffer."""

    _fixed: frozenset = frozenset()

    def __setattr__(self, name, value):
        if name in self._fixed and name in self.__dict__:
            raise AttributeError(f"{name} sized this object's buffers and cannot be changed: "
                                 f"make another {type(self).__name__}")
        super().__setattr__(name, value)

    @property
    def dims(self) -> B.Dims:
        return B.Dims.from_buffer_copy(self._dims)


class GqaDecode(_Sized):
    """Buffers + launches of grouped-head decode attention for ranks
    ``[rank_begin, rank_begin + num_ranks)``."""

    _fixed = frozenset(("_dims", "kv_heads", "head_dim", "kv_dtype", "rank_begin", "num_ranks",
                        "workspace_bytes"))

    def __init__(self, dims: B.Dims, kv_heads: int, head_dim: int, kv_dtype: int, device=None,
                 rank_begin: int = 0, num_ranks: int | None = None):
        B.dcp_mla_check_dims(dims, rank_begin, num_ranks)
        self._dims = dims = B.Dims.from_buffer_copy(dims)
        self.kv_heads = kv_heads
        self.head_dim = head_dim
        self.kv_dtype = kv_dtype
        self.rank_begin = rank_begin
        self.num_ranks = dims.dcp - rank_begin if num_ranks is None else num_ranks
        dev = torch.device(device or "cuda")
        R, H = dims.rows, dims.num_heads
        self.workspace_bytes = B.dcp_gqa_workspace_size(dims, kv_heads, head_dim, self.num_ranks)
        self.workspace = torch.empty(self.workspace_bytes, dtype=torch.uint8, device=dev)
        self.out = torch.empty((R, H, head_dim), dtype=torch.bfloat16, device=dev)
        self.lse = torch.empty((R, H), dtype=torch.float32, device=dev)
        self.status = torch.zeros(1, dtype=torch.int32, device=dev)

    def __call__(self, q, k_pool, v_pool, k_scale, v_scale, softmax_scale, seq_lens, block_table,
                 stream=None):
        B.dcp_gqa_decode(self._dims, self.kv_heads, self.head_dim, seq_lens, block_table, q, k_pool,
                         v_pool, self.kv_dtype, k_scale, v_scale, softmax_scale, self.rank_begin,
                         self.num_ranks, self.out, self.lse, self.workspace, self.status, stream,
                         workspace_bytes=self.workspace_bytes)
        return self.out, self.lse

    def read_status(self) -> int:
        return int(self.status.item()) & 0xFFFFFFFF


class KvEviction(_Sized):
    """Accumulated weights, selection and compaction for ranks
    ``[rank_begin, rank_begin + num_ranks)``.

    ``accumulate`` after every step, ``select`` and ``compact`` when sequences outgrow
    ``budget`` (global tokens; None: weights only). After ``compact`` a sequence is served
    with ``new_lens`` in the place of its length; its weights have moved with its rows.

    ``weights`` outlast the sequence they belong to: a step adds to whatever stands at the
    tokens before its own. When a batch slot takes another sequence, ``reset`` the slot, or
    the new prompt's tokens inherit the old one's weights.
    """

    _fixed = frozenset(("_dims", "budget", "max_keep", "rank_begin", "num_ranks",
                        "workspace_bytes"))

    def __init__(self, dims: B.Dims, budget: int | None = None, sink: int = 0, recent: int = 0,
                 decay: float = 1.0, device=None, rank_begin: int = 0,
                 num_ranks: int | None = None):
        B.dcp_mla_check_dims(dims, rank_begin, num_ranks)
        self._dims = dims = B.Dims.from_buffer_copy(dims)
        self.budget = budget
        self.sink = sink
        self.recent = recent
        self.decay = decay
        self.rank_begin = rank_begin
        self.num_ranks = dims.dcp - rank_begin if num_ranks is None else num_ranks
        dev = torch.device(device or "cuda")
        nr, Bt, i32 = self.num_ranks, dims.batch, torch.int32
        self.weights = torch.zeros((nr, Bt, dims.max_local_len), dtype=torch.float32, device=dev)
        self.workspace_bytes = B.dcp_mla_key_weights_workspace_size(dims, nr)
        self.workspace = torch.empty(self.workspace_bytes, dtype=torch.uint8, device=dev)
        self.status = torch.zeros(1, dtype=i32, device=dev)
        if budget is not None:
            self.max_keep = B.dcp_kv_evict_max_keep(dims, budget)
            self.keep_idx = torch.empty((nr, Bt, self.max_keep), dtype=i32, device=dev)
            self.keep_count = torch.empty((nr, Bt), dtype=i32, device=dev)
            self.new_lens = torch.empty(Bt, dtype=i32, device=dev)

    def accumulate(self, q, kv, kv_dtype, kv_scale, softmax_scale, lse, seq_lens, block_table,
                   history=None, stream=None):
        """Adds a step's attention weights (``lse``: the step's merged LSE) to ``decay``
        times ``history`` (this object's own weights where None)."""
        B.dcp_mla_key_weights(self._dims, seq_lens, block_table, q, kv, kv_dtype, kv_scale,
                              softmax_scale, lse, self.decay, self.rank_begin, self.num_ranks,
                              self.weights if history is None else history, self.weights,
                              self.workspace, self.status, stream,
                              workspace_bytes=self.workspace_bytes)
        return self.weights

    def reset(self, slots=None, stream=None):
        """Clears the weights of batch slots (a number or several; None: all of them)."""
        batch = self._dims.batch
        slots = (range(batch) if slots is None else (slots,) if isinstance(slots, int)
                 else [int(b) for b in slots])
        for b in slots:
            if not 0 <= b < batch:
                raise ValueError(f"slots are 0 .. {batch - 1}, got {b}")
        if isinstance(stream, int):
            stream = torch.cuda.ExternalStream(stream, device=self.weights.device)
        with torch.cuda.stream(stream):
            if len(slots) == batch == len(set(slots)):
                self.weights.zero_()
            else:
                for b in slots:
                    self.weights[:, b].zero_()

    def _need_budget(self):
        if self.budget is None:
            raise ValueError("this KvEviction has no budget")

    def select(self, seq_lens, weights=None, stream=None):
        """The local tokens each (rank, sequence) keeps: ``(keep_idx, keep_count, new_lens)``."""
        self._need_budget()
        B.dcp_kv_evict_select(self._dims, seq_lens, self.weights if weights is None else weights,
                              self.budget, self.sink, self.recent, self.rank_begin,
                              self.num_ranks, self.keep_idx, self.keep_count, self.new_lens,
                              self.status, stream, max_keep=self.max_keep)
        return self.keep_idx, self.keep_count, self.new_lens

    def compact(self, pool, block_table, new_block_table=None, keep_idx=None, keep_count=None,
                weights=None, move_weights=True, stream=None):
        """Moves the kept rows of ``pool`` (``[nr][NB][block_size][...]``) together, in place
        or into the blocks of ``new_block_table`` (blocks that no sequence of this call holds
        rows in), and the weights with them (once per eviction: ``move_weights=False`` for a
        second pool of the same tokens). ``keep_idx`` and ``keep_count``: ``select``'s where
        None, else of the same shapes."""
        self._need_budget()
        d = self._dims
        if pool.dim() < 4 or tuple(pool.shape[:3]) != (self.num_ranks, d.num_blocks, d.block_size):
            raise ValueError(f"pool must be [{self.num_ranks}][{d.num_blocks}][{d.block_size}][...], "
                             f"got {tuple(pool.shape)}")
        keep_idx = self.keep_idx if keep_idx is None else keep_idx
        keep_count = self.keep_count if keep_count is None else keep_count
        rows = (self.num_ranks, d.batch, self.max_keep)
        if tuple(keep_idx.shape) != rows or tuple(keep_count.shape) != rows[:2]:
            raise ValueError(f"keep_idx and keep_count must be {list(rows)} and {list(rows[:2])}, "
                             f"got {list(keep_idx.shape)} and {list(keep_count.shape)}")
        row_bytes = math.prod(pool.shape[3:]) * pool.element_size()
        w = (self.weights if weights is None else weights) if move_weights else None
        B.dcp_kv_compact(d, row_bytes, keep_idx, keep_count, self.max_keep, block_table,
                         block_table if new_block_table is None else new_block_table,
                         self.num_ranks, pool, w, w, self.status, stream)

    def read_status(self) -> int:
        return int(self.status.item()) & 0xFFFFFFFF
