"""Refusals of the grouped-head and eviction calls: checked on the host before anything is
launched (no GPU needed), with the message that names the argument."""

import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def dm():
    import __graft_entry__

    __graft_entry__.build()
    import decode_context_mla_causal_gb300 as mod

    return mod


def _dims(dm, **kw):
    base = dict(batch=2, qlen=2, num_heads=8, dcp=2, interleave=4, block_size=16,
                max_blocks_per_seq=8, max_local_len=100, num_blocks=64, num_splits=2)
    base.update(kw)
    return dm.make_dims(**base)


P = 1 << 12  # an aligned address that is never read: every call below is refused


def _decode(dm, d, kv_heads=4, dim=128, dtype=0, scale=0.1, ptrs=None, ranks=(0, 2)):
    a = dict(seq=P, table=P, q=P, k=P, v=P, out=P, lse=P, ws=P, status=P)
    a.update(ptrs or {})
    return dm.load().dcp_gqa_decode(ctypes.byref(d), kv_heads, dim, a["seq"], a["table"], a["q"], a["k"],
                                    a["v"], dtype, None, None, scale, *ranks, a["out"], a["lse"],
                                    a["ws"], a["status"], None)


@pytest.mark.parametrize("kw,code,word", [
    (dict(kv_heads=0), 1, "kv_heads"), (dict(kv_heads=3), 1, "multiple of kv_heads"),
    (dict(dim=96), 2, "head_dim"), (dict(dtype=7), 1, "kv_dtype"), (dict(scale=0.0), 1, "softmax_scale"),
    (dict(scale=float("nan")), 1, "softmax_scale"), (dict(ranks=(1, 2)), 1, "rank range"),
    (dict(ptrs=dict(q=None)), 1, "NULL"), (dict(ptrs=dict(ws=None)), 1, "NULL"),
    (dict(ptrs=dict(k=P + 8)), 1, "aligned"), (dict(ptrs=dict(out=P + 2)), 1, "aligned"),
])
def test_gqa_decode_refusals(dm, kw, code, word):
    assert _decode(dm, _dims(dm), **kw) == code
    assert word in dm.dcp_last_error()


def test_gqa_write_refusals(dm):
    d, lib = _dims(dm), dm.load()

    def call(kv_heads=4, dim=64, dtype=1, slots=P, k=P, ranks=2):
        return lib.dcp_gqa_kv_write(ctypes.byref(d), kv_heads, dim, slots, k, P, dtype, None, None, ranks, P, P, P, None)

    assert call(dim=32) == 2 and call(kv_heads=2000) == 1 and call(dtype=3) == 1
    assert call(slots=None) == 1 and call(k=P + 4) == 1 and call(ranks=3) == 1


def test_key_weights_refusals(dm):
    d, lib = _dims(dm), dm.load()

    def call(dtype=0, scale=0.1, decay=1.0, lse=P, kv=P, ws=P):
        return lib.dcp_mla_key_weights(ctypes.byref(d), P, P, P, kv, dtype, None, scale, lse, decay, 0, 2, P, P,
                                       ws, P, None)

    for kw, word in ((dict(dtype=2), "kv_dtype"), (dict(scale=-1.0), "softmax_scale"),
                     (dict(decay=-0.1), "decay"), (dict(decay=float("inf")), "decay"),
                     (dict(decay=float("nan")), "decay"), (dict(lse=None), "NULL"),
                     (dict(kv=P + 8), "aligned"), (dict(ws=None), "NULL"), (dict(ws=P + 4), "aligned")):
        assert call(**kw) == dm.DCP_ERR_INVALID_ARG and word in dm.dcp_last_error(), kw


def test_max_keep(dm):
    d = _dims(dm)  # span 8
    assert dm.dcp_kv_evict_max_keep(d, 8) == 4
    assert dm.dcp_kv_evict_max_keep(d, 13) == 8       # 4, and min(5, 4) more on rank 0
    assert dm.dcp_kv_evict_max_keep(d, 10000) == 100  # never above max_local_len
    with pytest.raises(dm.DcpError) as e:
        dm.dcp_kv_evict_max_keep(d, 7)
    assert e.value.code == dm.DCP_ERR_INVALID_ARG and "budget" in str(e.value)


def test_select_refusals(dm):
    d, lib = _dims(dm), dm.load()

    def call(budget=64, sink=0, recent=0, w=P):
        return lib.dcp_kv_evict_select(ctypes.byref(d), P, w, budget, sink, recent, 0, 2, P, P, P, P, None)

    # budget 64 may leave 57 tokens: 28 on the last rank
    for kw, word in ((dict(budget=7), "budget"), (dict(sink=-1), "sink"), (dict(recent=-1), "recent"),
                     (dict(sink=20, recent=9), "share"), (dict(w=None), "NULL")):
        assert call(**kw) == dm.DCP_ERR_INVALID_ARG and word in dm.dcp_last_error(), kw


def test_compact_refusals(dm):
    d, lib = _dims(dm), dm.load()

    def call(row=64, keep=10, idx=P, pool=P, w=(None, None)):
        return lib.dcp_kv_compact(ctypes.byref(d), row, idx, P, keep, P, P, 2, pool, *w, P, None)

    for kw, word in ((dict(row=8), "row_bytes"), (dict(row=72), "row_bytes"), (dict(keep=101), "max_keep"),
                     (dict(keep=-1), "max_keep"), (dict(idx=None), "NULL"), (dict(w=(P, None)), "both"),
                     (dict(pool=P + 8), "aligned")):
        assert call(**kw) == dm.DCP_ERR_INVALID_ARG and word in dm.dcp_last_error(), kw


def test_empty_batch_is_a_no_op(dm):
    d, lib = _dims(dm, batch=0), dm.load()
    assert _decode(dm, d, ptrs={n: None for n in ("seq", "q", "ws")}) == 0
    assert lib.dcp_kv_compact(ctypes.byref(d), 64, None, None, 10, None, None, 2, None, None, None, None, None) == 0
    assert lib.dcp_kv_evict_select(ctypes.byref(d), None, None, 64, 0, 0, 0, 2, None, None, None, None, None) == 0


def test_python_checks_tensors(dm):
    d = _dims(dm)
    t = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA device"):
        dm.dcp_kv_evict_select(d, t, t.float(), 64, 0, 0, 0, 2, t, t, t, t)
    with pytest.raises(TypeError, match="seq_lens must be"):
        dm.dcp_kv_evict_select(d, t.long(), t.float(), 64, 0, 0, 0, 2, t, t, t, t)


def test_what_sized_the_buffers_stays(dm):
    # a larger budget or batch would write past keep_idx and the workspace
    d = _dims(dm)
    ev, step = dm.KvEviction(d, 64, 2, 3, device="cpu"), dm.GqaDecode(d, 4, 64, dm.KV_BF16, device="cpu")
    for obj, names in ((ev, ("budget", "max_keep", "num_ranks", "rank_begin", "workspace_bytes", "dims")),
                       (step, ("kv_heads", "head_dim", "kv_dtype", "num_ranks", "rank_begin", "workspace_bytes", "dims"))):
        for name in names:
            with pytest.raises(AttributeError):
                setattr(obj, name, 1000)
    d.batch, d.max_local_len = 50, 128             # the caller's own, afterwards
    ev.dims.batch = step.dims.batch = 50           # a copy
    assert (ev.dims.batch, step.dims.max_local_len, ev.budget, ev.max_keep) == (2, 100, 64, 32)
    seen = []
    lib = dm.load()

    class Calls:                                   # what would reach the library
        def __getattr__(self, name):
            def call(dims, *args):
                seen.append((name, dims._obj.batch, dims._obj.max_local_len))
                return 0
            return call if name in ("dcp_kv_evict_select", "dcp_gqa_decode") else getattr(lib, name)

    with pytest.MonkeyPatch.context() as mp:
        mp.setattr(dm.binding, "_lib", Calls())
        mp.setattr(dm.binding, "_ptr", lambda *a, **k: 0)
        ev.select(None, stream=0)
        step(None, None, None, None, None, 0.1, None, None, stream=0)
    assert seen == [("dcp_kv_evict_select", 2, 100), ("dcp_gqa_decode", 2, 100)]
    ev.sink, ev.recent, ev.decay = 1, 2, 0.5       # checked by every call


def test_compact_takes_rows_of_its_own_length(dm):
    d = _dims(dm)
    ev = dm.KvEviction(d, 64, device="cpu")
    pool, table = torch.zeros(2, 64, 16, 8), torch.zeros(2, 8, dtype=torch.int32)
    idx, count = torch.zeros(2, 2, 40, dtype=torch.int32), torch.zeros(2, 2, dtype=torch.int32)
    for bad in (dict(keep_idx=idx, keep_count=count), dict(keep_idx=idx.view(-1), keep_count=count),
                dict(keep_idx=idx[..., :32].contiguous(), keep_count=count.view(-1))):
        with pytest.raises(ValueError, match=r"keep_idx and keep_count must be \[2, 2, 32\] and \[2, 2\]"):
            ev.compact(pool, table, **bad)
    with pytest.raises(ValueError, match="CUDA device"):
        ev.compact(pool, table, keep_idx=idx[..., :32].contiguous(), keep_count=count)


class _Elsewhere(torch.Tensor):
    """Stands for a tensor of another device than the current one."""

    is_cuda = property(lambda self: True)

    def get_device(self):
        return 1


def test_calls_that_took_any_reachable_tensor_still_do(dm, monkeypatch):
    # the grouped-head and eviction calls refuse another device's tensors, the verify path's take
    # them (a peer's memory can be mapped); a batch of 0 reaches the library and launches nothing
    monkeypatch.setattr(dm.binding, "_several_devices", True)
    monkeypatch.setattr(dm.binding, "_current_device", lambda: 0)
    d = _dims(dm, batch=0)
    other = lambda dtype, n=4: torch.zeros(n, dtype=dtype).as_subclass(_Elsewhere)  # noqa: E731
    i32, f32 = other(torch.int32), other(torch.float32)
    dm.dcp_mla_metadata(d, i32, i32, 0, 2, i32, i32, i32, i32, i32, stream=0)
    dm.dcp_lse_merge(d, 2, f32, f32, f32, other(torch.bfloat16), f32, status=i32, stream=0)
    dm.dcp_kv_slot_mapping(d, i32, i32, 0, 2, i32, i32, stream=0)
    with pytest.raises(ValueError, match="seq_lens is on cuda:1, the current device is cuda:0"):
        dm.dcp_kv_evict_select(d, i32, f32, 64, 0, 0, 0, 2, i32, i32, i32, i32, stream=0)
    with pytest.raises(ValueError, match="keep_idx is on cuda:1"):
        dm.dcp_kv_compact(d, 64, i32, i32, 0, i32, i32, 2, other(torch.float32, 1 << 15), None, None, i32, stream=0)


def test_loading_the_library_asks_for_no_device(dm, monkeypatch):
    # asking can leave a process that forks afterwards without CUDA in its children
    monkeypatch.setattr(dm.binding, "_lib", None)
    monkeypatch.setattr(torch.cuda, "device_count", lambda: pytest.fail("asked for the devices"))
    dm.load()


def test_a_budget_beyond_32_bits_is_refused(dm):
    # 2^32 + 64 tokens are no budget of 64
    d = _dims(dm)
    for n in (2 ** 32 + 64, -2 ** 32 + 64):
        with pytest.raises(ValueError, match="budget must fit 32 bits"):
            dm.dcp_kv_evict_max_keep(d, n)
        with pytest.raises(ValueError, match="budget must fit 32 bits"):
            dm.KvEviction(d, n, device="cpu")
        for kw in (dict(budget=n, sink=0, recent=0), dict(budget=64, sink=n, recent=0), dict(budget=64, sink=0, recent=n)):
            with pytest.MonkeyPatch.context() as mp, pytest.raises(ValueError, match="must fit 32 bits"):
                mp.setattr(dm.binding, "_ptr", lambda *a, **k: 0)
                dm.dcp_kv_evict_select(d, None, None, rank_begin=0, num_ranks=2, keep_idx=None, keep_count=None,
                                       new_lens=None, status=None, stream=0, max_keep=32, **kw)
    assert dm.KvEviction(d, 2 ** 31 - 1, device="cpu").max_keep == 100


def test_reset_clears_the_slots_it_names(dm):
    ev = dm.KvEviction(_dims(dm, batch=4), 64, device="cpu")
    for slots, gone in ((1, [1]), ([0, 3], [0, 3]), ([2, 2], [2]), ((), []), (None, [0, 1, 2, 3])):
        ev.weights.fill_(5.0)
        ev.reset(slots)
        assert ev.weights.amax((0, 2)).tolist() == ev.weights.amin((0, 2)).tolist() \
            == [0.0 if b in gone else 5.0 for b in range(4)]
    ev.weights.fill_(5.0)
    for bad in (4, -1, [0, 9]):
        with pytest.raises(ValueError, match="slots are 0 .. 3"):
            ev.reset(bad)
    assert bool((ev.weights == 5.0).all())
