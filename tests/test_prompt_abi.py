"""Refusals of the page, rotary, prompt and 4-bit calls: checked on the host before anything is
launched (no GPU needed), with the message that names the argument; and what is computed on the
host."""

import ctypes

import numpy as np
import pytest
import torch

import oracle


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
PLAN = ("targets", "lens", "new", "table", "free", "count", "new_count")
OUTS = ("slots", "positions", "cu", "ws", "status")


def _plan(dm, d, rows=10, ranks=(0, 2), **ptrs):
    a = {n: P for n in PLAN + OUTS}
    a.update(ptrs)
    return dm.load().dcp_kv_plan(ctypes.byref(d), *(a[n] for n in PLAN), *ranks, rows, *(a[n] for n in OUTS), None)


def test_plan_refusals(dm):
    d = _dims(dm)
    for kw, code, word in [(dict(rows=0), 1, "max_rows"), (dict(rows=-1), 1, "max_rows"),
                           (dict(rows=(1 << 30) + 1), 1, "max_rows"), (dict(ranks=(1, 2)), 1, "rank range")] + [
                               (dict([(n, None)]), 1, "NULL") for n in PLAN + OUTS]:
        assert _plan(dm, d, **kw) == code and word in dm.dcp_last_error(), kw
    assert _plan(dm, _dims(dm, batch=16385, qlen=1)) == 2 and "requests" in dm.dcp_last_error()
    big = _dims(dm, batch=16000, qlen=1, max_blocks_per_seq=200000)
    assert _plan(dm, big) == 2 and "max_blocks_per_seq" in dm.dcp_last_error()
    assert _plan(dm, _dims(dm, batch=0), targets=None, slots=None) == 0  # nothing to do


def test_rope_table(dm):
    for scaling, kw in ((None, {}), (dm.RopeScaling(1, 8.0), dict(kind="linear", factor=8.0)),
                        (dm.RopeScaling(2, 32.0, 4096.0, 32.0, 1.0, 0.0),
                         dict(kind="yarn", factor=32.0, original_len=4096)),
                        (dm.RopeScaling(2, 0.5, 1000.0, 4.0, 2.0, 1.25),
                         dict(kind="yarn", factor=0.5, original_len=1000, beta_fast=4.0, beta_slow=2.0, amplitude=1.25))):
        table, amp = dm.dcp_rope_table(96, 10000.0, scaling)
        freq, want = oracle.prompt.frequencies(96, 10000.0, **kw)
        assert len(table) == 48 and amp == np.float32(want)
        # rounded to units of 2^-64; powers and products in doubles are within a few 2^-53 of each other
        turns = np.array([x / 2.0 ** 64 for x in table])
        assert np.allclose(turns, np.mod(freq / (2 * np.pi), 1.0), rtol=2.0 ** -50, atol=2.0 ** -64)


def test_rope_table_refusals(dm):
    S = dm.RopeScaling
    for args, word in (((24, 1e4), "rot_dim"), ((0, 1e4), "rot_dim"), ((8192, 1e4), "rot_dim"), ((64, 1.0), "base"),
                       ((64, float("nan")), "base"), ((64, 1e4, S(3, 2.0)), "kind"), ((64, 1e4, S(1, 0.0)), "factor"),
                       ((64, 1e4, S(1, 5e-324)), "factor"),
                       ((64, 1e4, S(2, 2.0, 0.0, 32.0, 1.0, 0.0)), "original_len"),
                       ((64, 1e4, S(2, 2.0, 100.0, 1.0, 1.0, 0.0)), "beta"),
                       ((64, 1e4, S(2, 2.0, 100.0, 32.0, 1.0, -1.0)), "amplitude")):
        with pytest.raises(dm.DcpError) as e:
            dm.dcp_rope_table(*args)
        assert e.value.code == dm.DCP_ERR_INVALID_ARG and word in str(e.value), args
    for bad in (dict(kind="other", factor=2.0), dict(factor=2.0), dict(kind="yarn", factor=2.0),
                dict(kind="linear", factor=2.0, beta_fast=3.0)):
        with pytest.raises(ValueError):
            dm.Rope(64, scaling=bad)
    with pytest.raises(ValueError):
        dm.Rope(64, table=[1, 2, 3])


def test_rope_refusals(dm):
    lib = dm.load()
    from decode_context_mla_causal_gb300.binding import RopeHeads

    def call(rows=3, dim=64, rot=64, inter=0, pos=P, table=P, amp=1.0, a=None, b=None):
        side = dict(x=P, out=P, x_row=512, x_head=64, out_row=512, out_head=64, heads=8)
        pa = RopeHeads(**{**side, **(a or {})})
        pb = None if b is None else ctypes.byref(RopeHeads(**{**side, **b}))
        return lib.dcp_rope(rows, dim, rot, inter, pos, table, amp, ctypes.byref(pa), pb, None)

    for kw, word in ((dict(rows=-1), "rows"), (dict(rot=20), "rot_dim"), (dict(dim=48), "dim"), (dict(dim=68), "dim"),
                     (dict(dim=5000), "dim"), (dict(inter=2), "interleaved"), (dict(amp=float("inf")), "amplitude"),
                     (dict(amp=float("nan")), "amplitude"), (dict(pos=None), "NULL"), (dict(table=None), "NULL"),
                     (dict(table=P + 4), "aligned"), (dict(a=dict(heads=0)), "heads"), (dict(b=dict(heads=1025)), "heads"),
                     (dict(a=dict(x_row=516)), "strides"), (dict(b=dict(out_head=4)), "strides"),
                     (dict(a=dict(x=None)), "NULL"), (dict(a=dict(x=P + 8, out=P + 8)), "aligned"),
                     (dict(a=dict(out_row=1024)), "in place"),
                     # outputs that lie on one another
                     (dict(a=dict(x_head=0, out_head=0)), "overlap"), (dict(a=dict(x_row=0, out_row=0)), "overlap"),
                     (dict(b=dict(out=2 * P, out_head=56)), "overlap"), (dict(b=dict(out=2 * P, out_row=-56)), "overlap")):
        assert call(**kw) == dm.DCP_ERR_INVALID_ARG and word in dm.dcp_last_error(), kw
    assert call(rows=0, pos=None) == 0
    assert lib.dcp_rope(1, 64, 64, 0, P, P, 1.0, None, None, None) == 1 and "a is NULL" in dm.dcp_last_error()


def _prompt(dm, ptrs=None, scale=0.1, **kw):
    from decode_context_mla_causal_gb300.binding import PromptDims

    d = dict(batch=2, rows=10, keys=20, num_heads=8, kv_heads=2, qk_dim=128, v_dim=128, causal=1, q_row=1024,
             q_head=128, k_row=256, k_head=128, v_row=256, v_head=128)
    d.update(kw)
    a = dict(cu_q=P, cu_k=P, q=P, k=P, v=P, out=P, lse=P, ws=P, status=P)
    a.update(ptrs or {})
    return dm.load().dcp_prompt_attention(ctypes.byref(PromptDims(**d)), a["cu_q"], a["cu_k"], a["q"], a["k"], a["v"],
                                          scale, a["out"], a["lse"], a["ws"], a["status"], None)


def test_prompt_refusals(dm):
    cases = [(dict(batch=-1), 1, "batch"), (dict(rows=-1), 1, "rows"), (dict(keys=-1), 1, "keys"), (dict(keys=(1 << 30) + 1), 2, "keys"),
             (dict(num_heads=0), 1, "num_heads"), (dict(num_heads=1025), 1, "num_heads"), (dict(kv_heads=3), 1, "kv_heads"),
             (dict(kv_heads=0), 1, "kv_heads"), (dict(batch=8193), 2, "sequences"), (dict(rows=1 << 28), 2, "rows"),
             (dict(qk_dim=96), 2, "qk_dim"), (dict(qk_dim=192, v_dim=192), 2, "qk_dim"), (dict(v_dim=64), 2, "v_dim"),
             (dict(causal=2), 1, "causal"), (dict(q_row=1028), 1, "strides"), (dict(v_head=0), 1, "strides"),
             (dict(k_row=-256), 1, "strides"), (dict(k_head=1 << 40), 1, "strides"), (dict(scale=0.0), 1, "softmax_scale"),
             (dict(scale=float("nan")), 1, "softmax_scale"), (dict(ptrs=dict(q=P + 8)), 1, "aligned"),
             (dict(ptrs=dict(out=P + 16)), 1, "aligned"), (dict(ptrs=dict(ws=P + 8)), 1, "aligned")]
    cases += [(dict(ptrs={n: None}), 1, "NULL") for n in ("cu_q", "cu_k", "q", "k", "v", "out", "lse", "ws", "status")]
    for kw, code, word in cases:
        assert _prompt(dm, **kw) == code and word in dm.dcp_last_error(), kw
    assert _prompt(dm, batch=0, ptrs=dict(q=None)) == 0 and _prompt(dm, rows=0, ptrs=dict(q=None)) == 0
    with pytest.raises(dm.DcpError):
        dm.dcp_prompt_attention_workspace_size(10, 2, 8, 3, 128)
    with pytest.raises(dm.DcpError) as e:
        dm.dcp_prompt_attention_workspace_size(10, 2, 8, 2, 192)
    assert e.value.code == dm.DCP_ERR_UNSUPPORTED
    small, large = (dm.dcp_prompt_attention_workspace_size(n, 4, 8, 2, 128) for n in (10, 100000))
    assert 0 < small < large


def test_gather_refusals(dm):
    d, lib = _dims(dm), dm.load()

    def call(kv_heads=4, dim=64, cu=P, k=P, dtype=2, ranks=(0, 2), rows=5, out=P):
        return lib.dcp_gqa_kv_gather(ctypes.byref(d), kv_heads, dim, None, cu, P, k, P, dtype, None, None, *ranks, rows,
                                     out, P, P, None)

    for kw, code, word in ((dict(dim=96), 2, "head_dim"), (dict(kv_heads=0), 1, "kv_heads"), (dict(dtype=3), 1, "kv_dtype"),
                           (dict(cu=None), 1, "NULL"), (dict(k=P + 8), 1, "aligned"), (dict(out=P + 4), 1, "aligned"),
                           (dict(ranks=(1, 2)), 1, "rank range"), (dict(rows=-1), 1, "max_rows")):
        assert call(**kw) == code and word in dm.dcp_last_error(), kw
    assert call(rows=0, cu=None) == 0


def test_row_bytes(dm):
    for heads, dim in ((1, 64), (3, 64), (1, 128), (8, 128), (5, 128)):
        n = heads * dim
        assert dm.dcp_gqa_row_bytes(heads, dim, dm.KV_NVFP4) == oracle.fp4.row_bytes(n)
        assert dm.dcp_gqa_row_bytes(heads, dim, dm.KV_FP8_E4M3) == n
        assert dm.dcp_gqa_row_bytes(heads, dim, dm.KV_BF16) == 2 * n
    for bad in ((0, 64, 2), (1, 96, 2), (1, 64, 9)):
        with pytest.raises(dm.DcpError):
            dm.dcp_gqa_row_bytes(*bad)


def test_4_bit_pools_are_the_grouped_head_calls_alone(dm):
    d, lib = _dims(dm, num_splits=1), dm.load()
    assert lib.dcp_mla_partial(ctypes.byref(d), P, P, 2, None, 0.1, 0, 2, P, P, P, P, P, P, P, None, P, None) == 1
    assert "kv_dtype" in dm.dcp_last_error()
    assert lib.dcp_kv_write(ctypes.byref(d), P, P, 2, None, 2, P, P, None) == 1 and "kv_dtype" in dm.dcp_last_error()


def test_python_checks_tensors(dm):
    d = _dims(dm)
    t = torch.zeros(64, dtype=torch.int32)
    x = torch.zeros(2, 4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA device"):
        dm.dcp_kv_plan(d, t, t, t, t, t, t, t, 0, 2, t, t, t, t, t)
    with pytest.raises(ValueError, match="CUDA device"):
        dm.dcp_rope(t, t, 1.0, 64, False, x)
    with pytest.raises(TypeError, match="q must be"):
        dm.dcp_rope(t, t, 1.0, 64, False, x.float())
    with pytest.raises(ValueError, match="CUDA device"):
        dm.dcp_prompt_attention(1, True, t, t, x, x, x, 0.1, x, x.float(), t, t)
    with pytest.raises(ValueError, match="max_rows"):
        dm.PagePlan(d, 0, device="cpu")


def test_rope_table_with_the_slow_end_behind_the_last_pair(dm):
    # the pair that turns once within the original length is the 34.6th of 32, or the 64.3rd of 64: the
    # ramp goes on behind the last pair, by the formula, with ends worked out by hand
    for rot, original, lo, hi in ((64, 131072.0, 22, 35), (128, 65536.0, 40, 65)):
        table, _ = dm.dcp_rope_table(rot, 1e4, dm.RopeScaling(2, 4.0, original, 32.0, 1.0, 0.0))
        for i, x in enumerate(table):
            f = 1e4 ** (-2 * i / rot)
            r = max(0, i - lo) / (hi - lo)
            want = (f * (1 - r) + f / 4 * r) / (2 * np.pi)
            assert abs(x / 2.0 ** 64 - want) <= 2.0 ** -50 * want + 2.0 ** -64, (rot, i)


def test_rope_refuses_rows_that_lie_on_other_rows_heads(dm):
    # both strides leave room for a head, but places (row, head) coincide or overlap: counted out place
    # by place
    from decode_context_mla_causal_gb300.binding import RopeHeads

    def call(rows, heads, row, head, dim=64):
        a = RopeHeads(P, 1 << 30, 8 * dim, dim, row, head, heads)
        return dm.load().dcp_rope(rows, dim, 64, 0, P, P, 1.0, ctypes.byref(a), None, None)

    for rows, heads, row, head in ((2, 2, 64, 64), (3, 8, 448, 64), (2, 9, 512, 64), (5, 2, 64, 256), (2, 3, 128, 72),
                                   (3, 4, -192, 128), (100, 7, 128, 192), (6, 5, 256, -320), (2, 2, 1 << 62, 1 << 62)):
        at = sorted(i * row + j * head for i in range(rows) for j in range(heads))
        assert any(b - a < 64 for a, b in zip(at, at[1:])), (rows, heads, row, head)
        assert call(rows, heads, row, head) == dm.DCP_ERR_INVALID_ARG and "overlap" in dm.dcp_last_error(), (rows, row, head)
