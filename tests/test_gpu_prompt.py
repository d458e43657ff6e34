"""Attention of packed prompts on the GPU against the float64 oracle, at the sizes, layouts and
masks where it can go wrong."""

import math

import numpy as np
import pytest
import torch

import oracle
from tests import _cache_helpers as ch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dm():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    import decode_context_mla_causal_gb300 as mod

    return mod


def _cu(lens, first=0):
    return [first + sum(lens[:i]) for i in range(len(lens) + 1)]


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _inputs(rows, keys, heads, kv, dim, vdim, seed, big=1.0):
    g = torch.Generator().manual_seed(seed)
    return ((torch.randn(rows, heads, dim, generator=g) * big).bfloat16(),
            torch.randn(keys, kv, dim, generator=g).bfloat16(), torch.randn(keys, kv, vdim, generator=g).bfloat16())


def _assert(out, lse, ref, dim, what=""):
    """Rows of no sequence hold what they held (7); the others as the decode's tolerance."""
    rows = ~np.isnan(ref["lse"])
    o, s = ch.f64(out), ch.f64(lse)
    assert (o[~rows] == 7).all() and (s[~rows] == 7).all(), what
    at = rows.all(1)
    ch.assert_gqa(torch.tensor(o[at]), torch.tensor(s[at]), {n: x[at] for n, x in ref.items()}, dim, what)


def _run(dm, q, k, v, cu_q, cu_k, scale, causal=True, step=None):
    if step is None:
        step = dm.PromptAttention(q.shape[1], k.shape[1], q.shape[2], v.shape[2], max_rows=q.shape[0],
                                  max_seqs=len(cu_q) - 1, causal=causal)
    step.out.fill_(7.0)
    step.lse.fill_(7.0)
    step.workspace.fill_(0xFF)  # whatever it held
    out, lse = step(q.cuda(), k.cuda(), v.cuda(), _i32(cu_q), _i32(cu_k), scale)
    torch.cuda.synchronize()
    return out, lse, step


CASES = [  # rows of each sequence, keys in front of them, heads, kv_heads, dim, vdim
    ([1], 0, 1, 1, 64, 64),                       # one row, one key
    ([1, 2, 3], 0, 8, 8, 128, 128),
    ([5], 0, 4, 2, 192, 128),
    ([200], 0, 4, 1, 128, 128),
    ([127, 128, 129], 0, 2, 2, 64, 64),           # around a tile
    ([33, 1, 250], 0, 10, 2, 128, 128),           # groups of five: 125 rows of a tile
    ([70, 300], 0, 7, 1, 192, 128),
    ([40, 9], 0, 34, 2, 64, 64),                  # an odd group of 17
    ([6, 3], 0, 200, 1, 128, 128),                # more heads in a group than a tile has rows
    ([130], 0, 128, 1, 64, 64),                   # one token to a tile
    ([600, 0, 513], 0, 2, 2, 128, 128),           # several items, an empty sequence between
    ([20, 1, 65], 300, 4, 2, 128, 128),           # behind a context
    ([64], 1000, 2, 1, 192, 128),
    ([1, 1, 1, 1], 77, 8, 2, 64, 64),             # single tokens behind a context
    ([257, 255], 128, 3, 3, 64, 64),
]


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{'-'.join(map(str, c[0]))}+{c[1]}:{c[2]}:{c[3]}x{c[4]}")
def test_prompt_against_the_oracle(dm, case, causal):
    lens, ctx, H, K, d, dv = case
    cu_q, cu_k = _cu(lens), _cu([n + ctx if n else 0 for n in lens])
    q, k, v = _inputs(cu_q[-1], cu_k[-1], H, K, d, dv, sum(lens) + H)
    scale = d ** -0.5
    out, lse, step = _run(dm, q, k, v, cu_q, cu_k, scale, causal)
    assert step.read_status() == 0
    ref = oracle.prompt.attend(q=ch.f64(q), k=ch.f64(k), v=ch.f64(v), cu_q=cu_q, cu_k=cu_k, softmax_scale=scale,
                               causal=causal)
    _assert(out, lse, ref, d)
    first = (out.clone(), lse.clone())
    again = _run(dm, q, k, v, cu_q, cu_k, scale, causal)
    assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


@pytest.mark.parametrize("causal", [True, False])
def test_prompt_rows_without_a_key(dm, causal):
    # fewer keys than rows: the first rows see none; no keys at all; padding in front and behind
    lens, keys = [9, 140, 4, 30], [5, 20, 0, 30]
    cu_q, cu_k = _cu(lens, 3), _cu(keys, 2)
    q, k, v = _inputs(cu_q[-1] + 6, cu_k[-1] + 9, 6, 2, 128, 128, 5)
    q[:3], q[cu_q[-1]:] = math.nan, math.inf
    for x in (k, v):
        x[:2], x[cu_k[-1]:] = math.nan, math.inf
    out, lse, step = _run(dm, q, k, v, cu_q, cu_k, 0.1, causal)
    assert step.read_status() == 0
    ref = oracle.prompt.attend(q=ch.f64(q), k=ch.f64(k), v=ch.f64(v), cu_q=cu_q, cu_k=cu_k, softmax_scale=0.1,
                               causal=causal)
    assert np.isneginf(ref["lse"]).any()
    _assert(out, lse, ref, 128)
    # an empty k and v
    step = dm.PromptAttention(6, 2, 128, 128, max_rows=q.shape[0], max_seqs=4, causal=causal)
    out, lse = step(q.cuda(), k[:0].cuda(), v[:0].cuda(), _i32(cu_q), _i32([0] * 5), 0.1)
    assert bool((out[3:cu_q[-1]] == 0).all()) and bool(torch.isneginf(lse[3:cu_q[-1]]).all())
    assert step.read_status() == 0


@pytest.mark.parametrize("dim,vdim", [(64, 64), (128, 128), (192, 128)])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_prompt_what_a_row_does_not_see_never_meets_it(dm, dim, vdim, bad):
    # infinities and NaN in k and v from one key on, of one sequence: the rows in front of it and
    # the sequences beside it are as with finite values, the rows that see it are not
    lens, at = [150, 300, 140], 150 + 170
    cu = _cu(lens)
    q, k, v = _inputs(cu[-1], cu[-1], 4, 2, dim, vdim, 9)
    clean = _run(dm, q, k, v, cu, cu, 0.1)
    keep = [x.clone() for x in clean[:2]]
    v2 = v.clone()
    v2[at, :, 5], v2[at + 60, 0, vdim - 1] = bad, bad
    out, lse, step = _run(dm, q, k, v2, cu, cu, 0.1)
    same = torch.ones_like(out, dtype=torch.bool)
    same[at:450, :, 5] = False
    same[at + 60:450, :2, vdim - 1] = False
    assert torch.equal(out[same], keep[0][same]) and torch.equal(lse, keep[1])
    hit = out[~same].float()
    assert bool((torch.isnan(hit) if math.isnan(bad) else hit == bad).all())
    # in the keys: scores of nan, or of either infinity, from there on
    k2 = k.clone()
    k2[at:450] = bad
    out, lse, step = _run(dm, q, k2, v, cu, cu, 0.1)
    rows = torch.ones(cu[-1], dtype=torch.bool)
    rows[at:450] = False
    assert torch.equal(out[rows], keep[0][rows]) and torch.equal(lse[rows], keep[1][rows])
    assert not bool(torch.isfinite(lse[at:450]).all())
    assert step.read_status() == 0


@pytest.mark.parametrize("big", [30.0, 300.0])
def test_prompt_large_scores(dm, big):
    # scores far apart: the running maximum jumps, and most weights vanish
    cu = _cu([400, 260])
    q, k, v = _inputs(cu[-1], cu[-1], 2, 1, 128, 128, 4, big)
    out, lse, _ = _run(dm, q, k, v, cu, cu, 0.125)
    _assert(out, lse, oracle.prompt.attend(q=ch.f64(q), k=ch.f64(k), v=ch.f64(v), cu_q=cu, cu_k=cu,
                                           softmax_scale=0.125), 128)


def test_prompt_rising_and_falling_scores(dm):
    # keys whose scores rise tile by tile (every tile moves the maximum), and fall
    cu = _cu([700])
    q, k, v = _inputs(700, 700, 2, 2, 64, 64, 6)
    ramp = torch.linspace(0, 40, 700)
    q[..., 0] = 8.0
    k[:, 0, 0], k[:, 1, 0] = ramp.bfloat16(), (-ramp).bfloat16()
    out, lse, _ = _run(dm, q, k, v, cu, cu, 0.125)
    _assert(out, lse, oracle.prompt.attend(q=ch.f64(q), k=ch.f64(k), v=ch.f64(v), cu_q=cu, cu_k=cu,
                                           softmax_scale=0.125), 64)


def test_prompt_strided_views(dm):
    # q, k and v of one projection's rows, and k and v of rows of 128 + 128 by head
    lens = [60, 200]
    cu = _cu(lens)
    g = torch.Generator().manual_seed(2)
    fused = torch.randn(260, 8 + 2 + 2, 128, generator=g).bfloat16().cuda()
    q, k, v = fused[:, :8], fused[:, 8:10], fused[:, 10:]
    step = dm.PromptAttention(8, 2, 128, 128, max_rows=300, max_seqs=2)
    out, lse = step(q, k, v, _i32(cu), _i32(cu), 0.1)
    ref = oracle.prompt.attend(q=ch.f64(q), k=ch.f64(k), v=ch.f64(v), cu_q=cu, cu_k=cu, softmax_scale=0.1)
    _assert(out, lse, ref, 128)
    both = torch.randn(260, 3, 256, generator=g).bfloat16().cuda()
    rot = torch.randn(260, 3, 192, generator=g).bfloat16().cuda()
    step = dm.PromptAttention(3, 3, 192, 128, max_rows=260, max_seqs=2)
    out, lse = step(rot, rot, both[..., 128:], _i32(cu), _i32(cu), 0.07)
    ref = oracle.prompt.attend(q=ch.f64(rot), k=ch.f64(rot), v=ch.f64(both[..., 128:]), cu_q=cu, cu_k=cu,
                               softmax_scale=0.07)
    _assert(out, lse, ref, 192)


@pytest.mark.parametrize("dim,vdim", [(64, 64), (128, 128), (192, 128)])
def test_prompt_pieces_do_not_meet_newer_keys(dm, dim, vdim):
    # a unit cut into pieces, of which the last holds a value that only the later rows see
    lens, ctx, at = [40, 30], 7000, 20
    cu_q, cu_k = _cu(lens), _cu([n + ctx for n in lens])
    q, k, v = _inputs(cu_q[-1], cu_k[-1], 4, 2, dim, vdim, 21)
    out, lse, _ = _run(dm, q, k, v, cu_q, cu_k, 0.1)
    keep = out.clone(), lse.clone()
    v[ctx + at, 1, 7] = math.inf
    v[cu_k[1] + ctx + at, 0, 2] = math.nan
    out, lse, step = _run(dm, q, k, v, cu_q, cu_k, 0.1)
    assert step.read_status() == 0 and torch.equal(lse, keep[1])
    same = torch.ones_like(out, dtype=torch.bool)
    same[at:40, 2:, 7] = False
    same[40 + at:, :2, 2] = False
    assert torch.equal(out[same], keep[0][same])
    assert bool((out[at:40, 2:, 7] == math.inf).all()) and bool(torch.isnan(out[40 + at:, :2, 2]).all())


@pytest.mark.parametrize("dim,vdim", [(64, 64), (128, 128), (192, 128)])
def test_prompt_several_units_to_an_sm(dm, dim, vdim):
    # more units of a K/V head than SMs, some without a key; whichever SM takes them, and in the second
    # pass where a value meets the later rows alone, the result is the same bit for bit
    lens, heads = [700] * 6 + [300, 1], 16
    cu_q, cu_k = _cu(lens), _cu([700] * 6 + [0, 1])
    q, k, v = _inputs(cu_q[-1], cu_k[-1], heads, heads, dim, vdim, 31)
    out, lse, step = _run(dm, q, k, v, cu_q, cu_k, 0.1)
    keep = out.clone(), lse.clone()
    at = [3, 2, 9, 15]
    ref = oracle.prompt.attend(q=ch.f64(q[:, at]), k=ch.f64(k[:, at]), v=ch.f64(v[:, at]), cu_q=cu_q, cu_k=cu_k,
                               softmax_scale=0.1)
    _assert(out[:, at], lse[:, at], ref, dim)
    for i in range(3):
        again = _run(dm, q, k, v, cu_q, cu_k, 0.1, step=step)
        assert torch.equal(again[0], keep[0]) and torch.equal(again[1], keep[1])
    same = torch.ones_like(out, dtype=torch.bool)
    for b, h, t in ((0, 1, 20), (2, 5, 300), (2, 11, 699), (5, 0, 513), (5, 15, 128)):
        v[cu_k[b] + t, h, 7] = math.nan
        same[cu_q[b] + t:cu_q[b + 1], h, 7] = False
    for i in range(2):
        out, lse, _ = _run(dm, q, k, v, cu_q, cu_k, 0.1, step=step)
        assert torch.equal(lse, keep[1]) and torch.equal(out[same], keep[0][same])
        assert bool(torch.isnan(out[~same]).all())
    assert step.read_status() == 0


def test_prompt_one_row_of_a_view(dm):
    # single rows and heads have strides that mean nothing
    g = torch.Generator().manual_seed(5)
    base = torch.randn(4, 6, 128, generator=g).bfloat16().cuda()
    step = dm.PromptAttention(1, 1, 128, 128, max_rows=1, max_seqs=1)
    out, lse = step(base[1:2, 2:3], base[:, 3:4], base[:, 4:5], _i32([0, 1]), _i32([0, 4]), 0.3)
    ref = oracle.prompt.attend(q=ch.f64(base[1:2, 2:3]), k=ch.f64(base[:, 3:4]), v=ch.f64(base[:, 4:5]), cu_q=[0, 1],
                               cu_k=[0, 4], softmax_scale=0.3)
    _assert(out, lse, ref, 128)


def test_prompt_many_sequences(dm):
    # more sequences than the item kernel has threads, most of them a token or none
    lens = [(i * 7) % 4 for i in range(1500)] + [150]
    cu = _cu(lens)
    q, k, v = _inputs(cu[-1], cu[-1], 2, 1, 64, 64, 8)
    out, lse, step = _run(dm, q, k, v, cu, cu, 0.2)
    assert step.read_status() == 0
    _assert(out, lse, oracle.prompt.attend(q=ch.f64(q), k=ch.f64(k), v=ch.f64(v), cu_q=cu, cu_k=cu,
                                           softmax_scale=0.2), 64)


def test_prompt_bad_offsets_set_status(dm):
    # offsets that fall or leave the rows: those sequences are left out, the others are served
    q, k, v = _inputs(100, 100, 2, 2, 64, 64, 3)
    for cu_q, cu_k, good in (([0, 40, 30, 90], [0, 40, 30, 90], [(0, 40), (30, 90)]),
                             ([0, 40, 100, 130], [0, 40, 100, 130], [(0, 40), (40, 100)]),
                             ([-5, 40, 100, 100], [0, 40, 100, 100], [(40, 100)]),
                             ([0, 40, 100, 100], [0, 140, 40, 100], [])):
        out, lse, step = _run(dm, q, k, v, cu_q, cu_k, 0.2)
        assert step.read_status() == dm.STATUS_BAD_SEQ_LEN
        seen = torch.zeros(100, dtype=torch.bool)
        for a, b in good:
            ref = oracle.prompt.attend(q=ch.f64(q[a:b]), k=ch.f64(k[a:b]), v=ch.f64(v[a:b]), cu_q=[0, b - a],
                                       cu_k=[0, b - a], softmax_scale=0.2)
            if not bool(seen[a:b].any()) and (a, b) != (0, 40):
                _assert(out[a:b], lse[a:b], ref, 64)
            seen[a:b] = True
        assert bool((out[~seen] == 7).all()) and bool((lse[~seen] == 7).all())


def test_prompt_in_a_graph_and_on_two_streams(dm):
    lens = [90, 200]
    cu = _cu(lens)
    q, k, v = (x.cuda() for x in _inputs(290, 290, 8, 2, 128, 128, 3))
    cu_q = _i32(cu)
    a, b = (dm.PromptAttention(8, 2, 128, 128, max_rows=290, max_seqs=2) for _ in range(2))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        a(q, k, v, cu_q, cu_q, 0.1)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        a(q, k, v, cu_q, cu_q, 0.1)
    for lens in ([90, 200], [1, 150], [289, 1], [0, 0]):
        cu = _cu(lens)
        cu_q.copy_(torch.tensor(cu, dtype=torch.int32))
        a.out.fill_(7.0)
        a.lse.fill_(7.0)
        torch.cuda.synchronize()
        g.replay()
        with torch.cuda.stream(side):
            out, lse = b(q, k, v, _i32(cu), _i32(cu), 0.1)
        torch.cuda.synchronize()
        n = cu[-1]
        assert torch.equal(a.out[:n], out[:n]) and torch.equal(a.lse[:n], lse[:n])
        assert bool((a.out[n:] == 7).all())
        ref = oracle.prompt.attend(q=ch.f64(q), k=ch.f64(k), v=ch.f64(v), cu_q=cu, cu_k=cu, softmax_scale=0.1)
        _assert(a.out, a.lse, ref, 128)
    assert a.read_status() == 0 and b.read_status() == 0


def test_prompt_more_items_than_sms(dm):
    # every CTA takes several items, of different lengths: all roles go on from one to the next
    lens = [1500, 40, 700, 5, 900]
    cu = _cu(lens)
    q, k, v = _inputs(cu[-1], cu[-1], 32, 16, 64, 64, 12)
    out, lse, step = _run(dm, q, k, v, cu, cu, 0.125)
    assert step.read_status() == 0
    qd, kd, vd = (x.cuda().double() for x in (q, k, v))
    for b, n in enumerate(lens):
        of = slice(cu[b], cu[b + 1])
        kk, vv = (x[of].repeat_interleave(2, dim=1).permute(1, 0, 2) for x in (kd, vd))
        x = (qd[of].permute(1, 0, 2) @ kk.transpose(1, 2)) * 0.125
        x.masked_fill_(torch.ones(n, n, dtype=torch.bool, device="cuda").triu_(1), -math.inf)
        w = x.softmax(-1)
        ref, absv = (w @ vv).permute(1, 0, 2), (w @ vv.abs()).permute(1, 0, 2)
        # weights and output are rounded to bf16; scores of 64 products of N(0, 1) values: 2^-17
        assert bool(((out[of].double() - ref).abs() <= 2.0 ** -8 * (absv + ref.abs()) + 2.0 ** -16 * absv).all())
        assert bool(((lse[of].double() - x.logsumexp(-1).T).abs() <= 2.0 ** -17).all())


@pytest.mark.parametrize("lens,ctx,heads,kv,dim,vdim,causal", [
    ([5], 20000, 8, 2, 128, 128, True),         # few rows behind a long context: many pieces to a unit
    ([300, 1], 9000, 2, 1, 64, 64, True),
    ([40], 6000, 3, 3, 192, 128, True),
    ([200, 0, 70], 5000, 4, 2, 128, 128, False),
    ([2048], 2048, 16, 16, 64, 64, True),       # more units than SMs, in uneven waves
])
def test_prompt_cut_into_pieces(dm, lens, ctx, heads, kv, dim, vdim, causal):
    cu_q, cu_k = _cu(lens), _cu([n + ctx if n else 0 for n in lens])
    q, k, v = _inputs(cu_q[-1], cu_k[-1], heads, kv, dim, vdim, 17)
    k[cu_k[-2] + 7, :, 0] = 60.0                # one key far above the others, for half of the rows
    scale = dim ** -0.5
    out, lse, step = _run(dm, q, k, v, cu_q, cu_k, scale, causal)
    assert step.read_status() == 0
    first = out.clone(), lse.clone()
    again = _run(dm, q, k, v, cu_q, cu_k, scale, causal)
    assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
    for b, n in enumerate(lens):
        of, ok = slice(cu_q[b], cu_q[b + 1]), slice(cu_k[b], cu_k[b + 1])
        for h in range(heads if n else 0):
            kk, vv, qq = k[ok, h * kv // heads].cuda().double(), v[ok, h * kv // heads].cuda().double(), q[of, h].cuda().double()
            x = (qq @ kk.T) * scale
            if causal:
                x.masked_fill_(torch.ones_like(x, dtype=torch.bool).triu_(x.shape[1] - n + 1), -math.inf)
            w = x.softmax(-1)
            ref, absv = w @ vv, w @ vv.abs()
            ds = (dim + 4) * 2.0 ** -23 * scale * (qq.abs() @ kk.abs().T).amax(1) + 2.0 ** -20
            assert bool(((out[of, h].double() - ref).abs() <= 2.0 ** -8 * (absv + ref.abs()) + 2 * ds[:, None] * absv).all())
            fin = x.logsumexp(-1)
            assert bool(((lse[of, h].double() - fin).abs() <= ds + 2.0 ** -22 * fin.abs()).all())
    # a value that is not finite in the middle of the context reaches every row, through every join
    v[cu_k[-2] + 700, 0, 3] = math.nan
    out, lse, _ = _run(dm, q, k, v, cu_q, cu_k, scale, causal)
    last, group = slice(cu_q[-2], cu_q[-1]), heads // kv
    assert bool(torch.isnan(out[last, :group, 3]).all()) and torch.equal(lse, first[1])
    same = torch.ones_like(out, dtype=torch.bool)
    same[last, :group, 3] = False
    assert torch.equal(out[same], first[0][same])


@pytest.mark.parametrize("lens,ctx,heads,kv,dim,causal", [
    ([2560], 440, 16, 2, 128, False),         # eighty items of one length: three warps sort them
    ([300, 1900, 360], 440, 16, 2, 64, False),
    ([2048], 32832, 64, 8, 128, True),        # a context that is no multiple of a tile: ties across warps
    ([5120], 0, 8, 1, 128, False),            # more items than are placed by comparison
    ([35200], -27200, 8, 1, 64, False),       # more items than threads
])
def test_prompt_cut_units_repeat_themselves(dm, lens, ctx, heads, kv, dim, causal):
    # where items tie for their place in the list, which units are cut must not depend on the order
    # in which warps come by: the result is the same bit for bit, also beside other work
    cu_q, cu_k = _cu(lens), _cu([n + ctx for n in lens])
    g = torch.Generator(device="cuda").manual_seed(3)
    q, k, v = (torch.randn(n, h, dim, generator=g, device="cuda").bfloat16()
               for n, h in ((cu_q[-1], heads), (cu_k[-1], kv), (cu_k[-1], kv)))
    step = dm.PromptAttention(heads, kv, dim, dim, max_rows=cu_q[-1], max_seqs=len(lens), causal=causal)
    cu_q, cu_k = _i32(cu_q), _i32(cu_k)
    out, lse = step(q, k, v, cu_q, cu_k, dim ** -0.5)
    keep = out.clone(), lse.clone()
    other, side = torch.zeros(1 << 26, device="cuda"), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for i in range(40):
        if i % 2:
            with torch.cuda.stream(side):
                other.add_(1.0)
        out, lse = step(q, k, v, cu_q, cu_k, dim ** -0.5)
        assert torch.equal(out, keep[0]) and torch.equal(lse, keep[1]), i
    torch.cuda.synchronize()
    assert step.read_status() == 0


def test_prompt_sequences_beside_bad_ones_are_served(dm):
    # in front of a sequence whose offsets fall or leave the rows, and behind it
    q, k, v = _inputs(100, 100, 2, 2, 64, 64, 3)
    for cu_q, cu_k, good, skip in (
            ([0, 40, 100, 130], [0, 40, 100, 130], [((0, 40), (0, 40)), ((40, 100), (40, 100))], []),
            ([0, 40, 30, 90], [0, 40, 30, 90], [((0, 40), (0, 40)), ((30, 90), (30, 90))], range(30, 40)),  # two write 30..39
            ([0, 40, 60, 100], [0, 40, 10, 100], [((0, 40), (0, 40)), ((60, 100), (10, 100))], []),
            ([0, 25, 25, 70], [0, 25, 140, 30], [((0, 25), (0, 25))], [])):
        out, lse, step = _run(dm, q, k, v, cu_q, cu_k, 0.2)
        assert step.read_status() == dm.STATUS_BAD_SEQ_LEN
        left = torch.ones(100, dtype=torch.bool)
        for (a, b), (c, d) in good:
            ref = oracle.prompt.attend(q=ch.f64(q[a:b]), k=ch.f64(k[c:d]), v=ch.f64(v[c:d]), cu_q=[0, b - a],
                                       cu_k=[0, d - c], softmax_scale=0.2)
            own = [i for i in range(a, b) if i not in skip]
            at = [i - a for i in own]
            _assert(out[own], lse[own], {n: x[at] for n, x in ref.items()}, 64)
            left[a:b] = False
        assert bool((out[left] == 7).all()) and bool((lse[left] == 7).all())
