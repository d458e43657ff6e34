"""Grouped-head K/V caches on the GPU: the write bit for bit, the attention against the
float64 oracle, each at the sizes and masks where it can go wrong."""

import numpy as np
import pytest
import torch

import oracle
from oracle import kv_write as okw
from tests import _cache_helpers as ch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dm():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    import decode_context_mla_causal_gb300 as mod

    return mod


def _q(rows, heads, dim, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(rows, heads, dim, generator=g).bfloat16()


def _ref(c, q, qlen, scale, causal=True, **kw):
    return oracle.gqa.decode(q=ch.f64(q), k_pools=ch.raw(c.pools[0]), v_pools=ch.raw(c.pools[1]),
                             block_table=c.table.numpy(), seq_lens=c.lens, qlen=qlen, kv_dtype=c.dtype,
                             k_scale=c.scale, v_scale=c.scale * (1.5 if c.dtype == "fp8" else 1.0),
                             softmax_scale=scale, causal=causal, **c.geometry, **kw)


def _run(dm, c, q, qlen, hkv, dim, scale, splits, causal=True, rank_begin=0, num_ranks=None, step=None):
    dims = c.dims(dm, qlen, q.shape[1], splits, causal)
    if step is None:
        step = dm.GqaDecode(dims, hkv, dim, c.kv_dtype(dm), rank_begin=rank_begin, num_ranks=num_ranks)
    of = slice(rank_begin, rank_begin + step.num_ranks)
    step.out.fill_(float("nan"))
    step.lse.fill_(float("nan"))
    step.workspace.fill_(0xFF)                     # whatever it held
    out, lse = step(q.cuda(), c.pools[0][of].cuda().contiguous(), c.pools[1][of].cuda().contiguous(),
                    c.dev_scale(), c.dev_scale(1.5), scale, c.lens_dev(), c.table.cuda())
    torch.cuda.synchronize()
    return out, lse, step


CASES = [  # lens, qlen, heads, kv_heads, dim, dcp, interleave, block, dtype, splits
    ([1], 1, 1, 1, 64, 1, 1, 1, "bf16", 1),                       # one token, one head, one-token blocks
    ([1, 2, 3], 1, 8, 8, 128, 4, 1, 16, "fp8", 1),                # ranks without a token, no groups
    ([200], 1, 32, 8, 128, 2, 1, 16, "bf16", 3),
    ([65, 64, 63, 1], 1, 10, 2, 64, 1, 8, 8, "fp8", 2),           # groups of five, lengths around a tile
    ([700, 31], 2, 40, 8, 128, 3, 6, 24, "bf16", 4),              # blocks of 24, twenty rows to a K/V head
    ([513, 1030, 4], 4, 64, 4, 128, 2, 64, 64, "fp8", 5),         # 64 rows to a K/V head
    ([300, 129], 3, 16, 1, 64, 8, 1, 96, "bf16", 2),              # one K/V head, 48 rows
    ([1000], 1, 17, 1, 128, 1, 1, 128, "fp8", 7),                 # an odd group of 17
    ([2500, 9, 1777], 1, 16, 16, 64, 2, 1, 5, "bf16", 6),         # odd blocks, sixteen K/V heads
    ([90], 7, 6, 2, 128, 1, 3, 3, "fp8", 64),                     # more pieces than there is length
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{c[1]}x{c[2]}:{c[3]}x{c[4]}-W{c[5]}-bs{c[7]}-{c[8]}")
def test_decode_against_the_oracle(dm, case):
    lens, qlen, H, hkv, dim, W, S, bs, dtype, splits = case
    c = ch.Cache([max(n, qlen) for n in lens], dcp=W, interleave=S, block=bs, tails=[(hkv, dim)] * 2,
                 dtype=dtype, seed=sum(lens) + H)
    q = _q(c.B * qlen, H, dim, 7)
    scale = dim ** -0.5
    out, lse, step = _run(dm, c, q, qlen, hkv, dim, scale, splits)
    assert step.read_status() == 0
    ch.assert_gqa(out, lse, _ref(c, q, qlen, scale), dim)
    first = (out.clone(), lse.clone())
    again = _run(dm, c, q, qlen, hkv, dim, scale, splits)
    assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
def test_decode_not_causal_and_empty_sequences(dm, dtype):
    # every row sees the whole sequence; a padded batch slot of length 0 sees nothing
    c = ch.Cache([0, 37, 0, 2], dcp=2, interleave=1, block=16, tails=[(2, 64)] * 2, dtype=dtype, seed=3)
    q = _q(c.B * 3, 8, 64, 5)
    out, lse, step = _run(dm, c, q, 3, 2, 64, 0.2, 2, causal=False)
    assert step.read_status() == 0
    ch.assert_gqa(out, lse, _ref(c, q, 3, 0.2, causal=False), 64)


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
def test_decode_one_rank_per_call(dm, dtype):
    c = ch.Cache([150, 3], dcp=4, interleave=4, block=8, tails=[(2, 128)] * 2, dtype=dtype, seed=9)
    q = _q(c.B, 6, 128, 5)
    for r in range(4):
        out, lse, step = _run(dm, c, q, 1, 2, 128, 0.1, 3, rank_begin=r, num_ranks=1)
        assert step.read_status() == 0
        ch.assert_gqa(out, lse, _ref(c, q, 1, 0.1, ranks=[r]), 128, r)


@pytest.mark.parametrize("big", [30.0, 300.0])
def test_decode_large_scores(dm, big):
    # scores far apart: the running maximum jumps, and most weights vanish
    c = ch.Cache([400, 90], dcp=2, interleave=1, block=32, tails=[(2, 64)] * 2, dtype="bf16", seed=4)
    q = (_q(c.B, 8, 64, 6).float() * big).bfloat16()
    out, lse, _ = _run(dm, c, q, 1, 2, 64, 0.125, 3)
    ch.assert_gqa(out, lse, _ref(c, q, 1, 0.125), 64)


def test_decode_bad_inputs_set_status(dm):
    c = ch.Cache([120, 40, 60], dcp=2, interleave=1, block=16, tails=[(2, 64)] * 2, dtype="bf16", seed=8)
    q = _q(c.B * 2, 4, 64, 5)
    c.table[0, 1], c.table[2, 0] = c.NB + 5, -1
    out, lse, step = _run(dm, c, q, 2, 2, 64, 0.2, 2)
    assert step.read_status() == dm.STATUS_BAD_BLOCK_ID
    good = c.table.clamp(0, c.NB - 1)
    c2, c.table = c.table, good
    ref = _ref(c, q, 2, 0.2, skip=lambda b, li: not 0 <= int(c2[b, li // 16]) < c.NB)
    ch.assert_gqa(out, lse, ref, 64)
    # lengths below qlen, and above the static bound (clamped to it)
    c.lens = [1, 40, 60]
    _, lse, step = _run(dm, c, q, 2, 2, 64, 0.2, 2)
    assert step.read_status() == dm.STATUS_BAD_SEQ_LEN and bool(torch.isneginf(lse[0]).all())
    c.lens = [10 ** 6, 40, 60]
    _, _, step = _run(dm, c, q, 2, 2, 64, 0.2, 2)
    assert step.read_status() == dm.STATUS_LOCAL_OVER_BOUND


def test_decode_in_a_graph_and_on_two_streams(dm):
    c = ch.Cache([256, 190], dcp=2, interleave=1, block=16, tails=[(4, 128)] * 2, dtype="fp8", seed=2)
    q = _q(c.B, 16, 128, 3)
    dims = c.dims(dm, 1, 16, 4)
    k, v = (p.cuda() for p in c.pools)
    lens, table, qd = c.lens_dev(), c.table.cuda(), q.cuda()
    a, b = dm.GqaDecode(dims, 4, 128, dm.KV_FP8_E4M3), dm.GqaDecode(dims, 4, 128, dm.KV_FP8_E4M3)
    args = (qd, k, v, c.dev_scale(), c.dev_scale(1.5), 0.1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        a(*args, lens, table)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        a(*args, lens, table)
    for new in ([256, 190], [1, 64], [255, 17]):
        lens.copy_(torch.tensor(new, dtype=torch.int32))
        side.wait_stream(torch.cuda.current_stream())
        g.replay()
        with torch.cuda.stream(side):
            for _ in range(3):
                b(*args, lens, table)
        torch.cuda.synchronize()
        c.lens = new
        ref = _ref(c, q, 1, 0.1)
        ch.assert_gqa(a.out, a.lse, ref, 128, new)
        assert torch.equal(a.out, b.out) and torch.equal(a.lse, b.lse)
    assert a.read_status() == b.read_status() == 0


@pytest.mark.parametrize("hkv,dim,dtype,qlen", [(1, 64, "fp8", 1), (8, 128, "fp8", 3), (3, 128, "bf16", 5), (16, 64, "bf16", 40)])
def test_write_is_exact(dm, hkv, dim, dtype, qlen):
    c = ch.Cache([qlen, 3 * qlen + 50], dcp=3, interleave=4, block=8, tails=[(hkv, dim)] * 2, dtype=dtype, seed=qlen)
    dims = c.dims(dm, qlen, 8)
    g = torch.Generator().manual_seed(1)
    new = [(torch.randn(c.B * qlen, hkv, dim, generator=g) * 4).bfloat16() for _ in range(2)]
    new[0][0, 0, :4] = torch.tensor([float("inf"), -float("inf"), 0.0, -0.0])
    slots = torch.empty(3, c.B * qlen, dtype=torch.int32, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    dm.dcp_kv_slot_mapping(dims, c.lens_dev(), c.table.cuda(), 0, 3, slots, st)
    slots[1, -1] = c.NB * c.bs + 4                 # outside the pool: skipped and reported
    pools = [p.cuda() for p in c.pools]
    scales = (0.013, 0.4)
    ds = [torch.tensor([x], device="cuda") for x in scales] if dtype == "fp8" else [None, None]
    dm.dcp_gqa_kv_write(dims, hkv, dim, slots, new[0].cuda(), new[1].cuda(), c.kv_dtype(dm), *ds, 3, *pools, st)
    torch.cuda.synchronize()
    assert int(st.item()) == dm.STATUS_BAD_PAGE
    host = slots.cpu().numpy()
    host[host >= c.NB * c.bs] = -1
    for pool, before, x, scale in zip(pools, c.pools, new, scales):
        flat = ch.raw(before).reshape(3, c.NB, c.bs, hkv * dim)
        want = okw.write(flat, host, ch.raw(x).reshape(c.B * qlen, -1), dtype, scale)
        assert np.array_equal(ch.raw(pool).reshape(want.shape), want)


def test_write_then_decode_step_by_step(dm):
    # a sequence grows by two tokens a step: its rows are written, then attended
    W, S, bs, hkv, dim, H = 2, 2, 8, 2, 64, 6
    lens = [60, 37]
    c = ch.Cache(lens, dcp=W, interleave=S, block=bs, tails=[(hkv, dim)] * 2, dtype="fp8", seed=11, bound=64)
    dims = c.dims(dm, 2, H, 2)
    pools = [p.cuda() for p in c.pools]
    step = dm.GqaDecode(dims, hkv, dim, dm.KV_FP8_E4M3)
    slots = torch.empty(W, c.B * 2, dtype=torch.int32, device="cuda")
    for n in range(3):
        c.lens = [x + 2 for x in c.lens]
        new = [_q(c.B * 2, hkv, dim, 20 + 2 * n + i) for i in range(2)]
        q = _q(c.B * 2, H, dim, 40 + n)
        dm.dcp_kv_slot_mapping(dims, c.lens_dev(), c.table.cuda(), 0, W, slots, step.status)
        dm.dcp_gqa_kv_write(dims, hkv, dim, slots, new[0].cuda(), new[1].cuda(), dm.KV_FP8_E4M3, c.dev_scale(),
                            c.dev_scale(1.5), W, *pools, step.status)
        out, lse = step(q.cuda(), *pools, c.dev_scale(), c.dev_scale(1.5), 0.125, c.lens_dev(), c.table.cuda())
        torch.cuda.synchronize()
        assert step.read_status() == 0
        c.pools = [p.cpu() for p in pools]
        ch.assert_gqa(out, lse, _ref(c, q, 2, 0.125), dim, n)


@pytest.mark.parametrize("scale", [0.013, 1.0, 2.0 ** -7, 0.75, 3.3e4, 1e-31, 1e33, 1e-40, -0.5])
def test_write_divides_like_ieee(dm, scale):
    # every bf16 number: quotients on and next to a tie, subnormal, saturated, infinite, NaN
    bits = np.arange(65536, dtype=np.uint16)
    x = torch.from_numpy(bits.view(np.int16).copy()).view(torch.bfloat16).view(512, 1, 128)
    d = dm.make_dims(batch=512, qlen=1, num_heads=1, dcp=1, interleave=1, block_size=64, max_blocks_per_seq=1,
                     max_local_len=1, num_blocks=8, num_splits=1)
    pools = [torch.zeros(1, 8, 64, 1, 128, dtype=torch.uint8, device="cuda") for _ in range(2)]
    s = torch.tensor([scale], dtype=torch.float32, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    slots = torch.arange(512, dtype=torch.int32, device="cuda").view(1, 512)
    dm.dcp_gqa_kv_write(d, 1, 128, slots, x.cuda(), x.cuda(), dm.KV_FP8_E4M3, s, s, 1, *pools, st)
    with np.errstate(all="ignore"):
        want = okw.quantize_rows(bits.reshape(512, 128), np.float32(scale)).reshape(-1)
    for p in pools:
        got = p.cpu().numpy().reshape(-1)
        nan = want == 0x7F                         # either NaN code is a NaN
        assert np.array_equal(got[~nan], want[~nan]) and (got[nan] & 0x7F == 0x7F).all()
    assert int(st.item()) == 0


LONG = [  # lens, qlen, heads, kv_heads, dim, dcp, interleave, block, dtype: the work of several SMs per sequence
    ([9000, 4, 5000, 12001], 2, 64, 2, 64, 2, 1, 16, "fp8"),      # 64 rows to a K/V head
    ([7000, 333], 4, 24, 3, 128, 1, 8, 8, "bf16"),                # 32 rows, three K/V heads
    ([5000, 2600, 900], 1, 24, 12, 128, 2, 16, 32, "fp8"),        # twelve K/V heads
    ([4100], 5, 32, 2, 64, 3, 1, 24, "bf16"),                     # 80 rows
    ([30000], 1, 1, 1, 128, 1, 1, 64, "bf16"),                    # one head: one sequence on every SM
    ([2100] * 40, 1, 8, 1, 64, 1, 1, 64, "fp8"),                  # sequences across the shares' ends
]


@pytest.mark.parametrize("case", LONG, ids=lambda c: f"{c[1]}x{c[2]}:{c[3]}x{c[4]}-{max(c[0])}-{c[8]}")
def test_decode_long(dm, case):
    lens, qlen, H, hkv, dim, W, S, bs, dtype = case
    c = ch.Cache(lens, dcp=W, interleave=S, block=bs, tails=[(hkv, dim)] * 2, dtype=dtype, seed=len(lens) + H)
    q = _q(c.B * qlen, H, dim, 7)
    out, lse, step = _run(dm, c, q, qlen, hkv, dim, dim ** -0.5, 1)
    assert step.read_status() == 0
    ch.assert_gqa(out, lse, _ref(c, q, qlen, dim ** -0.5), dim)
    first = (out.clone(), lse.clone())
    again = _run(dm, c, q, qlen, hkv, dim, dim ** -0.5, 1)
    assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_decode_long_with_empty_sequences(dm):
    c = ch.Cache([0, 6000, 0, 0, 3000, 1, 0], dcp=2, interleave=1, block=16, tails=[(4, 128)] * 2, dtype="fp8", seed=3)
    q = _q(c.B * 2, 16, 128, 5)
    out, lse, step = _run(dm, c, q, 2, 4, 128, 0.1, 1, causal=False)
    assert step.read_status() == 0
    ch.assert_gqa(out, lse, _ref(c, q, 2, 0.1, causal=False), 128)
    for r in range(2):                             # a rank may hold none of a short one
        out, lse, step = _run(dm, c, q, 2, 4, 128, 0.1, 1, causal=False, rank_begin=r, num_ranks=1)
        ch.assert_gqa(out, lse, _ref(c, q, 2, 0.1, causal=False, ranks=[r]), 128)


@pytest.mark.parametrize("where", [0, 1])          # in K, in V
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_decode_rows_do_not_meet_tokens_they_do_not_see(dm, where, bad):
    # the last of three new tokens is not finite: the first two rows stay as they are
    c = ch.Cache([70, 33], dcp=2, interleave=1, block=16, tails=[(2, 64)] * 2, dtype="bf16", seed=8)
    q = _q(c.B * 3, 8, 64, 5)
    for b, n in enumerate(c.lens):
        p = n - 1
        c.pools[where][p % 2, c.table[b, p // 2 // 16], p // 2 % 16, 1, 7] = bad
    out, lse, step = _run(dm, c, q, 3, 2, 64, 0.2, 1)
    assert step.read_status() == 0
    with np.errstate(invalid="ignore"):
        ref = _ref(c, q, 3, 0.2)
    seen = np.array([2, 5])                        # rows that see it, through K/V head 1
    rows = np.array([0, 1, 3, 4])
    part = {k: v[rows] for k, v in ref.items()}
    ch.assert_gqa(out[torch.as_tensor(rows)], lse[torch.as_tensor(rows)], part, 64)
    o, s = ch.f64(out)[seen], ch.f64(lse)[seen]
    assert np.isfinite(o[:, :4]).all() and np.isfinite(s[:, :4]).all()
    if where == 1:
        assert not np.isfinite(o[:, 4:, 7]).any() and np.isfinite(s).all()
        assert np.isfinite(np.delete(o, 7, axis=2)).all()
    elif np.isnan(bad):
        assert np.isnan(o[:, 4:]).all() and np.isnan(s[:, 4:]).all()


def test_decode_of_nothing_but_nan_is_nan(dm):
    c = ch.Cache([40], dcp=1, interleave=1, block=16, tails=[(1, 64)] * 2, dtype="fp8", seed=8)
    c.pools[0].fill_(ch.NAN_CODE)
    out, lse, _ = _run(dm, c, _q(1, 4, 64, 5), 1, 1, 64, 0.2, 1)
    assert bool(torch.isnan(out).all()) and bool(torch.isnan(lse).all())


def test_offsets_past_32_bits(dm):
    NB, hkv, dim = 36000, 8, 128                   # pools of 4.7 GB whose last blocks are used
    c = ch.Cache([500, 90], dcp=1, interleave=1, block=64, tails=[(hkv, dim)] * 2, dtype="bf16", seed=2)
    far = torch.tensor([[NB - 1 - 2 * i for i in range(c.MB)], [NB - 2 - 2 * i for i in range(c.MB)]], dtype=torch.int32)
    big = []
    for p in c.pools:
        b = torch.empty((1, NB, 64, hkv, dim), dtype=p.dtype, device="cuda")
        assert b.numel() * b.element_size() > 1 << 32
        for i in range(2):
            for j in range(c.MB):
                b[0, int(far[i, j])] = p[0, int(c.table[i, j])].cuda()
        big.append(b)
    d = dm.make_dims(batch=2, qlen=1, num_heads=16, dcp=1, interleave=1, block_size=64, max_blocks_per_seq=c.MB,
                     max_local_len=c.ML, num_blocks=NB, num_splits=1)
    step = dm.GqaDecode(d, hkv, dim, dm.KV_BF16)
    q = _q(2, 16, dim, 3)
    out, lse = step(q.cuda(), *big, None, None, 0.1, c.lens_dev(), far.cuda())
    torch.cuda.synchronize()
    ch.assert_gqa(out, lse, _ref(c, q, 1, 0.1), dim)
    slots = torch.tensor([[int(far[0, 0]) * 64 + 63, -1]], dtype=torch.int32, device="cuda")
    new = _q(2, hkv, dim, 4)
    dm.dcp_gqa_kv_write(d, hkv, dim, slots, new.cuda(), new.cuda(), dm.KV_BF16, None, None, 1, *big, step.status)
    torch.cuda.synchronize()
    assert step.read_status() == 0
    for b in big:
        assert torch.equal(b[0, int(far[0, 0]), 63].cpu(), new[0])


def test_tensors_of_another_device_are_refused(dm, monkeypatch):
    c = ch.Cache([20], dcp=1, interleave=1, block=16, tails=[(1, 64)] * 2, dtype="bf16", seed=2)
    step = dm.GqaDecode(c.dims(dm, 1, 2), 1, 64, dm.KV_BF16)
    args = (_q(1, 2, 64, 1).cuda(), c.pools[0].cuda(), c.pools[1].cuda(), None, None, 0.1, c.lens_dev(), c.table.cuda())
    step(*args)
    monkeypatch.setattr(dm.binding, "_several_devices", True)
    step(*args)
    monkeypatch.setattr(dm.binding, "_current_device", lambda: 1)
    with pytest.raises(ValueError, match="is on cuda:0, the current device is cuda:1"):
        step(*args)
    torch.cuda.synchronize()


@pytest.mark.parametrize("bits", [25.3, 30.0])
@pytest.mark.parametrize("dim,dtype", [(64, "fp8"), (128, "fp8"), (128, "bf16")])
def test_decode_tail_behind_tokens_that_take_the_weight(dm, dim, dtype, bits):
    # every 50th token takes the weight and has no value; the others hold 2^-bits of it each, and the output
    # is theirs alone. The tolerance is of what they add, so each of their weights counts
    c = ch.Cache([900, 64, 20], dcp=2, interleave=1, block=16, tails=[(2, dim)] * 2, dtype=dtype, seed=5, scale=1.0)
    code = lambda x: (torch.tensor(x).to(torch.float8_e4m3fn).view(torch.uint8) if dtype == "fp8"  # noqa: E731
                      else torch.tensor(x).bfloat16())
    rng = np.random.default_rng(6)
    for b, n in enumerate(c.lens):
        for p in range(n):
            at = p % 2, c.table[b, p // 2 // 16], p // 2 % 16
            k = np.zeros((2, dim), np.float32)
            k[:, 3] = 32.0 * (p % 50 == 0)
            c.pools[0][at] = code(k)
            c.pools[1][at] = code((rng.uniform(1, 2, (2, dim)) * (p % 50 != 0)).astype(np.float32))
    q = torch.zeros(3, 8, dim).bfloat16()
    q[:, :, 3] = 1.0
    scale = bits * float(np.log(2)) / 32
    out, lse, step = _run(dm, c, q, 1, 2, dim, scale, 1)
    assert step.read_status() == 0
    ch.assert_gqa(out, lse, _ref(c, q, 1, scale), dim)
