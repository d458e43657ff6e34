"""Eviction on the GPU: accumulated weights against the float64 oracle, selection and
compaction exactly, and the run of them between two verify steps."""

import math

import numpy as np
import pytest
import torch

import oracle
from oracle import attention
from tests import _cache_helpers as ch
from tests import _helpers as h

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dm():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    import decode_context_mla_causal_gb300 as mod

    return mod


def _q(rows, heads, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(rows, heads, 576, generator=g) * scale).bfloat16()


def _lse(c, q, qlen, scale, causal=True):
    """The merged LSE of every row, as float32 numbers."""
    raw = ch.raw(c.pools[0])
    out = np.full(q.shape[:2], -np.inf)
    for b, L in enumerate(c.lens):
        if L <= 0:
            continue
        K = attention.gather_sequence(raw, c.table[b].numpy(), L, dcp=c.W, interleave=c.S, block_size=c.bs,
                                      kv_dtype=c.dtype, kv_scale=c.scale)
        for j in range(qlen):
            g = L - qlen + 1 + j if causal else L
            out[b * qlen + j] = attention.attend(ch.f64(q[b * qlen + j]), K, [g] * q.shape[1], scale)[1]
    return torch.tensor(out, dtype=torch.float32)


def _history(c, qlen, seed):
    """Weights of earlier steps; NaN where a token has none (the step's own, and behind them)."""
    g = torch.Generator().manual_seed(seed)
    w = torch.rand(c.W, c.B, c.ML, generator=g)
    for r in range(c.W):
        for b, L in enumerate(c.lens):
            w[r, b, oracle.evict.local_count(L - qlen, r, c.W, c.S):] = math.nan
    return w


def _weights_ref(c, q, qlen, scale, lse, decay, history, causal=True):
    return oracle.evict.key_weights(q=ch.f64(q), pools=ch.raw(c.pools[0]), block_table=c.table.numpy(),
                                    seq_lens=c.lens, qlen=qlen, kv_dtype=c.dtype, kv_scale=c.scale,
                                    softmax_scale=scale, lse=ch.f64(lse), decay=decay, history=ch.f64(history),
                                    causal=causal, **c.geometry)


CASES = [  # lens, qlen, heads, dcp, interleave, block, dtype, decay
    ([1], 1, 1, 1, 1, 1, "bf16", 1.0),
    ([200], 3, 8, 2, 1, 16, "bf16", 0.5),
    ([3, 2], 1, 16, 4, 1, 16, "fp8", 1.0),                # ranks without a token
    ([129, 128, 127, 5], 2, 24, 1, 1, 64, "fp8", 0.9),    # lengths around a tile, 48 rows
    ([700, 31], 5, 128, 2, 64, 64, "fp8", 0.98),          # 640 rows
    ([700, 31], 5, 128, 2, 64, 64, "bf16", 0.0),
    ([333, 64], 3, 96, 3, 6, 24, "fp8", 1.0),             # 288 rows, blocks of 24
    ([400], 1, 128, 1, 1, 96, "bf16", 1.0),
    ([90, 257], 2, 5, 2, 1, 5, "fp8", 1.0),               # blocks of five tokens, ten rows
    ([515, 3], 3, 7, 1, 1, 8, "bf16", 1.0),
    # more tiles than CTAs run at once: shares that end inside sequences, odd numbers of half tiles
    ([7 + 131 * i % 900 for i in range(90)], 2, 16, 3, 1, 16, "fp8", 0.9),
    ([7 + 277 * i % 1100 for i in range(70)], 5, 56, 5, 8, 8, "bf16", 1.0),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{c[1]}x{c[2]}-W{c[3]}-bs{c[5]}-{c[6]}")
def test_key_weights_against_the_oracle(dm, case):
    lens, qlen, H, W, S, bs, dtype, decay = case
    c = ch.Cache([max(n, qlen) for n in lens], dcp=W, interleave=S, block=bs, tails=[(576,)], dtype=dtype,
                 seed=sum(lens))
    scale = 1 / math.sqrt(192)
    q = _q(c.B * qlen, H, 5)
    lse = _lse(c, q, qlen, scale)
    hist = _history(c, qlen, 3)
    ev = dm.KvEviction(c.dims(dm, qlen, H), decay=decay)
    ev.workspace.fill_(0xFF)
    ev.weights.fill_(-3.0)
    args = (q.cuda(), c.pools[0].cuda(), c.kv_dtype(dm), c.dev_scale(), scale, lse.cuda(), c.lens_dev(), c.table.cuda())
    got = ev.accumulate(*args, history=hist.cuda()).cpu()
    assert ev.read_status() == 0
    ref, added, slack = _weights_ref(c, q, qlen, scale, lse, decay, hist)
    past = np.ones_like(ref, bool)                 # rows behind a sequence: left as they were
    for r in range(W):
        for b, L in enumerate(c.lens):
            past[r, b, :oracle.evict.local_count(L, r, W, S)] = False
    assert (got.numpy()[past] == -3.0).all()
    ref[past], got[torch.as_tensor(past)] = 0.0, 0.0
    ch.assert_key_weights(got, ref, added, slack, ch.f64(lse), decay)
    # in place: the same numbers, and the same bits again
    ev.weights.copy_(hist.cuda())
    ev.accumulate(*args)
    inplace = ev.weights.cpu()
    assert torch.equal(inplace[~torch.as_tensor(past)], got[~torch.as_tensor(past)])
    # one rank per call
    for r in range(W):
        one = dm.KvEviction(c.dims(dm, qlen, H), decay=decay, rank_begin=r, num_ranks=1)
        one.accumulate(args[0], args[1][r:r + 1].contiguous(), *args[2:], history=hist[r:r + 1].cuda().contiguous())
        mine = ~torch.as_tensor(past[r])
        assert torch.equal(one.weights[0].cpu()[mine], got[r][mine])


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
def test_key_weights_not_causal_and_rows_without_weight(dm, dtype):
    c = ch.Cache([0, 150, 2], dcp=2, interleave=1, block=16, tails=[(576,)], dtype=dtype, seed=6)
    q = _q(c.B * 3, 8, 5)
    lse = _lse(c, q, 3, 0.07, causal=False)
    lse[4, 2:5] = -math.inf                        # rows that attended nothing add nothing
    hist = torch.zeros(2, 3, c.ML)
    ev = dm.KvEviction(c.dims(dm, 3, 8, causal=False))
    got = ev.accumulate(q.cuda(), c.pools[0].cuda(), c.kv_dtype(dm), c.dev_scale(), 0.07, lse.cuda(), c.lens_dev(),
                        c.table.cuda(), history=hist.cuda())
    assert ev.read_status() == 0
    ref, added, slack = _weights_ref(c, q, 3, 0.07, lse, 1.0, hist, causal=False)
    ch.assert_key_weights(got, ref, added, slack, ch.f64(lse), 1.0)


def test_key_weights_of_queries_with_outliers(dm):
    # a row's largest element is thousands of times its others
    c = ch.Cache([300], dcp=1, interleave=1, block=64, tails=[(576,)], dtype="fp8", seed=6)
    q = _q(2, 8, 5, 0.5)
    q[:, :, 70] *= 3000.0
    q[1, 3] = 0.0
    lse = _lse(c, q, 2, 0.002)
    hist = torch.zeros(1, 1, c.ML)
    ev = dm.KvEviction(c.dims(dm, 2, 8))
    got = ev.accumulate(q.cuda(), c.pools[0].cuda(), dm.KV_FP8_E4M3, c.dev_scale(), 0.002, lse.cuda(), c.lens_dev(),
                        c.table.cuda(), history=hist.cuda())
    ref, added, slack = _weights_ref(c, q, 2, 0.002, lse, 1.0, hist)
    ch.assert_key_weights(got, ref, added, slack, ch.f64(lse), 1.0)


def test_key_weights_bad_inputs_set_status(dm):
    c = ch.Cache([120, 40, 60], dcp=2, interleave=1, block=16, tails=[(576,)], dtype="fp8", seed=8)
    q = _q(c.B * 2, 8, 5)
    lse = _lse(c, q, 2, 0.07)
    table = c.table.clone()
    table[0, 1], table[2, 0] = c.NB + 5, -1
    ev = dm.KvEviction(c.dims(dm, 2, 8))

    def run(lens, tab):
        ev.status.zero_()
        ev.weights.fill_(-3.0)
        hist = torch.zeros_like(ev.weights)
        ev.accumulate(q.cuda(), c.pools[0].cuda(), dm.KV_FP8_E4M3, c.dev_scale(), 0.07, lse.cuda(),
                      torch.tensor(lens, dtype=torch.int32, device="cuda"), tab.cuda(), history=hist)
        torch.cuda.synchronize()
        return ev.weights.cpu().numpy().copy(), ev.read_status()

    whole, st = run(c.lens, c.table)
    assert st == 0
    part, st = run(c.lens, table)
    assert st == dm.STATUS_BAD_BLOCK_ID
    lost = np.zeros_like(whole, bool)
    lost[:, 0, 16:32] = lost[:, 2, 0:16] = True
    assert (part[lost] == -3.0).all() and np.array_equal(part[~lost], whole[~lost])
    w, st = run([1, 40, 60], c.table)              # shorter than qlen
    assert st == dm.STATUS_BAD_SEQ_LEN and np.array_equal(w[:, 1:], whole[:, 1:])
    w, st = run([120, -5, 60], c.table)
    assert st == dm.STATUS_BAD_SEQ_LEN and (w[:, 1] == -3.0).all()
    _, st = run([120, 10 ** 6, 60], c.table)
    assert st & dm.STATUS_LOCAL_OVER_BOUND


SELECT = [  # lens, dcp, interleave, budget, sink, recent
    ([100], 1, 1, 30, 2, 5),
    ([1, 31, 32, 100, 4096], 2, 1, 32, 2, 3),
    ([1000, 64, 65], 4, 16, 130, 0, 0),
    ([5000, 20000], 3, 6, 4000, 0, 600),
    ([60000, 9, 33000], 1, 1, 20000, 7, 1),
    ([2000], 8, 8, 64, 0, 0),                      # the smallest budget: one span
    ([777], 2, 4, 700, 40, 260),                   # almost all protected
    ([150000], 1, 1, 149999, 0, 0),                # one goes
    ([150000], 1, 1, 1, 0, 0),                     # one stays
]


@pytest.mark.parametrize("kind", ["random", "ties", "zeros", "special"])
@pytest.mark.parametrize("case", SELECT, ids=lambda c: f"{len(c[0])}x{max(c[0])}-W{c[1]}S{c[2]}-to{c[3]}")
def test_select_is_exact(dm, case, kind):
    lens, W, S, budget, sink, recent = case
    rng = np.random.default_rng(budget)
    ML = max(oracle.evict.local_count(n, 0, W, S) for n in lens)
    w = rng.exponential(size=(W, len(lens), ML)).astype(np.float32)
    if kind == "ties":
        w = np.round(w * 3).astype(np.float32)
    elif kind == "zeros":
        w[:] = 0.0
        w[:, :, ::2] = -0.0
    elif kind == "special":
        w = rng.choice(np.float32([0.0, -0.0, 1.0, 1.0 + 2.0 ** -23, 1e-45, 3e38, math.inf, -math.inf, math.nan, -1.0]), w.shape)
    for r in range(W):                             # behind a sequence there may be anything
        for b, n in enumerate(lens):
            w[r, b, oracle.evict.local_count(n, r, W, S):] = math.inf
    dims = dm.make_dims(batch=len(lens), qlen=1, num_heads=1, dcp=W, interleave=S, block_size=max(S, 8) // S * S,
                        max_blocks_per_seq=ML, max_local_len=ML, num_blocks=4, num_splits=1)
    ev = dm.KvEviction(dims, budget, sink, recent)
    idx, count, new = ev.select(torch.tensor(lens, dtype=torch.int32, device="cuda"), torch.tensor(w, device="cuda"))
    assert ev.read_status() == 0
    kept, want = oracle.evict.select(weights=w, seq_lens=lens, budget=budget, sink=sink, recent=recent, dcp=W, interleave=S)
    idx, count = idx.cpu().numpy(), count.cpu().numpy()
    assert new.cpu().tolist() == want
    for r in range(W):
        for b in range(len(lens)):
            k = kept[r][b]
            assert count[r, b] == len(k) and idx[r, b, :len(k)].tolist() == k and (idx[r, b, len(k):] == -1).all()
    one = dm.KvEviction(dims, budget, sink, recent, rank_begin=W - 1, num_ranks=1)
    i1, c1, n1 = one.select(torch.tensor(lens, dtype=torch.int32, device="cuda"), torch.tensor(w[-1:], device="cuda"))
    assert np.array_equal(i1.cpu().numpy()[0], idx[-1]) and n1.cpu().tolist() == want


@pytest.mark.parametrize("ML", [450004, 450001])     # rows of weights on 16-byte boundaries, and not
def test_select_of_more_than_shared_memory_holds(dm, ML):
    n, budget = 450001, 200003
    rng = np.random.default_rng(ML)
    w = np.round(rng.exponential(size=(1, 2, ML)) * 1000).astype(np.float32)     # many ties
    dims = dm.make_dims(batch=2, qlen=1, num_heads=1, dcp=1, interleave=1, block_size=8, max_blocks_per_seq=ML,
                        max_local_len=ML, num_blocks=4, num_splits=1)
    ev = dm.KvEviction(dims, budget, 5, 1000)
    lens = [n, 420000]
    idx, count, new = ev.select(torch.tensor(lens, dtype=torch.int32, device="cuda"), torch.tensor(w, device="cuda"))
    kept, want = oracle.evict.select(weights=w, seq_lens=lens, budget=budget, sink=5, recent=1000, dcp=1, interleave=1)
    assert new.cpu().tolist() == want and count.cpu().tolist() == [want]
    idx = idx.cpu().numpy()
    for b in range(2):
        assert np.array_equal(idx[0, b, :len(kept[0][b])], kept[0][b]) and (idx[0, b, len(kept[0][b]):] == -1).all()


def test_select_bad_lengths_keep_nothing(dm):
    dims = dm.make_dims(batch=3, qlen=1, num_heads=1, dcp=2, interleave=1, block_size=8, max_blocks_per_seq=20,
                        max_local_len=100, num_blocks=4, num_splits=1)
    ev = dm.KvEviction(dims, 50)
    idx, count, new = ev.select(torch.tensor([-1, 60, 201], dtype=torch.int32, device="cuda"))
    assert ev.read_status() == dm.STATUS_BAD_SEQ_LEN | dm.STATUS_LOCAL_OVER_BOUND
    assert count.cpu().tolist() == [[0, 25, 0]] * 2 and new.cpu().tolist() == [0, 50, 0]
    assert bool((idx[:, [0, 2]] == -1).all())


@pytest.mark.parametrize("in_place", [True, False], ids=["in place", "to blocks"])
@pytest.mark.parametrize("lens,W,S,bs,tail,dtype,budget", [
    ([100], 1, 1, 16, (576,), "fp8", 30),
    ([700, 5, 333], 2, 4, 8, (576,), "bf16", 200),
    ([3000, 2900], 3, 1, 24, (2, 64), "bf16", 1000),
    ([1200, 40], 1, 1, 5, (16,), "fp8", 900),        # one 16-byte piece to a row
    ([2000], 2, 32, 32, (3, 64), "fp8", 1900),       # twelve pieces, nearly all stay
])
def test_compact_is_exact(dm, in_place, lens, W, S, bs, tail, dtype, budget):
    c = ch.Cache(lens, dcp=W, interleave=S, block=bs, tails=[tail], dtype=dtype, seed=budget, spare=1)
    g = torch.Generator().manual_seed(1)
    w = torch.rand(W, c.B, c.ML, generator=g)
    kept, want = oracle.evict.select(weights=w.numpy(), seq_lens=lens, budget=budget, sink=3, recent=4, dcp=W, interleave=S)
    ev = dm.KvEviction(c.dims(dm), budget, 3, 4)
    ev.weights.copy_(w)
    _, _, new = ev.select(c.lens_dev())
    assert new.cpu().tolist() == want
    pool, table = c.pools[0].cuda(), c.table.cuda()
    ev.compact(pool, table, None if in_place else c.other.cuda())
    torch.cuda.synchronize()
    assert ev.read_status() == 0
    ref = oracle.evict.compact(ch.raw(c.pools[0]), kept, c.table.numpy(), (c.table if in_place else c.other).numpy(), bs)
    assert np.array_equal(ch.raw(pool), ref)
    ww = w.clone()
    for r in range(W):
        for b in range(c.B):
            ww[r, b, :len(kept[r][b])] = w[r, b, torch.tensor(kept[r][b], dtype=torch.long)]
    assert torch.equal(ev.weights.cpu(), ww)


@pytest.mark.parametrize("in_place", [True, False])
def test_compact_skips_bad_entries(dm, in_place):
    c = ch.Cache([64, 64], dcp=1, interleave=1, block=16, tails=[(32,)], dtype="bf16", seed=1, spare=1)
    ev = dm.KvEviction(c.dims(dm), 32)
    idx = torch.arange(32, dtype=torch.int32).mul(2).expand(1, 2, 32).contiguous()
    idx[0, 0, 5], idx[0, 0, 9], idx[0, 0, 7] = 1 << 20, -7, 3   # outside, negative, before its place
    table = c.table.clone()
    table[1, 2] = c.NB                             # rows 32 .. 47 of the second sequence
    pool = c.pools[0].cuda()
    tab = table.cuda()
    ev.compact(pool, tab, None if in_place else c.other.cuda(), keep_idx=idx.cuda(),
               keep_count=torch.tensor([[32, 32]], dtype=torch.int32, device="cuda"), move_weights=False)
    torch.cuda.synchronize()
    assert ev.read_status() == dm.STATUS_BAD_PAGE | dm.STATUS_BAD_BLOCK_ID
    to = c.table if in_place else c.other
    want = c.pools[0].clone()
    for b in range(2):
        for i in range(32):
            if (b == 0 and i in (5, 7, 9)) or (b == 1 and 32 <= 2 * i < 48):
                continue
            want[0, to[b, i // 16], i % 16] = c.pools[0][0, c.table[b, 2 * i // 16], 2 * i % 16]
    assert np.array_equal(ch.raw(pool), ch.raw(want))
    before = pool.clone()
    ev.status.zero_()
    ev.compact(pool, tab, keep_idx=idx.cuda(), keep_count=torch.tensor([[33, -1]], dtype=torch.int32, device="cuda"),
               move_weights=False)
    assert ev.read_status() == dm.STATUS_BAD_PAGE and torch.equal(ch_bits(before), ch_bits(pool))


def ch_bits(t):
    return t.view(torch.int16)


def test_pool_shape_is_checked(dm):
    c = ch.Cache([64], dcp=1, interleave=1, block=16, tails=[(32,)], dtype="bf16", seed=1)
    ev = dm.KvEviction(c.dims(dm), 32)
    with pytest.raises(ValueError, match="pool must be"):
        ev.compact(c.pools[0].cuda().view(-1, 32), c.table.cuda())
    with pytest.raises(ValueError, match="no budget"):
        dm.KvEviction(c.dims(dm)).select(c.lens_dev())


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
def test_verify_accumulate_evict_verify(dm, dtype):
    # three verify steps, each adding its weights; eviction in place; a step on what is left
    W, S, bs, H, qlen, budget = 2, 4, 16, 16, 2, 160
    c = ch.Cache([300, 150, 290], dcp=W, interleave=S, block=bs, tails=[(576,)], dtype=dtype, seed=12, bound=160)
    scale = 1 / math.sqrt(192)
    dims = c.dims(dm, qlen, H, 2)
    step = dm.VerifyStep(dims, c.kv_dtype(dm))
    ev = dm.KvEviction(dims, budget, sink=2, recent=8, decay=0.9)
    pool, table, ks = c.pools[0].cuda(), c.table.cuda(), c.dev_scale()
    total, slack = np.zeros((W, c.B, c.ML)), 0.0
    final = list(c.lens)
    for n in range(3):                             # the last two steps' tokens are already in the pools
        c.lens = [x - 2 * (2 - n) for x in final]
        q = _q(c.B * qlen, H, 50 + n)
        _, lse = step(q.cuda(), pool, ks, scale, c.lens_dev(), table)
        ev.accumulate(q.cuda(), pool, c.kv_dtype(dm), ks, scale, lse, c.lens_dev(), table)
        total, added, loose = _weights_ref(c, q, qlen, scale, lse.cpu(), 0.9, torch.tensor(total))
        slack = 0.9 * slack + loose
    assert step.read_status() == ev.read_status() == 0
    ch.assert_key_weights(ev.weights, total, total, slack, ch.f64(lse), 0.9)
    kept, want = oracle.evict.select(weights=ev.weights.cpu().numpy(), seq_lens=c.lens, budget=budget, sink=2,
                                     recent=8, dcp=W, interleave=S)
    ev.select(c.lens_dev())
    ev.compact(pool, table)
    assert ev.new_lens.cpu().tolist() == want and max(want) <= budget
    q = _q(c.B * qlen, H, 60)
    out, lse = step(q.cuda(), pool, ks, scale, ev.new_lens, table)
    torch.cuda.synchronize()
    assert step.read_status() == ev.read_status() == 0
    raw = ch.raw(c.pools[0])
    for b in range(c.B):
        rows, pos = [], []
        for r in range(W):                         # the kept tokens by their old positions
            for t in kept[r][b]:
                rows.append(raw[r, c.table[b, t // bs], t % bs])
                pos.append(t // S * S * W + r * S + t % S)
        order = np.argsort(pos)
        K = attention.decode_pool_rows(np.array(rows)[order], dtype, c.scale)
        n = len(K)
        assert n == want[b]
        for j in range(qlen):
            o, l = attention.attend(ch.f64(q[b * qlen + j]), K, [n - qlen + 1 + j] * H, scale)
            h.assert_parity(ch.f64(out[b * qlen + j]), ch.f64(lse[b * qlen + j]), o, l, (b, j))


def test_evict_in_a_graph(dm):
    # the whole eviction captured once and replayed with other lengths and weights
    c = ch.Cache([500, 320], dcp=2, interleave=1, block=16, tails=[(2, 64), (2, 64)], dtype="bf16", seed=5)
    ev = dm.KvEviction(c.dims(dm), 200, 4, 16)
    lens, table = c.lens_dev(), c.table.cuda()
    fresh = [p.cuda() for p in c.pools]
    pools = [p.clone() for p in fresh]

    def evict():
        ev.select(lens)
        ev.compact(pools[0], table)
        ev.compact(pools[1], table, move_weights=False)

    evict()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        evict()
    for n, new in enumerate(([500, 320], [200, 7], [499, 201])):
        w = torch.rand(2, 2, c.ML, generator=torch.Generator().manual_seed(n))
        ev.weights.copy_(w)
        lens.copy_(torch.tensor(new, dtype=torch.int32))
        for p, f in zip(pools, fresh):
            p.copy_(f)
        g.replay()
        torch.cuda.synchronize()
        kept, want = oracle.evict.select(weights=w.numpy(), seq_lens=new, budget=200, sink=4, recent=16, dcp=2, interleave=1)
        assert ev.new_lens.cpu().tolist() == want
        for p, f in zip(pools, c.pools):
            assert np.array_equal(ch.raw(p), oracle.evict.compact(ch.raw(f), kept, c.table.numpy(), c.table.numpy(), 16))
    assert ev.read_status() == 0


def test_compact_into_a_copy_of_the_table_is_refused(dm):
    # the rows' own blocks, through another tensor: moving them side by side would race
    c = ch.Cache([64], dcp=1, interleave=1, block=16, tails=[(32,)], dtype="bf16", seed=1)
    ev = dm.KvEviction(c.dims(dm), 32)
    idx = torch.arange(32, dtype=torch.int32, device="cuda").mul(2).view(1, 1, 32).contiguous()
    pool, table = c.pools[0].cuda(), c.table.cuda()
    ev.compact(pool, table, table.clone(), keep_idx=idx, move_weights=False,
               keep_count=torch.tensor([[32]], dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    assert ev.read_status() == dm.STATUS_BAD_PAGE and np.array_equal(ch.raw(pool), ch.raw(c.pools[0]))


def test_key_weights_in_a_graph_on_two_objects(dm):
    # a captured and an eager object of the same shapes side by side, lengths changing
    c = ch.Cache([300, 170], dcp=2, interleave=1, block=16, tails=[(576,)], dtype="fp8", seed=5)
    q = _q(c.B * 3, 100, 5)                        # 300 rows: two row groups and their workspace
    dims = c.dims(dm, 3, 100)
    a, b = dm.KvEviction(dims, decay=0.5), dm.KvEviction(dims, decay=0.5)
    qd, kv, table, ks = q.cuda(), c.pools[0].cuda(), c.table.cuda(), c.dev_scale()
    lens = c.lens_dev()
    lse = torch.zeros(c.B * 3, 100, device="cuda")
    hist = torch.rand(2, 2, c.ML, device="cuda")
    args = (qd, kv, dm.KV_FP8_E4M3, ks, 0.07, lse, lens, table)
    a.accumulate(*args, history=hist)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        a.accumulate(*args, history=hist)
    side = torch.cuda.Stream()
    for new in ([300, 170], [3, 169], [129, 4]):
        c.lens = new
        lens.copy_(torch.tensor(new, dtype=torch.int32))
        lse.copy_(_lse(c, q, 3, 0.07))
        for ev in (a, b):
            ev.weights.fill_(-1.0)
        side.wait_stream(torch.cuda.current_stream())
        for _ in range(3):
            g.replay()
        with torch.cuda.stream(side):
            for _ in range(3):
                b.accumulate(*args, history=hist)
        torch.cuda.synchronize()
        ref, added, slack = _weights_ref(c, q, 3, 0.07, lse.cpu(), 0.5, hist.cpu())
        got = a.weights.cpu()
        live = torch.zeros_like(got, dtype=torch.bool)
        for r in range(2):
            for i, n in enumerate(new):
                live[r, i, :oracle.evict.local_count(n, r, 2, 1)] = True
        assert torch.equal(got, b.weights.cpu()) and bool((got[~live] == -1.0).all())
        ref[~live.numpy()], got[~live] = 0.0, 0.0
        ch.assert_key_weights(got, ref, added, slack, ch.f64(lse), 0.5, new)
    assert a.read_status() == b.read_status() == 0


def test_offsets_past_32_bits(dm):
    # pools of more than 4 GB whose last blocks are used
    for dtype, NB in (("fp8", 120000), ("bf16", 60000)):
        c = ch.Cache([400], dcp=1, interleave=1, block=64, tails=[(576,)], dtype=dtype, seed=2, scale=0.01)
        small, table = c.pools[0], c.table.clone()
        big = torch.empty((1, NB, 64, 576), dtype=small.dtype, device="cuda")
        assert big.numel() * big.element_size() > 1 << 32
        far = torch.tensor([[NB - 1 - 3 * i for i in range(table.shape[1])]], dtype=torch.int32)
        for i in range(table.shape[1]):
            big[0, int(far[0, i])] = small[0, int(table[0, i])].cuda()
        q = _q(2, 16, 5)
        lse = _lse(c, q, 2, 0.07)
        hist = _history(c, 2, 1)
        d = dm.make_dims(batch=1, qlen=2, num_heads=16, dcp=1, interleave=1, block_size=64, max_blocks_per_seq=c.MB,
                         max_local_len=c.ML, num_blocks=NB, num_splits=1)
        ev = dm.KvEviction(d, 200, 2, 3)
        ev.accumulate(q.cuda(), big, c.kv_dtype(dm), c.dev_scale(), 0.07, lse.cuda(), c.lens_dev(), far.cuda(),
                      history=hist.cuda())
        ref, added, slack = _weights_ref(c, q, 2, 0.07, lse, 1.0, hist)
        ch.assert_key_weights(ev.weights, ref, added, slack, ch.f64(lse), 1.0)
        w = ev.weights.cpu().numpy()
        kept, _ = oracle.evict.select(weights=w, seq_lens=[400], budget=200, sink=2, recent=3, dcp=1, interleave=1)
        ev.select(c.lens_dev())
        ev.compact(big, far.cuda())
        torch.cuda.synchronize()
        assert ev.read_status() == 0
        rows = torch.cat([small[0, int(b)] for b in table[0]])[torch.tensor(kept[0][0])]
        got = torch.cat([big[0, int(b)].cpu() for b in far[0]])[:len(kept[0][0])]
        assert np.array_equal(ch.raw(got), ch.raw(rows))
        del big


def test_grouped_head_cache_write_evict_decode(dm):
    # K and V rows of three steps written, the tokens cut by weight in both pools, attended
    W, S, bs, hkv, dim, H, budget = 2, 2, 8, 2, 64, 8, 90
    c = ch.Cache([150, 61], dcp=W, interleave=S, block=bs, tails=[(hkv, dim)] * 2, dtype="bf16", seed=4, bound=80)
    dims = c.dims(dm, 1, H)
    ev = dm.KvEviction(dims, budget, sink=1, recent=6)
    step = dm.GqaDecode(dims, hkv, dim, dm.KV_BF16)
    pools = [p.cuda() for p in c.pools]
    table = c.table.cuda()
    slots = torch.empty(W, c.B, dtype=torch.int32, device="cuda")
    g = torch.Generator().manual_seed(9)

    def grow():
        new = [torch.randn(c.B, hkv, dim, generator=g).bfloat16() for _ in range(2)]
        c.lens = [n + 1 for n in c.lens]
        dm.dcp_kv_slot_mapping(dims, c.lens_dev(), table, 0, W, slots, step.status)
        dm.dcp_gqa_kv_write(dims, hkv, dim, slots, new[0].cuda(), new[1].cuda(), dm.KV_BF16, None, None, W, *pools,
                            step.status)

    for _ in range(3):
        grow()
    ev.weights.copy_(torch.rand(W, c.B, c.ML, generator=g))
    kept, want = oracle.evict.select(weights=ev.weights.cpu().numpy(), seq_lens=c.lens, budget=budget, sink=1, recent=6,
                                     dcp=W, interleave=S)
    before = [p.cpu() for p in pools]
    ev.select(c.lens_dev())
    ev.compact(pools[0], table)
    ev.compact(pools[1], table, move_weights=False)
    torch.cuda.synchronize()
    assert ev.new_lens.cpu().tolist() == want
    for i in range(2):
        moved = oracle.evict.compact(ch.raw(before[i]), kept, c.table.numpy(), c.table.numpy(), bs)
        assert np.array_equal(ch.raw(pools[i]), moved)
    c.lens = want
    grow()                                         # the next token lands behind the kept ones
    c.pools = [p.cpu() for p in pools]
    q = torch.randn(c.B, H, dim, generator=g).bfloat16()
    out, lse = step(q.cuda(), *pools, None, None, 0.125, c.lens_dev(), table)
    torch.cuda.synchronize()
    assert step.read_status() == ev.read_status() == 0
    ref = oracle.gqa.decode(q=ch.f64(q), k_pools=ch.raw(c.pools[0]), v_pools=ch.raw(c.pools[1]),
                            block_table=c.table.numpy(), seq_lens=c.lens, qlen=1, kv_dtype="bf16", k_scale=1, v_scale=1,
                            softmax_scale=0.125, **c.geometry)
    ch.assert_gqa(out, lse, ref, dim)


def _near_float_scale():
    """A softmax scale whose product with log2(e) is nearly a float, and how far it is from one."""
    s = np.float32(0.6875) + np.arange(1 << 16, dtype=np.float32) * np.float32(2.0 ** -24)
    x = s.astype(np.float64) * math.log2(math.e)
    off = np.abs(x - x.astype(np.float32).astype(np.float64))
    i = int(off.argmin())
    return float(s[i]), float(off[i])


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
def test_key_weights_of_exact_scores(dm, dtype):
    # q.k is a whole number that every order of sums holds exactly, a power of two, and the LSE 0: a
    # weight is 2^(n * scale * log2 e). The product is exact, the exponential is off by 2^-22, the sum of
    # one weight and no history by 2^-24
    c = ch.Cache([600], dcp=2, interleave=1, block=16, tails=[(576,)], dtype=dtype, seed=3, scale=1.0)
    scale, off = _near_float_scale()
    rng = np.random.default_rng(4)
    n = rng.choice([-64, -32, -16, -1, 1, 16, 32, 64], 600)
    for p in range(600):
        x = np.zeros(576, np.float32)
        at = rng.permutation(576)
        x[at[:abs(n[p])]] = np.sign(n[p])
        x[at[64:264]], x[at[264:464]] = 2.0, -2.0
        k = torch.tensor(x).to(torch.float8_e4m3fn).view(torch.uint8) if dtype == "fp8" else torch.tensor(x).bfloat16()
        c.pools[0][p % 2, c.table[0, p // 2 // 16], p // 2 % 16] = k
    q = torch.ones(1, 1, 576).bfloat16()
    ev = dm.KvEviction(c.dims(dm, 1, 1))
    got = ev.accumulate(q.cuda(), c.pools[0].cuda(), c.kv_dtype(dm), c.dev_scale(), scale, torch.zeros(1, 1, device="cuda"),
                        c.lens_dev(), c.table.cuda(), history=torch.zeros_like(ev.weights)).cpu().double().numpy()
    assert ev.read_status() == 0
    want = np.exp(scale * n.astype(np.float64))
    have = np.array([got[p % 2, 0, p // 2] for p in range(600)])
    assert (np.abs(have / want - 1) <= 2.0 ** -22 + 2.0 ** -24 + 64 * math.log(2) * off).all(), np.abs(have / want - 1).max()


@pytest.mark.parametrize("in_place", [True, False])
def test_compact_leaves_the_weight_of_a_row_that_it_skips(dm, in_place):
    c = ch.Cache([64] * 4, dcp=1, interleave=1, block=16, tails=[(32,)], dtype="bf16", seed=1, spare=1)
    ev = dm.KvEviction(c.dims(dm), 32)
    idx = torch.arange(32, dtype=torch.int32).mul(2).expand(1, 4, 32).contiguous()
    idx[0, 0, 5], idx[0, 0, 9], idx[0, 0, 7] = 1 << 20, -7, 3   # outside, negative, before its place
    idx[0, :3, 11] = 63                            # out of order, and behind the last one
    idx[0, 2, 31] = -1
    src, dst = c.table.clone(), (c.table if in_place else c.other).clone()
    src[1, 2] = c.NB                               # the second sequence's rows 32 .. 47 cannot be read
    src[3, 3] = -1                                 # and the last one's rows 48 .. 63
    if in_place:
        dst = src
    else:
        dst[0, 1] = -1                             # the first one's rows 16 .. 31 cannot be written
        dst[3, 0] = src[3, 0]                      # a copy of the source's block
    w = torch.rand(1, 4, c.ML, generator=torch.Generator().manual_seed(1))
    ev.weights.copy_(w)
    tab = src.cuda()
    pool = c.pools[0].cuda()
    ev.compact(pool, tab, None if in_place else dst.cuda(), keep_idx=idx.cuda(),
               keep_count=torch.full((1, 4), 32, dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    assert ev.read_status() == dm.STATUS_BAD_PAGE | dm.STATUS_BAD_BLOCK_ID
    want, rows = w.clone(), c.pools[0].clone()
    for b in range(4):
        for i in range(32):
            t = int(idx[0, b, i])
            if not i <= t < 64 or not 0 <= int(src[b, t // 16]) < c.NB or not 0 <= int(dst[b, i // 16]) < c.NB:
                continue
            if not in_place and src[b, i // 16] == dst[b, i // 16]:
                continue
            want[0, b, i] = w[0, b, t]
            rows[0, dst[b, i // 16], i % 16] = c.pools[0][0, src[b, t // 16], t % 16]
    assert torch.equal(ev.weights.cpu(), want) and np.array_equal(ch.raw(pool), ch.raw(rows))


def test_select_where_no_rank_may_hold_a_token(dm):
    # a bound of zero: sequences of no token, and others that are over it
    dims = dm.make_dims(batch=3, qlen=1, num_heads=1, dcp=2, interleave=1, block_size=8, max_blocks_per_seq=1,
                        max_local_len=0, num_blocks=4, num_splits=1)
    ev = dm.KvEviction(dims, 50)
    ev.new_lens.fill_(-9)
    ev.keep_count.fill_(-9)
    idx, count, new = ev.select(torch.tensor([0, 60, 1], dtype=torch.int32, device="cuda"))
    assert ev.read_status() == dm.STATUS_LOCAL_OVER_BOUND
    assert idx.shape == (2, 3, 0) and count.cpu().tolist() == [[0, 0, 0]] * 2 and new.cpu().tolist() == [0, 0, 0]


def test_a_slot_that_takes_another_sequence(dm):
    # without a reset the longer prompt's tokens would start from the first sequence's weights
    first = ch.Cache([120, 90], dcp=2, interleave=1, block=16, tails=[(576,)], dtype="fp8", seed=8, bound=120)
    c = ch.Cache([200, 90], dcp=2, interleave=1, block=16, tails=[(576,)], dtype="fp8", seed=9, bound=120)
    q = _q(2, 8, 5)
    ev = dm.KvEviction(c.dims(dm, 1, 8), 100, 2, 4)
    side = torch.cuda.Stream()
    total = np.zeros((2, 2, 120))
    for n, cache in enumerate((first, c)):
        lse = _lse(cache, q, 1, 0.07)
        args = (q.cuda(), cache.pools[0].cuda(), dm.KV_FP8_E4M3, cache.dev_scale(), 0.07, lse.cuda(), cache.lens_dev(),
                cache.table.cuda())
        if n == 1:
            side.wait_stream(torch.cuda.current_stream())
            ev.reset(0, stream=side)
            torch.cuda.current_stream().wait_stream(side)
            total[:, 0] = 0.0
        ev.accumulate(*args)
        total, added, slack = _weights_ref(cache, q, 1, 0.07, lse, 1.0, torch.tensor(total))
        ch.assert_key_weights(ev.weights, total, added, slack, ch.f64(lse), 1.0, n)
    assert ev.read_status() == 0
    # captured with the step that follows it
    weights = ev.weights.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ev.reset([0])
        ev.accumulate(*args)
    ev.weights.copy_(torch.rand_like(weights))
    before = ev.weights.clone()
    g.replay()
    torch.cuda.synchronize()
    for r in range(2):
        assert torch.equal(ev.weights[r, 0, :100], weights[r, 0, :100]) and bool((ev.weights[r, 0, 100:] == 0).all())
        assert bool((ev.weights[r, 1, :45] > before[r, 1, :45]).any()) and torch.equal(ev.weights[r, 1, 45:], before[r, 1, 45:])


@pytest.mark.parametrize("in_place", [True, False], ids=["in place", "to blocks"])
@pytest.mark.parametrize("lens,W,S,bs,tail,dtype,budget", [
    ([21000], 1, 1, 16, (576,), "fp8", 19000),              # many rounds, lookups and rounds of weights
    ([9000, 20000], 2, 1, 64, (2, 64), "bf16", 9000),
    ([3000 + 7 * i for i in range(40)], 4, 2, 8, (576,), "fp8", 2000),  # 160 (rank, sequence) pairs: two slices of 18 pieces
    ([2500 + i for i in range(130)], 1, 1, 24, (4, 28), "bf16", 1500),  # 14 pieces: slices of 6, 6 and 2
    ([1700] * 30, 5, 1, 16, (5, 16), "bf16", 1300),                     # ten pieces: slices of 4, 4 and 2
])
def test_compact_in_many_rounds_is_exact(dm, in_place, lens, W, S, bs, tail, dtype, budget):
    c = ch.Cache(lens, dcp=W, interleave=S, block=bs, tails=[tail], dtype=dtype, seed=budget, spare=1)
    w = torch.rand(W, c.B, c.ML, generator=torch.Generator().manual_seed(1))
    kept, want = oracle.evict.select(weights=w.numpy(), seq_lens=lens, budget=budget, sink=3, recent=4, dcp=W, interleave=S)
    ev = dm.KvEviction(c.dims(dm), budget, 3, 4)
    ev.weights.copy_(w)
    _, _, new = ev.select(c.lens_dev())
    assert new.cpu().tolist() == want
    pool, table = c.pools[0].cuda(), c.table.cuda()
    ev.compact(pool, table, None if in_place else c.other.cuda())
    torch.cuda.synchronize()
    assert ev.read_status() == 0
    ref = oracle.evict.compact(ch.raw(c.pools[0]), kept, c.table.numpy(), (c.table if in_place else c.other).numpy(), bs)
    assert np.array_equal(ch.raw(pool), ref)
    ww = w.clone()
    for r in range(W):
        for b in range(c.B):
            ww[r, b, :len(kept[r][b])] = w[r, b, torch.tensor(kept[r][b], dtype=torch.long)]
    assert torch.equal(ev.weights.cpu(), ww)


def test_compact_of_many_long_sequences_to_blocks(dm):
    # so many sequences that a CTA takes more than 1024 rows of one: several lookups to a segment
    B, bs, n, keep = 1300, 16, 2400, 2300
    MB = n // bs
    g = torch.Generator(device="cuda").manual_seed(1)
    perm = torch.randperm(2 * B * MB, generator=g, device="cuda").to(torch.int32)
    src, dst = perm[:B * MB].view(B, MB).contiguous(), perm[B * MB:].view(B, MB).contiguous()
    pool = torch.randint(0, 1 << 30, (1, 2 * B * MB, bs, 4), generator=g, device="cuda", dtype=torch.int32)
    idx = torch.rand(1, B, n, generator=g, device="cuda").argsort(-1)[..., :keep].sort(-1).values
    w = torch.rand(1, B, n, generator=g, device="cuda")
    count = torch.randint(keep - 200, keep + 1, (1, B), generator=g, device="cuda").to(torch.int32)
    count[0, 0] = 0
    d = dm.make_dims(batch=B, qlen=1, num_heads=1, dcp=1, interleave=1, block_size=bs, max_blocks_per_seq=MB,
                     max_local_len=n, num_blocks=2 * B * MB, num_splits=1)
    ev = dm.KvEviction(d, keep)
    ev.weights.copy_(w)
    i = torch.arange(keep, device="cuda")
    live = i < count[0, :, None]
    at = src.long().gather(1, idx[0] // bs) * bs + idx[0] % bs
    to = dst.long()[:, i // bs] * bs + i % bs
    flat = pool.view(-1, 4)
    want, ww = flat.clone(), w.clone()
    want[to[live]] = flat[at[live]]
    ww[0, :, :keep][live] = w[0].gather(1, idx[0])[live]
    ev.compact(pool, src, dst, keep_idx=idx.to(torch.int32), keep_count=count)
    torch.cuda.synchronize()
    assert ev.read_status() == 0 and torch.equal(pool.view(-1, 4), want) and torch.equal(ev.weights, ww)


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
@pytest.mark.parametrize("heads", [64, 65, 96, 128, 129, 192, 193, 256])
def test_key_weights_of_every_width(dm, heads, dtype):
    # products of 64 to 256 columns, several tiles to a pair of CTAs, most of them of another sequence
    # than the last: every buffer of the accumulators is used again and again
    c = ch.Cache([12 + 37 * i % 70 for i in range(160)], dcp=6, interleave=1, block=8, tails=[(576,)], dtype=dtype,
                 seed=heads)
    scale = 1 / math.sqrt(192)
    q = _q(c.B, heads, 5)
    lse = _lse(c, q, 1, scale)
    hist = _history(c, 1, 3)
    ev = dm.KvEviction(c.dims(dm, 1, heads), decay=0.9)
    got = ev.accumulate(q.cuda(), c.pools[0].cuda(), c.kv_dtype(dm), c.dev_scale(), scale, lse.cuda(), c.lens_dev(),
                        c.table.cuda(), history=hist.cuda()).cpu()
    assert ev.read_status() == 0
    ref, added, slack = _weights_ref(c, q, 1, scale, lse, 0.9, hist)
    for r in range(6):
        for b, n in enumerate(c.lens):
            k = oracle.evict.local_count(n, r, 6, 1)
            ref[r, b, k:], got[r, b, k:] = 0.0, 0.0
    ch.assert_key_weights(got, ref, added, slack, ch.f64(lse), 0.9)
    again = ev.accumulate(q.cuda(), c.pools[0].cuda(), c.kv_dtype(dm), c.dev_scale(), scale, lse.cuda(), c.lens_dev(),
                          c.table.cuda(), history=hist.cuda()).cpu()
    live = ref != 0.0
    assert np.array_equal(again.numpy()[live], got.numpy()[live])
