"""4-bit grouped-head pools on the GPU: rows in bit for bit, rows out, and the attention over them
against the float64 oracle; and a prompt's whole way into them."""

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


class Cache4:
    """Shuffled 4-bit K and V pools. Rows that hold no token of a sequence have block scales of NaN."""

    def __init__(self, lens, *, heads, dim, dcp, interleave, block, seed, scale=0.002, bound=None):
        self.lens, self.W, self.S, self.bs = list(lens), dcp, interleave, block
        self.B, self.K, self.D, self.scale = len(self.lens), heads, dim, scale
        longest = max(oracle.evict.local_count(n, 0, dcp, interleave) for n in self.lens)
        self.ML = max(1, longest if bound is None else bound)
        self.MB = -(-self.ML // block)
        self.NB = self.B * self.MB + 3
        g = torch.Generator().manual_seed(seed)
        self.table = torch.randperm(self.NB, generator=g).to(torch.int32)[: self.B * self.MB].view(self.B, -1).contiguous()
        n = heads * dim
        self.pools, self.values = [], []
        for factor in (1.0, 1.5):
            x = torch.randn(dcp, self.NB, block, n, generator=g).bfloat16()
            rows = oracle.fp4.quantize_rows(ch.raw(x), scale * factor)
            full = np.full_like(rows, 0x7F)
            for b, length in enumerate(self.lens):
                p = np.arange(max(length, 0))
                r, li = oracle.metadata.owner(p, dcp, interleave), oracle.metadata.local_index(p, dcp, interleave)
                ok = li < self.ML
                at = (r[ok], self.table[b].numpy()[li[ok] // block], li[ok] % block)
                full[at] = rows[at]
            self.pools.append(torch.from_numpy(full))
            self.values.append(oracle.fp4.decode_rows(full, n).reshape(dcp, self.NB, block, heads, dim))

    def dims(self, dm, qlen=1, heads=8, causal=True):
        return dm.make_dims(batch=self.B, qlen=qlen, num_heads=heads, dcp=self.W, interleave=self.S, block_size=self.bs,
                            max_blocks_per_seq=self.MB, max_local_len=self.ML, num_blocks=self.NB, num_splits=1,
                            causal=causal)

    def scales(self):
        return (torch.tensor([self.scale], device="cuda"), torch.tensor([self.scale * 1.5], device="cuda"))

    def ref(self, q, qlen, scale, causal=True, **kw):
        f = np.float32
        return oracle.gqa.decode(q=ch.f64(q), k_pools=self.values[0], v_pools=self.values[1], block_table=self.table.numpy(),
                                 seq_lens=self.lens, qlen=qlen, kv_dtype="values", k_scale=f(self.scale),
                                 v_scale=f(self.scale * 1.5), softmax_scale=scale, causal=causal, dcp=self.W,
                                 interleave=self.S, block_size=self.bs, **kw)


def _run(dm, c, q, qlen, scale, causal=True, rank_begin=0, num_ranks=None):
    step = dm.GqaDecode(c.dims(dm, qlen, q.shape[1], causal), c.K, c.D, dm.KV_NVFP4, rank_begin=rank_begin,
                        num_ranks=num_ranks)
    of = slice(rank_begin, rank_begin + step.num_ranks)
    step.out.fill_(float("nan"))
    step.lse.fill_(float("nan"))
    step.workspace.fill_(0xFF)
    lens = torch.tensor(c.lens, dtype=torch.int32, device="cuda")
    out, lse = step(q.cuda(), c.pools[0][of].cuda().contiguous(), c.pools[1][of].cuda().contiguous(), *c.scales(), scale,
                    lens, c.table.cuda())
    torch.cuda.synchronize()
    return out, lse, step


def _q(rows, heads, dim, seed=7):
    return torch.randn(rows, heads, dim, generator=torch.Generator().manual_seed(seed)).bfloat16()


CASES = [  # lens, qlen, heads, kv_heads, dim, dcp, interleave, block
    ([1], 1, 1, 1, 64, 1, 1, 1),
    ([1, 2, 3], 1, 8, 8, 128, 4, 1, 16),
    ([200], 1, 32, 8, 128, 2, 1, 16),
    ([65, 64, 63, 1], 1, 10, 2, 64, 1, 8, 8),
    ([700, 31], 2, 40, 8, 128, 3, 6, 24),        # twenty rows to a K/V head: a team of two warps
    ([513, 1030, 4], 4, 64, 4, 128, 2, 64, 64),  # 64 rows: a team of four
    ([300, 129], 3, 16, 1, 64, 8, 1, 96),
    ([1000], 1, 17, 1, 128, 1, 1, 128),
    ([2500, 9, 1777], 1, 16, 16, 64, 2, 1, 5),
    ([90], 7, 6, 2, 128, 1, 3, 3),
    ([3000, 2900, 40, 700], 1, 8, 1, 128, 1, 1, 64),  # shares that cut sequences
    ([5000, 100], 8, 12, 3, 64, 2, 16, 32),
    ([77, 64, 9], 4, 4, 2, 128, 2, 1, 16),            # eight rows of four boundaries: one set
    ([130, 3], 3, 5, 5, 64, 1, 4, 8),                 # three rows
    ([4000, 17, 0], 2, 16, 4, 128, 4, 8, 32),         # eight rows, shares that cut a sequence
    ([999, 250], 3, 10, 2, 64, 2, 2, 16),             # fifteen rows: two sets
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{c[1]}x{c[2]}:{c[3]}x{c[4]}-W{c[5]}-bs{c[7]}")
def test_decode4_against_the_oracle(dm, case):
    lens, qlen, H, hkv, dim, W, S, bs = case
    c = Cache4([max(n, qlen) for n in lens], heads=hkv, dim=dim, dcp=W, interleave=S, block=bs, seed=sum(lens) + H)
    q = _q(c.B * qlen, H, dim)
    out, lse, step = _run(dm, c, q, qlen, dim ** -0.5)
    assert step.read_status() == 0
    ch.assert_gqa(out, lse, c.ref(q, qlen, dim ** -0.5), dim)
    again = _run(dm, c, q, qlen, dim ** -0.5)
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])


def test_decode4_not_causal_and_empty_sequences(dm):
    c = Cache4([0, 37, 0, 2], heads=2, dim=64, dcp=2, interleave=1, block=16, seed=3)
    q = _q(c.B * 3, 8, 64)
    out, lse, step = _run(dm, c, q, 3, 0.2, causal=False)
    assert step.read_status() == 0
    ch.assert_gqa(out, lse, c.ref(q, 3, 0.2, causal=False), 64)


def test_decode4_one_rank_per_call(dm):
    c = Cache4([150, 3], heads=2, dim=128, dcp=4, interleave=4, block=8, seed=9)
    q = _q(c.B, 6, 128)
    for r in range(4):
        out, lse, step = _run(dm, c, q, 1, 0.1, rank_begin=r, num_ranks=1)
        assert step.read_status() == 0
        ch.assert_gqa(out, lse, c.ref(q, 1, 0.1, ranks=[r]), 128, r)


def test_decode4_small_and_large_block_scales(dm):
    # block scales from the least to the largest E4M3 value: products with codes are exact
    c = Cache4([300], heads=1, dim=64, dcp=1, interleave=1, block=16, seed=5, scale=1.0)
    g = np.random.default_rng(1)
    for pool, values in zip(c.pools, range(2)):
        rows = pool.numpy()
        rows[..., 32:36] = g.integers(0, 0x7F, rows[..., 32:36].shape)
        if values == 0:
            rows[..., 32:36] = g.integers(0, 0x30, rows[..., 32:36].shape)  # scores stay finite
        c.values[values] = oracle.fp4.decode_rows(rows, 64).reshape(c.values[values].shape)
    q = _q(1, 4, 64)
    out, lse, step = _run(dm, c, q, 1, 0.125)
    ch.assert_gqa(out, lse, c.ref(q, 1, 0.125), 64)


@pytest.mark.parametrize("heads,kv,dim", [(4, 2, 128), (2, 1, 64), (10, 2, 128), (40, 2, 64)])
def test_decode4_rows_do_not_meet_newer_tokens(dm, heads, kv, dim):
    # the newest token's scales are NaN: only the newest row is
    lens, qlen = [70, 33], 3
    c = Cache4(lens, heads=kv, dim=dim, dcp=2, interleave=1, block=16, seed=6)
    q = _q(len(lens) * qlen, heads, dim)
    out, lse, _ = _run(dm, c, q, qlen, 0.1)
    keep = out.clone(), lse.clone()
    n = kv * dim
    for b, length in enumerate(lens):
        p = length - 1
        r, li = p % 2, p // 2
        for pool in c.pools:
            pool[r, int(c.table[b, li // 16]), li % 16, n // 2:n // 2 + n // 16] = 0x7F
    out, lse, step = _run(dm, c, q, qlen, 0.1)
    assert step.read_status() == 0
    for b in range(len(lens)):
        old, new = slice(b * qlen, b * qlen + qlen - 1), b * qlen + qlen - 1
        assert torch.equal(out[old], keep[0][old]) and torch.equal(lse[old], keep[1][old])
        assert bool(torch.isnan(out[new]).all()) and bool(torch.isnan(lse[new]).all())


def test_decode4_bad_blocks(dm):
    c = Cache4([120, 40, 60], heads=2, dim=64, dcp=2, interleave=1, block=16, seed=8)
    q = _q(c.B * 2, 4, 64)
    good = c.table.clone()
    c.table[0, 1], c.table[2, 0] = c.NB + 5, -1
    out, lse, step = _run(dm, c, q, 2, 0.2)
    assert step.read_status() == dm.STATUS_BAD_BLOCK_ID
    bad, c.table = c.table, good
    ch.assert_gqa(out, lse, c.ref(q, 2, 0.2, skip=lambda b, li: not 0 <= int(bad[b, li // 16]) < c.NB), 64)


# ------------------------------------------------------------------ rows in and out


@pytest.mark.parametrize("heads,dim,dcp,inter,block,qlen", [
    (1, 64, 1, 1, 1, 1), (1, 128, 2, 1, 16, 5), (8, 128, 4, 16, 32, 40), (3, 64, 3, 2, 24, 7), (5, 128, 8, 1, 5, 33)])
def test_write4_bit_for_bit_and_back(dm, heads, dim, dcp, inter, block, qlen):
    lens = [qlen + 90, qlen, qlen + 11]
    c = Cache4(lens, heads=heads, dim=dim, dcp=dcp, interleave=inter, block=block, seed=qlen)
    n = heads * dim
    g = torch.Generator().manual_seed(1)
    new = [torch.randn(3 * qlen, n, generator=g).bfloat16() * 2.0 ** torch.randint(-14, 4, (3 * qlen, n // 16), generator=g)
           .repeat_interleave(16, 1) for _ in range(2)]
    new = [x.bfloat16() for x in new]
    new[0][0, :16] = 0.0           # a block of zeros
    new[0][0, 16:32] = 2.0 ** -130  # and one too small for any scale
    new[1][-1, :16] = 3.0e38       # one that saturates
    dims = c.dims(dm, qlen)
    lens_d, table = torch.tensor(lens, dtype=torch.int32, device="cuda"), c.table.cuda()
    slots = torch.empty(dcp, 3 * qlen, dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    dm.dcp_kv_slot_mapping(dims, lens_d, table, 0, dcp, slots, status)
    k, v = (x.cuda() for x in c.pools)
    dm.dcp_gqa_kv_write(dims, heads, dim, slots, new[0].cuda(), new[1].cuda(), dm.KV_NVFP4, *c.scales(), dcp, k, v, status)
    assert int(status) == 0
    begins = (lens_d - qlen).contiguous()
    cu = torch.arange(4, dtype=torch.int32, device="cuda") * qlen
    outs = [torch.full((3 * qlen + 2, heads, dim), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    dm.dcp_gqa_kv_gather(dims, heads, dim, begins, cu, table, k, v, dm.KV_NVFP4, *c.scales(), 0, dcp, *outs, status)
    assert int(status) == 0
    for pool, got, x, factor, back in ((c.pools[0], k, new[0], 1.0, outs[0]), (c.pools[1], v, new[1], 1.5, outs[1])):
        rows = oracle.fp4.quantize_rows(ch.raw(x), c.scale * factor)
        want = pool.numpy().reshape(dcp, -1, rows.shape[-1]).copy()
        s = slots.cpu().numpy()
        used = n // 2 + n // 16
        for r in range(dcp):
            at = s[r] >= 0
            want[r, s[r][at], :used] = rows[at, :used]
        assert np.array_equal(got.cpu().numpy().reshape(want.shape), want)
        values = (oracle.fp4.decode_rows(rows, n).astype(np.float32) * np.float32(c.scale * factor))
        exp = torch.from_numpy(values).bfloat16().view(3 * qlen, heads, dim)
        assert torch.equal(back[:-2].cpu(), exp) and bool((back[-2:] == 7).all())


@pytest.mark.parametrize("scale", [0.002, 1.0 / 3.0, 1e-37, 3e37, 7.77e-9])
def test_write4_many_values(dm, scale):
    # every rounding of the quotient counts: values of all exponents around the scale's, and bf16's
    # smallest and largest
    rows, n = 512, 8 * 128
    g = torch.Generator().manual_seed(4)
    x = torch.randn(2 * rows, n, generator=g).double()
    x *= 2.0 ** torch.randint(-8, 9, (2 * rows, n // 16), generator=g).repeat_interleave(16, 1).double() * scale * 200
    x = x.clamp(-3e38, 3e38).float().bfloat16()
    x[0, :16] = 1e-40
    x[1, :16] = 3.3e38
    x[2, :16] = -0.0
    x[3, ::2] = 0.0
    dims = dm.make_dims(batch=rows, qlen=1, num_heads=1, dcp=1, interleave=1, block_size=16, max_blocks_per_seq=1,
                        max_local_len=16, num_blocks=rows // 16, num_splits=1)
    slots = torch.randperm(rows, generator=g).to(torch.int32).view(1, rows).cuda()
    width = dm.dcp_gqa_row_bytes(8, 128, dm.KV_NVFP4)
    k, v = (torch.zeros(1, rows // 16, 16, width, dtype=torch.uint8, device="cuda") for _ in range(2))
    s = torch.tensor([scale], device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    dm.dcp_gqa_kv_write(dims, 8, 128, slots, x[:rows].cuda(), x[rows:].cuda(), dm.KV_NVFP4, s, s, 1, k, v, status)
    with np.errstate(over="ignore"):
        want = oracle.fp4.quantize_rows(ch.raw(x), np.float32(scale))
    for pool, w in ((k, want[:rows]), (v, want[rows:])):
        assert np.array_equal(pool.view(rows, width)[slots[0].long()].cpu().numpy(), w)


def test_gather_many_sequences(dm):
    # more sequences than a warp looks at at once, most of them short or empty
    lens = [(i * 13) % 7 for i in range(1300)] + [40]
    c = Cache4(lens, heads=1, dim=64, dcp=2, interleave=1, block=4, seed=3)
    cu = torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int32, device="cuda")
    n = int(cu[-1])
    outs = [torch.empty(n, 1, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    dm.dcp_gqa_kv_gather(c.dims(dm), 1, 64, None, cu, c.table.cuda(), *(p.cuda() for p in c.pools), dm.KV_NVFP4,
                         *c.scales(), 0, 2, *outs, status)
    assert int(status) == 0
    for value, s, out in zip(c.values, c.scales(), outs):
        rows = np.concatenate([oracle.gqa.token_rows(value, c.table[b].numpy(), np.arange(m), dcp=2, interleave=1,
                                                     block_size=4)[0] for b, m in enumerate(lens)])
        want = rows.astype(np.float32) * np.float32(s.item())
        assert torch.equal(out.cpu(), torch.from_numpy(want).bfloat16().view(n, 1, 64))


@pytest.mark.parametrize("kind", ["bf16", "fp8", "fp4"])
def test_gather_a_context(dm, kind):
    # whole contexts, one rank at a time: each rank fills in its own rows
    lens = [70, 0, 33]
    if kind == "fp4":
        c = Cache4(lens, heads=2, dim=64, dcp=3, interleave=2, block=4, seed=3)
        pools, scales, kv = c.pools, c.scales(), dm.KV_NVFP4
        values = [(x.astype(np.float32) * np.float32(s.item())) for x, s in zip(c.values, scales)]
    else:
        c = ch.Cache(lens, dcp=3, interleave=2, block=4, tails=[(2, 64)] * 2, dtype=kind, seed=3)
        pools, kv = c.pools, c.kv_dtype(dm)
        scales = (c.dev_scale(), c.dev_scale(1.5))
        values = [oracle.gqa.decode_values(ch.raw(x), kind, 1.0 if s is None else np.float32(s.item())).astype(np.float32)
                  for x, s in zip(pools, scales)]
    dims = c.dims(dm)
    cu = torch.tensor([2, 72, 72, 105], dtype=torch.int32, device="cuda")
    outs = [torch.full((107, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for r in range(3):
        dm.dcp_gqa_kv_gather(dims, 2, 64, None, cu, c.table.cuda(), pools[0][r:r + 1].cuda().contiguous(),
                             pools[1][r:r + 1].cuda().contiguous(), kv, *scales, r, 1, *outs, status)
    assert int(status) == 0
    for value, out in zip(values, outs):
        for b, (first, n) in enumerate(((2, 70), (72, 0), (72, 33))):
            rows, _, _ = oracle.gqa.token_rows(value, c.table[b].numpy(), np.arange(n), dcp=3, interleave=2, block_size=4)
            assert torch.equal(out[first:first + n].cpu(), torch.from_numpy(rows.astype(np.float32)).bfloat16().view(n, 2, 64))
        assert bool((out[:2] == 7).all()) and bool((out[105:] == 7).all())
    # bad blocks, positions beyond the table, offsets below zero: those rows stay
    bad = c.table.clone()
    bad[0, 0] = c.NB
    begins = torch.tensor([0, 0, -4], dtype=torch.int32, device="cuda")
    outs[0].fill_(7.0)
    dm.dcp_gqa_kv_gather(dims, 2, 64, begins, torch.tensor([0, 3, 3, 6], dtype=torch.int32, device="cuda"), bad.cuda(),
                         pools[0].cuda(), pools[1].cuda(), kv, *scales, 0, 3, *outs, status)
    assert int(status) == dm.STATUS_BAD_BLOCK_ID | dm.STATUS_BAD_SEQ_LEN and bool((outs[0] == 7).all())
    status.zero_()
    begins = torch.tensor([c.MB * 4 * 3, 0, 0], dtype=torch.int32, device="cuda")
    dm.dcp_gqa_kv_gather(dims, 2, 64, begins, torch.tensor([0, 3, 3, 3], dtype=torch.int32, device="cuda"), bad.cuda(),
                         pools[0].cuda(), pools[1].cuda(), kv, *scales, 0, 3, *outs, status)
    assert int(status) == dm.STATUS_LOCAL_OVER_BOUND and bool((outs[0] == 7).all())


def test_write4_bad_slots_set_status(dm):
    c = Cache4([8], heads=1, dim=64, dcp=1, interleave=1, block=8, seed=1)
    dims = c.dims(dm, 4)
    k, v = (x.cuda() for x in c.pools)
    before = k.clone()
    slots = torch.tensor([[-2, c.NB * 8, -1, 1 << 30]], dtype=torch.int32, device="cuda")
    x = torch.ones(4, 1, 64, dtype=torch.bfloat16, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    dm.dcp_gqa_kv_write(dims, 1, 64, slots, x, x, dm.KV_NVFP4, *c.scales(), 1, k, v, status)
    assert int(status) == dm.STATUS_BAD_PAGE and torch.equal(k, before)


# ------------------------------------------------------------------ a run of them together


def test_prompts_into_the_cache_and_on(dm):
    """Two steps of a server: prompts are planned, rotated, attended and written in 4 bits; then a
    chunk with its context read back beside a new prompt; then single tokens over the cache."""
    W, S, bs, K, H, D, B, rows = 2, 1, 16, 2, 8, 128, 3, 220
    scale, c_scale = D ** -0.5, 0.002
    bound, NB = 200, 64
    g = torch.Generator().manual_seed(0)
    pages = dm.make_dims(batch=B, qlen=1, num_heads=H, dcp=W, interleave=S, block_size=bs, max_blocks_per_seq=16,
                         max_local_len=bound, num_blocks=NB, num_splits=1)
    packed = dm.make_dims(batch=rows, qlen=1, num_heads=1, dcp=W, interleave=S, block_size=bs, max_blocks_per_seq=16,
                          max_local_len=bound, num_blocks=NB, num_splits=1)
    plan, rope = dm.PagePlan(pages, rows), dm.Rope(D, base=10000.0)
    attend = dm.PromptAttention(H, K, D, D, max_rows=rows, max_seqs=B)
    decode = dm.GqaDecode(pages, K, D, dm.KV_NVFP4)
    freq, amp = oracle.prompt.frequencies(D, 10000.0)
    i32 = dict(dtype=torch.int32, device="cuda")
    lens, table = torch.zeros(B, **i32), torch.full((B, 16), -1, **i32)
    free, count = torch.randperm(NB, generator=g).to(torch.int32).cuda(), torch.tensor([NB], **i32)
    width = dm.dcp_gqa_row_bytes(K, D, dm.KV_NVFP4)
    pools = [torch.full((W, NB, bs, width), 0x7F, dtype=torch.uint8, device="cuda") for _ in range(2)]
    scales = [torch.tensor([c_scale], device="cuda") for _ in range(2)]
    status = torch.zeros(1, **i32)
    held = [[np.zeros((0, K, D)), np.zeros((0, K, D))] for _ in range(B)]  # what the pools stand for
    for targets in ([70, 0, 130], [99, 60, 131]):
        old = lens.tolist()
        q, k, v = (torch.randn(rows, n, D, generator=g).bfloat16() for n in (H, K, K))
        slots, positions, cu = plan(torch.tensor(targets, **i32), lens, table, free, count)
        assert lens.tolist() == targets and plan.read_status() == 0
        qd, kd = rope(positions, q.cuda(), k.cuda())
        dm.dcp_gqa_kv_write(packed, K, D, slots, kd, v.cuda(), dm.KV_NVFP4, *scales, W, *pools, status)
        # keys of every sequence as the cache holds them, context and new rows
        cu_k = torch.zeros(B + 1, **i32)
        cu_k[1:] = lens.cumsum(0)
        keys = [torch.empty(sum(targets), K, D, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        dm.dcp_gqa_kv_gather(pages, K, D, None, cu_k, table, *pools, dm.KV_NVFP4, *scales, 0, W, *keys, status)
        out, lse = attend(qd, *keys, cu, cu_k, scale)
        assert int(status) == 0 and attend.read_status() == 0
        cu_h, ck_h = cu.tolist(), cu_k.tolist()
        pos = np.concatenate([np.arange(a, t) for a, t in zip(old, targets)])
        assert positions[: len(pos)].tolist() == pos.tolist()
        for b in range(B):
            of = slice(cu_h[b], cu_h[b + 1])
            for i, x in enumerate((kd, v)):
                rowsq = oracle.fp4.quantize_rows(ch.raw(x[of].reshape(-1, K * D)), c_scale)
                val = oracle.fp4.decode_rows(rowsq, K * D).astype(np.float32) * np.float32(c_scale)
                held[b][i] = np.concatenate([held[b][i], val.reshape(-1, K, D)])
        # the rotation, against float64
        ref_k = oracle.prompt.rotate(ch.f64(k[: len(pos)]), pos, freq, amp, False)
        assert (np.abs(ch.f64(kd[: len(pos)]) - ref_k) <= 2.0 ** -8 * np.abs(ref_k) + 2.0 ** -16).all()
        want = [torch.from_numpy(np.concatenate([held[b][i] for b in range(B)])).bfloat16() for i in range(2)]
        assert all(torch.equal(a.cpu(), w) for a, w in zip(keys, want))
        ref = oracle.prompt.attend(q=ch.f64(qd), k=ch.f64(keys[0]), v=ch.f64(keys[1]), cu_q=cu_h, cu_k=ck_h,
                                   softmax_scale=scale)
        n = cu_h[-1]
        ch.assert_gqa(out[:n], lse[:n], {a: x[:n] for a, x in ref.items()}, D)
    q = _q(B, H, D, 3)
    out, lse = decode(q.cuda(), *pools, *scales, scale, lens, table)
    assert decode.read_status() == 0
    for b in range(B):
        ref = oracle.prompt.attend(q=ch.f64(q[b:b + 1]), k=held[b][0], v=held[b][1], cu_q=[0, 1],
                                   cu_k=[0, len(held[b][0])], softmax_scale=scale)
        ch.assert_gqa(out[b:b + 1], lse[b:b + 1], ref, D)


@pytest.mark.parametrize("heads,dim", [(1, 64), (8, 128)])
def test_write4_infinities_and_nan_read_as_nan(dm, heads, dim):
    # values that have no code: their blocks read as NaN, whatever else is in them; the others of the row
    # and the other rows as with finite values; and the decode's rows that see them are not finite
    n, lens = heads * dim, [20, 20, 20]
    c = Cache4(lens, heads=heads, dim=dim, dcp=2, interleave=1, block=16, seed=2)
    g = torch.Generator().manual_seed(5)
    k, v = (torch.randn(3, n, generator=g).bfloat16() for _ in range(2))
    k[0, 3], k[0, n - 1], v[1, 16], v[1, 40], v[1, 41] = math.nan, -math.inf, math.inf, -math.nan, 3.0e38
    dims = c.dims(dm, 1, heads)
    lens_d, table = torch.tensor(lens, dtype=torch.int32, device="cuda"), c.table.cuda()
    slots = torch.empty(2, 3, dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    dm.dcp_kv_slot_mapping(dims, lens_d, table, 0, 2, slots, status)
    pools = [x.cuda() for x in c.pools]
    dm.dcp_gqa_kv_write(dims, heads, dim, slots, k.cuda(), v.cuda(), dm.KV_NVFP4, *c.scales(), 2, *pools, status)
    outs = [torch.empty(3, heads, dim, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    cu = torch.arange(4, dtype=torch.int32, device="cuda")
    dm.dcp_gqa_kv_gather(dims, heads, dim, lens_d - 1, cu, table, *pools, dm.KV_NVFP4, *c.scales(), 0, 2, *outs, status)
    assert int(status) == 0
    width = oracle.fp4.row_bytes(n)
    for pool, x, factor, back in ((pools[0], k, 1.0, outs[0]), (pools[1], v, 1.5, outs[1])):
        rows = oracle.fp4.quantize_rows(ch.raw(x), c.scale * factor)
        flat = pool.cpu().numpy().reshape(2, -1, width)
        s = slots.cpu().numpy()
        for i in range(3):
            r = int(np.argmax(s[:, i]))
            assert np.array_equal(flat[r, s[r, i], : n // 2 + n // 16], rows[i, : n // 2 + n // 16])
        want = oracle.fp4.decode_rows(rows, n).astype(np.float32) * np.float32(c.scale * factor)
        bad = ~np.isfinite(ch.f64(x)).reshape(3, -1, 16).all(-1).repeat(16, axis=-1)
        got = back.cpu().view(3, n)
        assert np.array_equal(np.isnan(want), bad) and bool((torch.isnan(got) == torch.from_numpy(bad)).all())
        assert torch.equal(got[~bad], torch.from_numpy(want).bfloat16()[~bad])
    step = dm.GqaDecode(dims, heads, dim, dm.KV_NVFP4)
    q = _q(3, heads, dim)
    out, lse = step(q.cuda(), *pools, *c.scales(), 0.1, lens_d, table)
    assert step.read_status() == 0
    hit = torch.zeros(3, heads, dtype=torch.bool)
    hit[0, 0] = hit[0, heads - 1] = True                # keys of the first and the last head
    assert bool((torch.isnan(lse).cpu() == hit).all()) and bool(torch.isnan(out[0, 0]).all())
    assert bool((torch.isnan(out[1].flatten()).cpu() == torch.isnan(outs[1][1].flatten()).cpu()).all())
    assert bool(torch.isfinite(out[2]).all())


@pytest.mark.parametrize("heads,dim", [(0, 64), (-2, 64), (2, 0), (2, 96), (1025, 64)])
def test_gather_refuses_heads_and_dims_by_name(dm, heads, dim):
    c = Cache4([20], heads=1, dim=64, dcp=1, interleave=1, block=16, seed=1)
    cu = torch.tensor([0, 4], dtype=torch.int32, device="cuda")
    outs = [torch.empty(1 << 18, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    pool = torch.empty(1 << 24, dtype=torch.uint8, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    with pytest.raises(dm.DcpError, match="head_dim" if heads == 2 else "kv_heads"):
        dm.dcp_gqa_kv_gather(c.dims(dm), heads, dim, None, cu, c.table.cuda(), pool, pool, dm.KV_NVFP4, *c.scales(), 0, 1,
                             *outs, status)


def test_compaction_of_4_bit_rows_and_their_read_back(dm):
    # kept rows move byte for byte; what is read back and decoded is the kept tokens
    W, S, bs, heads, dim, budget = 2, 2, 8, 2, 64, 40
    c = Cache4([95, 40, 61], heads=heads, dim=dim, dcp=W, interleave=S, block=bs, seed=11)
    n, width = heads * dim, oracle.fp4.row_bytes(heads * dim)
    dims = c.dims(dm, 1, 4)
    g = torch.Generator().manual_seed(2)
    ev = dm.KvEviction(dims, budget=budget, sink=2, recent=3)
    ev.weights.copy_(torch.rand(ev.weights.shape, generator=g))
    lens, table = torch.tensor(c.lens, dtype=torch.int32, device="cuda"), c.table.cuda()
    keep_idx, keep_count, new_lens = ev.select(lens)
    pools = [x.view(W, c.NB, bs, width).cuda() for x in c.pools]
    ev.compact(pools[0], table, move_weights=False)
    ev.compact(pools[1], table)
    assert ev.read_status() == 0 and new_lens.tolist() == [39, 40, 37]
    short = new_lens.tolist()
    cu = torch.tensor([0, *np.cumsum(short)], dtype=torch.int32, device="cuda")
    outs = [torch.empty(sum(short), heads, dim, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    dm.dcp_gqa_kv_gather(dims, heads, dim, None, cu, table, *pools, dm.KV_NVFP4, *c.scales(), 0, W, *outs, status)
    assert int(status) == 0
    kept = [[], []]  # rows of the old pools that a sequence's positions now stand for
    for b, length in enumerate(short):
        p = np.arange(length)
        r, li = oracle.metadata.owner(p, W, S), oracle.metadata.local_index(p, W, S)
        old = keep_idx[:, b].cpu().numpy()[r, li]
        assert (old >= li).all()
        at = (r, c.table[b].numpy()[old // bs], old % bs)
        for i in range(2):
            kept[i].append(c.values[i][at])
    for i, s in enumerate(c.scales()):
        want = np.concatenate(kept[i]).astype(np.float32) * np.float32(s.item())
        assert torch.equal(outs[i].cpu(), torch.from_numpy(want).bfloat16().view(-1, heads, dim))
    q = _q(3, 4, dim)
    step = dm.GqaDecode(dims, heads, dim, dm.KV_NVFP4)
    out, lse = step(q.cuda(), *pools, *c.scales(), 0.2, new_lens, table)
    assert step.read_status() == 0
    for b in range(3):
        values = [np.float64(np.float32(s.item())) * x[b] for s, x in zip(c.scales(), kept)]
        ref = oracle.prompt.attend(q=ch.f64(q[b:b + 1]), k=values[0], v=values[1], cu_q=[0, 1], cu_k=[0, short[b]],
                                   softmax_scale=0.2)
        ch.assert_gqa(out[b:b + 1], lse[b:b + 1], ref, dim, b)
