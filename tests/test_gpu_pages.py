"""A step's pages and rotary positions on the GPU: the pages entry for entry against the oracle's
free list, the rotation against float64."""

import ctypes
import random

import numpy as np
import pytest
import torch

import oracle

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dm():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    import decode_context_mla_causal_gb300 as mod

    return mod


# ------------------------------------------------------------------ pages


class Pages:
    """Requests of random lengths over a shuffled pool; the rest of it is free."""

    def __init__(self, lens, *, dcp, interleave, block, bound, spare, seed):
        self.W, self.S, self.bs, self.B = dcp, interleave, block, len(lens)
        self.ML = oracle.evict.local_count(bound, 0, dcp, interleave)
        self.MB = max(1, -(-self.ML // block))
        held = [-(-oracle.evict.local_count(n, 0, dcp, interleave) // block) for n in lens]
        self.NB = sum(held) + spare + 2
        perm = list(range(self.NB))
        random.Random(seed).shuffle(perm)
        self.table = torch.full((self.B, self.MB), -7, dtype=torch.int32)
        for b, n in enumerate(held):
            self.table[b, :n] = torch.tensor(perm[:n], dtype=torch.int32)
            perm = perm[n:]
        self.free = torch.full((self.NB,), -9, dtype=torch.int32)
        self.count = spare
        self.free[:spare] = torch.tensor(perm[:spare], dtype=torch.int32)
        self.lens = torch.tensor(lens, dtype=torch.int32)

    def dims(self, dm):
        return dm.make_dims(batch=self.B, qlen=1, num_heads=1, dcp=self.W, interleave=self.S,
                            block_size=self.bs, max_blocks_per_seq=self.MB, max_local_len=self.ML,
                            num_blocks=self.NB, num_splits=1)

    def expect(self, targets, rows, **kw):
        return oracle.pages.plan(targets=targets, seq_lens=self.lens.numpy(), block_table=self.table.numpy(),
                                 free_list=self.free.numpy(), free_count=self.count, max_rows=rows, dcp=self.W,
                                 interleave=self.S, block_size=self.bs, max_local_len=self.ML,
                                 num_blocks=self.NB, **kw)

    def device(self):
        return dict(seq_lens=self.lens.cuda(), block_table=self.table.cuda(), free_list=self.free.cuda(),
                    free_count=torch.tensor([self.count], dtype=torch.int32, device="cuda"))


def _check(plan, state, ref, status=None):
    torch.cuda.synchronize()
    assert plan.read_status() == (ref["status"] if status is None else status)
    for name, got in (("new_lens", state["seq_lens"]), ("block_table", state["block_table"]),
                      ("free_list", state["free_list"]), ("slot_mapping", plan.slot_mapping),
                      ("positions", plan.positions), ("cu_rows", plan.cu_rows)):
        assert np.array_equal(got.cpu().numpy(), ref[name]), name
    assert int(state["free_count"]) == ref["free_count"]
    assert int(plan.workspace) == 0


PLANS = [  # lens, targets, dcp, interleave, block, spare, max_rows
    ([0], [1], 1, 1, 1, 1, 1),                                         # the first token of all
    ([5], [5], 2, 1, 4, 0, 3),                                         # nothing to do
    ([7, 0, 9], [0, 13, 0], 2, 2, 4, 0, 16),                           # a prompt in the blocks of those that ended
    ([100, 64, 63, 1], [101, 65, 64, 2], 4, 16, 16, 3, 4),             # one token each, at block borders
    ([30, 200, 0, 17], [25, 190, 40, 0], 3, 6, 24, 2, 64),             # drafts dropped, a prompt, one that ended
    ([10, 10, 10, 10], [12, 50, 11, 9], 1, 1, 8, 1, 100),              # the second does not fit: the third waits too
    ([0, 0, 0], [40, 40, 40], 8, 1, 5, 50, 90),                        # rows run out before blocks
    (list(range(60)), [x * 7 % 90 for x in range(60)], 2, 8, 8, 40, 1700),
    ([3] * 700, [4 + i % 5 for i in range(700)], 2, 1, 4, 900, 2800),  # more requests than threads, several CTAs
]


@pytest.mark.parametrize("case", PLANS, ids=lambda c: f"{len(c[0])}-W{c[2]}-S{c[3]}-bs{c[4]}")
def test_plan_against_the_oracle(dm, case):
    lens, targets, W, S, bs, spare, rows = case
    pages = Pages(lens, dcp=W, interleave=S, block=bs, bound=max(max(lens), max(targets), 1), spare=spare, seed=len(lens))
    plan, state = dm.PagePlan(pages.dims(dm), rows), pages.device()
    plan(torch.tensor(targets, dtype=torch.int32, device="cuda"), **state)
    _check(plan, state, pages.expect(targets, rows))


def test_plan_apart_can_be_repeated(dm):
    lens, targets = [40, 0, 300, 11], [0, 77, 301, 5]
    pages = Pages(lens, dcp=2, interleave=4, block=8, bound=400, spare=4, seed=1)
    plan, state = dm.PagePlan(pages.dims(dm), 90), pages.device()
    ref = pages.expect(targets, 90)
    for _ in range(3):
        plan(torch.tensor(targets, dtype=torch.int32, device="cuda"), **state, new_lens=plan.new_lens,
             new_count=plan.new_count)
        assert torch.equal(state["seq_lens"].cpu(), pages.lens) and int(state["free_count"]) == pages.count
        _check(plan, dict(state, seq_lens=plan.new_lens, free_count=plan.new_count), ref)


def test_plan_there_and_back_leaves_the_list(dm):
    # a verify step grows every request by its drafts; rejecting all of them undoes it
    lens = [31, 64, 7, 0, 129]
    pages = Pages(lens, dcp=2, interleave=1, block=4, bound=200, spare=30, seed=3)
    plan, state = dm.PagePlan(pages.dims(dm), 64), pages.device()
    plan((pages.lens + 9).cuda(), **state)
    assert int(state["free_count"]) < pages.count
    plan(pages.lens.cuda(), **state)
    assert torch.equal(state["free_list"].cpu()[:pages.count], pages.free[:pages.count])
    assert int(state["free_count"]) == pages.count and torch.equal(state["seq_lens"].cpu(), pages.lens)
    assert int(plan.cu_rows[-1]) == 0 and bool((plan.slot_mapping == -1).all()) and plan.read_status() == 0


def test_plan_many_steps_keep_every_block_once(dm):
    rng = random.Random(5)
    pages = Pages([0] * 24, dcp=3, interleave=2, block=4, bound=120, spare=160, seed=6)
    plan, state = dm.PagePlan(pages.dims(dm), 500), pages.device()
    for _ in range(30):
        targets = [rng.choice([0, n, n + 1, rng.randrange(0, 121)]) for n in pages.lens.tolist()]
        targets = [min(120, t) for t in targets]
        ref = pages.expect(targets, 500)
        plan(torch.tensor(targets, dtype=torch.int32, device="cuda"), **state)
        plan.status.zero_()
        _check(plan, state, ref, status=0)
        pages.lens = torch.tensor(ref["new_lens"], dtype=torch.int32)
        pages.table = torch.tensor(ref["block_table"], dtype=torch.int32)
        pages.free, pages.count = torch.tensor(ref["free_list"], dtype=torch.int32), ref["free_count"]
        held = [int(x) for b, n in enumerate(ref["new_lens"])
                for x in pages.table[b, :-(-oracle.evict.local_count(int(n), 0, 3, 2) // 4)]]
        ids = held + pages.free[:pages.count].tolist()
        assert len(set(ids)) == len(ids) == 160


def test_plan_one_rank_per_call(dm):
    lens, targets = [40, 3, 0], [44, 3, 21]
    pages = Pages(lens, dcp=4, interleave=2, block=6, bound=60, spare=9, seed=2)
    for r in range(4):
        plan, state = dm.PagePlan(pages.dims(dm), 30, rank_begin=r, num_ranks=1), pages.device()
        plan(torch.tensor(targets, dtype=torch.int32, device="cuda"), **state)
        _check(plan, state, pages.expect(targets, 30, rank_begin=r, num_ranks=1))


def test_plan_bad_inputs_set_status(dm):
    # lengths below zero and above the bound stay; the others go on
    pages = Pages([10, 20, 30, 5], dcp=2, interleave=1, block=4, bound=64, spare=20, seed=4)
    pages.lens[1] = -3
    targets = [-1, 4, 500, 9]
    plan, state = dm.PagePlan(pages.dims(dm), 16), pages.device()
    plan(torch.tensor(targets, dtype=torch.int32, device="cuda"), **state)
    ref = pages.expect(targets, 16)
    assert ref["status"] == dm.STATUS_BAD_SEQ_LEN | dm.STATUS_LOCAL_OVER_BOUND
    _check(plan, state, ref)
    # ids outside the pool, in the table and in the list
    pages = Pages([6, 0], dcp=1, interleave=1, block=4, bound=16, spare=2, seed=4)
    pages.table[0, 1] = pages.NB
    pages.free[1] = -4
    plan, state = dm.PagePlan(pages.dims(dm), 16), pages.device()
    plan(torch.tensor([8, 4], dtype=torch.int32, device="cuda"), **state)
    ref = pages.expect([8, 4], 16)
    assert ref["status"] == dm.STATUS_BAD_BLOCK_ID
    _check(plan, state, ref)
    # counts outside the pool, and a list that would outgrow it
    for count in (-5, pages.NB + 3):
        pages = Pages([6, 9], dcp=1, interleave=1, block=4, bound=16, spare=2, seed=4)
        pages.count = count
        plan, state = dm.PagePlan(pages.dims(dm), 16), pages.device()
        plan(torch.tensor([0, 9], dtype=torch.int32, device="cuda"), **state)
        _check(plan, state, pages.expect([0, 9], 16))
        assert plan.read_status() == dm.STATUS_BAD_PAGE


def test_plan_in_a_graph(dm):
    pages = Pages([31, 0, 64], dcp=2, interleave=1, block=16, bound=100, spare=9, seed=3)
    plan, state = dm.PagePlan(pages.dims(dm), 600), pages.device()
    targets = pages.lens.cuda()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        plan(targets, **state)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        plan(targets, **state)
    for step in ([32, 40, 64], [33, 41, 0], [0, 42, 17]):
        ref = pages.expect(step, 600)
        targets.copy_(torch.tensor(step, dtype=torch.int32))
        g.replay()
        _check(plan, state, ref)
        pages.lens = torch.tensor(ref["new_lens"], dtype=torch.int32)
        pages.table = torch.tensor(ref["block_table"], dtype=torch.int32)
        pages.free, pages.count = torch.tensor(ref["free_list"], dtype=torch.int32), ref["free_count"]


# ------------------------------------------------------------------ rotary positions


def _rope_tolerance(ref, x, rot):
    """Cosine and sine: the turn is cut to 2^-32 of a turn and rounded to fp32 (2^-25 half turns):
    together below 2^-23 rad; two ulp of sincospi and the amplitude's product, 2^-22. Two products
    and a sum: 3 roundings of at most 2^-24 of |a| + |b|; then half a bf16 step."""
    size = np.abs(x[..., :rot]).max() * 2
    return 2.0 ** -8 * np.abs(ref) + 2.0 ** -20 * size * 3


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rows,heads,kv,dim,rot", [
    (1, 1, 1, 16, 16), (3, 5, 1, 64, 32), (17, 8, 2, 128, 128), (300, 3, 3, 80, 48), (700, 2, 1, 256, 256),
    (40, 128, 1, 64, 64), (5, 1, 1, 1024, 1024)])
def test_rope_against_float64(dm, rows, heads, kv, dim, rot, interleaved):
    g = torch.Generator().manual_seed(rows + dim)
    q, k = (torch.randn(rows, h, dim, generator=g).bfloat16() for h in (heads, kv))
    pos = torch.randint(-(1 << 31), (1 << 31) - 1, (rows,), generator=g, dtype=torch.int64).to(torch.int32)
    pos[: rows // 2] %= 4096
    pos[0] = 0
    rope = dm.Rope(rot, base=10000.0, interleaved=interleaved)
    freq, amp = oracle.prompt.frequencies(rot, 10000.0)
    outs = rope(pos.cuda(), q.cuda(), k.cuda(), out_q=torch.full_like(q, float("nan"), device="cuda"),
                out_k=torch.full_like(k, float("nan"), device="cuda"))
    for x, y in zip((q, k), outs):
        # the frequency is rounded to 2^-53 of itself: far positions move by 2^31 of that
        ref = oracle.prompt.rotate(x.double().numpy(), pos.numpy(), freq, amp, interleaved)
        got = y.double().cpu().numpy()
        assert (np.abs(got - ref) <= _rope_tolerance(ref, x.double().numpy(), rot)).all()
        assert np.array_equal(got[..., rot:], x.double().numpy()[..., rot:])
        assert np.array_equal(got[0], x.double().numpy()[0])  # position 0 turns nothing
    # in place gives the same bits, and one operand alone too
    q2, k2 = q.cuda(), k.cuda()
    rope(pos.cuda(), q2, k2)
    assert torch.equal(q2, outs[0]) and torch.equal(k2, outs[1])
    alone, none = rope(pos.cuda(), q.cuda())
    assert torch.equal(alone, outs[0]) and none is None


def test_rope_scaled(dm):
    pos = torch.tensor([0, 1, 100, 4095, 131071, 1 << 20], dtype=torch.int32)
    x = torch.randn(6, 2, 64, generator=torch.Generator().manual_seed(1)).bfloat16()
    for scaling, kw in ((dict(kind="linear", factor=8.0), dict(kind="linear", factor=8.0)),
                        (dict(kind="yarn", factor=32.0, original_len=4096),
                         dict(kind="yarn", factor=32.0, original_len=4096)),
                        (dict(kind="yarn", factor=4.0, original_len=1024, beta_fast=20.0, beta_slow=2.0, amplitude=1.5),
                         dict(kind="yarn", factor=4.0, original_len=1024, beta_fast=20.0, beta_slow=2.0, amplitude=1.5))):
        rope = dm.Rope(64, base=50000.0, scaling=scaling)
        freq, amp = oracle.prompt.frequencies(64, 50000.0, **kw)
        got = rope(pos.cuda(), x.cuda())[0].double().cpu().numpy()
        ref = oracle.prompt.rotate(x.double().numpy(), pos.numpy(), freq, amp, False)
        assert (np.abs(got - ref) <= 2 * _rope_tolerance(ref, x.double().numpy(), 64)).all()


def test_rope_strided_views_and_back(dm):
    # the rotary part of latent heads, from one buffer's rows to another's, nothing else touched
    g = torch.Generator().manual_seed(3)
    src = torch.randn(9, 4, 192, generator=g).bfloat16().cuda()
    dst = torch.full((9, 4, 576), 7.0, dtype=torch.bfloat16, device="cuda")
    before = src.clone()
    pos = torch.arange(9, dtype=torch.int32, device="cuda") * 70001
    rope = dm.Rope(64, interleaved=True)
    rope(pos, src[..., 128:], out_q=dst[..., 512:])
    freq, amp = oracle.prompt.frequencies(64, 10000.0)
    x = src[..., 128:].double().cpu().numpy()
    ref = oracle.prompt.rotate(x, pos.cpu().numpy(), freq, amp, True)
    assert (np.abs(dst[..., 512:].double().cpu().numpy() - ref) <= _rope_tolerance(ref, x, 64)).all()
    assert torch.equal(src, before) and bool((dst[..., :512] == 7.0).all())
    # and back: two roundings to bf16 and two rotations' tolerance
    back = dst[..., 512:].contiguous()
    rope(-pos, back)
    tol = 2 * _rope_tolerance(x, x, 64) + 2.0 ** -8 * np.abs(x).max()
    assert (np.abs(back.double().cpu().numpy() - x) <= tol).all()


@pytest.mark.parametrize("rows,heads,row,head", [(3, 2, 128, 192), (7, 6, 384, 64), (7, 6, 64, 448), (3, 2, -128, 192),
                                                 (3, 2, 128, -64)])
def test_rope_outputs_that_interleave_without_meeting(dm, rows, heads, row, head):
    # rows inside a head's step, heads inside a row's, and places of both between each other
    dim = 64
    g = torch.Generator().manual_seed(1)
    x = torch.randn(rows, heads, dim, generator=g).bfloat16().cuda()
    at = [[i * row + j * head for j in range(heads)] for i in range(rows)]
    low = min(min(a) for a in at)
    pos = torch.arange(rows, dtype=torch.int32, device="cuda") * 1001
    rope = dm.Rope(dim)
    want, _ = rope(pos, x, out_q=torch.empty_like(x))
    flat = torch.full((max(max(a) for a in at) - low + dim,), 7.0, dtype=torch.bfloat16, device="cuda")
    from decode_context_mla_causal_gb300.binding import RopeHeads

    side = RopeHeads(x.data_ptr(), flat.data_ptr() - 2 * low, heads * dim, dim, row, head, heads)
    code = dm.load().dcp_rope(rows, dim, dim, 0, pos.data_ptr(), rope.table.data_ptr(), 1.0, ctypes.byref(side), None,
                              torch.cuda.current_stream().cuda_stream)
    assert code == dm.DCP_OK, dm.dcp_last_error()
    torch.cuda.synchronize()
    left = torch.ones_like(flat, dtype=torch.bool)
    for i in range(rows):
        for j in range(heads):
            of = slice(at[i][j] - low, at[i][j] - low + dim)
            assert torch.equal(flat[of], want[i, j]) and bool(left[of].all())
            left[of] = False
    assert bool((flat[left] == 7).all())


@pytest.mark.parametrize("bad", [-1, 1 << 30, "first behind"])
def test_plan_bad_ids_given_back_set_status(dm, bad):
    # a request that ends gives back an id outside the pool: known at once, not when it is handed out again
    pages = Pages([30, 9, 0], dcp=2, interleave=1, block=4, bound=64, spare=5, seed=7)
    pages.table[0, 2] = pages.NB if bad == "first behind" else bad
    targets = [0, 10, 3]  # two blocks are handed out, the third of those given back goes onto the list
    plan, state = dm.PagePlan(pages.dims(dm), 16), pages.device()
    plan(torch.tensor(targets, dtype=torch.int32, device="cuda"), **state)
    ref = pages.expect(targets, 16)
    assert ref["status"] == dm.STATUS_BAD_BLOCK_ID
    _check(plan, state, ref)
