"""Cases of the cache operators next to the verify path, and their plain forms.

Five operators over paged, interleaved rank pools (token p of a sequence lives on rank
(p // S) % dcp at local index (p // (S*dcp))*S + p % S; block_table[b] names its blocks):

* ``decode``:  grouped-head attention of the newest tokens over a paged K/V cache,
  split over the cache's length and joined.
* ``write``:   the new tokens' K and V rows into the pools (E4M3 or BF16).
* ``weights``: the attention weight that each cached latent row receives from a verify
  step, accumulated per (rank, sequence, local index).
* ``select``:  which cached tokens a budget keeps: a protected head and tail and the
  heaviest tokens between them, in order.
* ``compact``: the kept rows moved together, in place or into other blocks.

``run`` computes the plain form with elementary torch operations where ``own`` is
false, and calls this package where it is true.
"""

import math
import random

import torch

own = False

D_LATENT = 576
SOFTMAX_SCALE = 1.0 / math.sqrt(192.0)  # of the latent cache's queries


# ------------------------------------------------------------------ the cases


def listed():
    return [
        # one short request, the smallest call: latency counts
        dict(name="decode one request", op="decode", batch=1, qlen=1, heads=32, kv_heads=8, dim=128,
             lo=200, hi=200, dcp=2, interleave=1, block=16, dtype="bf16", len_seed=1),
        # a batch of ragged requests with two rows each and an odd number of heads in a group
        dict(name="decode ragged bf16", op="decode", batch=24, qlen=2, heads=40, kv_heads=8, dim=128,
             lo=512, hi=32768, dcp=4, interleave=16, block=32, dtype="bf16", len_seed=2),
        # the single-token decode workload's lengths over an FP8 cache: bandwidth counts
        dict(name="decode batch fp8", op="decode", batch=32, qlen=1, heads=64, kv_heads=8, dim=128,
             lo=32768, hi=32768, dcp=8, interleave=1, block=64, dtype="fp8", len_seed=3),
        # one decode step's rows of a batch
        dict(name="write one step", op="write", batch=32, qlen=1, kv_heads=8, dim=128, lo=32, hi=4096,
             dcp=8, interleave=1, block=64, dtype="fp8", len_seed=4),
        # a prompt chunk of a few sequences
        dict(name="write prompt chunk", op="write", batch=5, qlen=4000, kv_heads=8, dim=128, lo=4000,
             hi=16384, dcp=4, interleave=16, block=64, dtype="fp8", len_seed=5),
        # the tiny verify workload
        dict(name="weights tiny bf16", op="weights", batch=1, qlen=3, heads=8, lo=200, hi=200, dcp=2,
             interleave=1, block=16, dtype="bf16", decay=1.0, len_seed=6),
        # the speculative verify workload's lengths, half its batch
        dict(name="weights verify fp8", op="weights", batch=16, qlen=5, heads=128, lo=8192, hi=131072,
             dcp=8, interleave=64, block=64, dtype="fp8", decay=0.98, len_seed=7),
        # the long-context workload
        dict(name="weights long fp8", op="weights", batch=4, qlen=3, heads=128, lo=1048576, hi=1048576,
             dcp=8, interleave=1, block=64, dtype="fp8", decay=1.0, len_seed=8),
        # a small ragged batch, some of it within the budget
        dict(name="select small", op="select", batch=4, lo=1024, hi=4096, dcp=2, interleave=1, block=64,
             budget=2000, sink=4, recent=128, len_seed=9),
        # the long-context workload cut to a quarter
        dict(name="select long", op="select", batch=4, lo=1048576, hi=1048576, dcp=8, interleave=1,
             block=64, budget=262144, sink=16, recent=1024, len_seed=10),
        # the decode workload cut to half, in place: a full pool has no blocks to spare
        dict(name="compact in place fp8", op="compact", batch=32, lo=32768, hi=32768, dcp=8,
             interleave=1, block=64, row=576, dtype="fp8", budget=16384, sink=4, recent=256,
             in_place=True, len_seed=11),
        # ragged sequences of a K/V cache into other blocks
        dict(name="compact to blocks bf16", op="compact", batch=12, lo=8192, hi=131072, dcp=4,
             interleave=16, block=32, row=1024, dtype="bf16", budget=30000, sink=64, recent=512,
             in_place=False, len_seed=12),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """One more case of the same ranges; no drawn case costs more than the largest listed."""
    op = rng.choice(["decode", "decode", "write", "weights", "weights", "select", "compact"])
    block = rng.choice([8, 16, 24, 32, 64, 96, 128])
    dcp = rng.choice([1, 2, 3, 4, 8])
    inter = rng.choice([1, 1, block, block // 2])
    case = dict(op=op, dcp=dcp, interleave=inter, block=block, len_seed=rng.randrange(1 << 30))
    if op != "select":
        case["dtype"] = rng.choice(["fp8", "bf16"])
    if op in ("decode", "write"):
        group = rng.choice([1, 2, 4, 5, 8, 16])
        case.update(kv_heads=rng.choice([1, 2, 4, 8, 16]), dim=rng.choice([64, 128]))
    if op == "decode":
        hi = _log_int(rng, 64, 65536)
        most = max(1, min(64, (1 << 20) // hi))  # tokens of the batch
        case.update(batch=_log_int(rng, 1, most), qlen=rng.choice([1, 1, 2, 4]),
                    heads=case["kv_heads"] * group, hi=hi, lo=max(4, hi // rng.choice([1, 2, 16])))
    elif op == "write":
        qlen = _log_int(rng, 1, 4000)
        batch = _log_int(rng, 1, max(1, 20000 // qlen))
        hi = qlen + rng.randrange(1, 4096)
        case.update(batch=min(batch, 64), qlen=qlen, lo=qlen, hi=hi)
    elif op == "weights":
        heads, qlen = rng.choice([8, 16, 24, 64, 96, 128]), rng.choice([1, 2, 3, 5, 8])
        hi = _log_int(rng, 64, 400000)
        most = max(1, min(48, (3 << 20) // hi))
        case.update(batch=_log_int(rng, 1, most), qlen=qlen, heads=heads, hi=hi,
                    lo=max(qlen, hi // rng.choice([1, 2, 16])), decay=rng.choice([1.0, 0.9, 0.0]))
    else:
        span = dcp * inter
        hi = _log_int(rng, 40 * span + 64, 600000)
        most = max(1, min(48, (1 << 20) // hi))
        case.update(batch=_log_int(rng, 1, most), hi=hi, lo=max(8, hi // rng.choice([1, 2, 16])))
        budget = max(4 * span + 8, int(hi * rng.uniform(0.1, 0.9)))
        local = (budget // span - 2) * inter
        case.update(budget=budget, sink=rng.randrange(0, local // 4 + 1),
                    recent=rng.randrange(0, local // 2 + 1))
        if op == "compact":
            case.update(row=rng.choice([128, 512, 576, 1024]), in_place=rng.random() < 0.5)
    most = [work(c) for c in listed() if c["op"] == op]
    while any(work(case)[n] > max(w[n] for w in most) for n in ("bytes", "flops")):
        if case["batch"] > 1:
            case["batch"] = (case["batch"] + 1) // 2
        else:
            case["row"] //= 2
    return case


# ------------------------------------------------------------------ sizes that follow from a case


def _lengths(case):
    r, lo, hi = random.Random(case["len_seed"]), case["lo"], case["hi"]
    return [hi if lo == hi else min(hi, max(lo, _log_int(r, lo, hi))) for _ in range(case["batch"])]


def _local(g, rank, dcp, inter):
    """Local length on a rank of a sequence of g tokens."""
    if g <= 0:
        return 0
    span = dcp * inter
    return g // span * inter + min(max(g % span - rank * inter, 0), inter)


def _bound(case):
    return max(1, _local(case["hi"], 0, case["dcp"], case["interleave"]))


def _kept_length(length, budget, span):
    return length if length <= budget else length - -(-(length - budget) // span) * span


def _max_keep(case):
    return min(_bound(case), _local(case["budget"], 0, case["dcp"], case["interleave"]))


def _elem(case):
    return 1 if case["dtype"] == "fp8" else 2


def work(case):
    op, tokens = case["op"], sum(_lengths(case))
    rows = case["batch"] * case.get("qlen", 1)
    if op == "decode":
        kv_row = 2 * case["kv_heads"] * case["dim"] * _elem(case)
        qo = rows * case["heads"] * (4 * case["dim"] + 4)
        return dict(bytes=tokens * kv_row + qo, flops=4 * case["qlen"] * tokens * case["heads"] * case["dim"])
    if op == "write":
        n = rows * case["kv_heads"] * case["dim"] * 2
        return dict(bytes=n * (2 + _elem(case)), flops=0)
    if op == "weights":
        row = D_LATENT * _elem(case)
        return dict(bytes=tokens * (row + 8) + rows * case["heads"] * (2 * D_LATENT + 4),
                    flops=2 * case["qlen"] * tokens * case["heads"] * D_LATENT)
    span = case["dcp"] * case["interleave"]
    kept = sum(_kept_length(n, case["budget"], span) for n in _lengths(case))
    if op == "select":
        return dict(bytes=4 * tokens + 4 * case["dcp"] * case["batch"] * _max_keep(case), flops=0)
    return dict(bytes=kept * (2 * case["row"] * _elem(case) + 12), flops=0)


# ------------------------------------------------------------------ inputs


def _values(shape, dtype, gen, scale=1.0):
    """N(0, 1) values: BF16, or E4M3 codes (uint8) of the values over `scale`."""
    n = math.prod(shape)
    out = torch.empty(n, dtype=torch.uint8 if dtype == "fp8" else torch.bfloat16, device="cuda")
    for i in range(0, n, 1 << 27):
        x = torch.randn(min(1 << 27, n - i), generator=gen, device="cuda")
        if dtype == "fp8":
            x = (x / scale).clamp_(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)
        out[i:i + x.numel()] = x
    return out.view(shape)


def _key_scale():
    return 6.0 / 448.0  # six standard deviations reach the largest code


def _tables(case, gen, spare=0):
    """Shuffled blocks: [batch][blocks of the longest sequence] (twice of them where spare)."""
    per = -(-_bound(case) // case["block"])
    total = case["batch"] * per * (2 if spare else 1) + 8
    perm = torch.randperm(total, generator=gen, device="cuda").to(torch.int32)
    first = perm[:case["batch"] * per].view(case["batch"], per).contiguous()
    second = perm[case["batch"] * per:2 * case["batch"] * per].view(case["batch"], per).contiguous() if spare else None
    return per, total, first, second


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op, W, bs, B = case["op"], case["dcp"], case["block"], case["batch"]
    ML = _bound(case)
    s = dict(case=case, seq_lens=torch.tensor(_lengths(case), dtype=torch.int32, device="cuda"))
    per, NB, table, other = _tables(case, gen, op == "compact" and not case["in_place"])
    s.update(blocks=per, num_blocks=NB, table=table)
    scale = _key_scale()
    s["scale"] = torch.tensor([scale], device="cuda") if case.get("dtype") == "fp8" else None
    R = B * case.get("qlen", 1)
    if op in ("decode", "write"):
        shape = (W, NB, bs, case["kv_heads"], case["dim"])
        s["k"] = _values(shape, case["dtype"], gen, scale)
        s["v"] = _values(shape, case["dtype"], gen, scale)
        s["v_scale"] = torch.tensor([0.75 * scale], device="cuda") if case["dtype"] == "fp8" else None
    if op == "decode":
        s["q"] = torch.randn(R, case["heads"], case["dim"], generator=gen, device="cuda").bfloat16()
    elif op == "write":
        s["k_new"] = torch.randn(R, case["kv_heads"], case["dim"], generator=gen, device="cuda").bfloat16()
        s["v_new"] = torch.randn(R, case["kv_heads"], case["dim"], generator=gen, device="cuda").bfloat16()
        # the slot mapping that the step's plan holds: one rank's row, -1 on the others
        pos = (s["seq_lens"].long()[:, None] - case["qlen"] + torch.arange(case["qlen"], device="cuda"))
        span, inter = W * case["interleave"], case["interleave"]
        local = pos // span * inter + pos % inter
        slot = table.long().gather(1, local // bs) * bs + local % bs
        mine = (pos // inter % W)[None] == torch.arange(W, device="cuda")[:, None, None]
        s["slots"] = torch.where(mine, slot[None], -1).to(torch.int32).view(W, R).contiguous()
    elif op == "weights":
        s["kv"] = _values((W, NB, bs, D_LATENT), case["dtype"], gen, scale)
        s["q"] = torch.randn(R, case["heads"], D_LATENT, generator=gen, device="cuda").bfloat16()
        # what earlier steps left; behind a sequence's old tokens the slots hold anything
        s["history"] = torch.rand(W, B, ML, generator=gen, device="cuda")
        old = _local_lens(s["seq_lens"].long() - case["qlen"], case)
        s["history"][torch.arange(ML, device="cuda") >= old[:, :, None]] = math.nan
        s["lse"] = _lse_of(s)
    elif op in ("select", "compact"):
        # accumulated weights: heavy tails, and many tokens that nothing attends
        w = torch.randn(W, B, ML, generator=gen, device="cuda").mul_(3.0).exp_()
        s["weights"] = w.mul_((torch.rand(W, B, ML, generator=gen, device="cuda") > 0.2).float())
    if op == "compact":
        s["keep_idx"], s["keep_count"], _ = _plain_select(s)
        s["pool"] = _values((W, NB, bs, case["row"]), case["dtype"], gen, scale)
        s["to"] = table if case["in_place"] else other
    return s


def _lse_of(s):
    """The natural-log LSE that the verify step returned for these queries."""
    case, rows, out = s["case"], s["case"]["qlen"] * s["case"]["heads"], []
    seen = _visible(s)  # [W][B][ML][qlen]
    for b in range(case["batch"]):
        q = s["q"][b * case["qlen"]:(b + 1) * case["qlen"]].float().reshape(rows, D_LATENT)
        lse = torch.full((rows,), -math.inf, device="cuda")
        for r in range(case["dcp"]):
            key = _latent_rows(s, r, b)
            x = (q @ key.T) * (SOFTMAX_SCALE * _scale_of(s))
            m = seen[r, b].T[:, None, :].expand(-1, case["heads"], -1).reshape(rows, -1)
            lse = torch.logaddexp(lse, x.masked_fill_(~m, -math.inf).logsumexp(1))
        out.append(lse.view(case["qlen"], case["heads"]))
    return torch.cat(out)


def _latent_rows(s, r, b):
    rows = _pool_rows(s["table"][b:b + 1], _bound(s["case"]), s["case"]["block"])[0]
    return _decode(s["kv"][r].view(-1, D_LATENT)[rows], s["case"])


# ------------------------------------------------------------------ the plain forms


def _scale_of(s):
    return _key_scale() if s["case"]["dtype"] == "fp8" else 1.0


def _decode(x, case):
    return (x.view(torch.float8_e4m3fn) if case["dtype"] == "fp8" else x).float()


def _local_lens(g, case):
    """[W][B] local lengths of global lengths g [B]."""
    inter = case["interleave"]
    span = case["dcp"] * inter
    ranks = torch.arange(case["dcp"], device=g.device)[:, None]
    return torch.where(g > 0, g // span * inter + (g % span - ranks * inter).clamp(0, inter), 0)


def _visible(s):
    """[W][B][ML][qlen]: whether row j sees local token t."""
    case = s["case"]
    q = case["qlen"]
    g = s["seq_lens"].long()[:, None] - q + 1 + torch.arange(q, device="cuda")  # [B][q]
    n = _local_lens(g.reshape(-1), case).view(case["dcp"], case["batch"], 1, q)
    return torch.arange(_bound(case), device="cuda")[:, None] < n


def _pool_rows(table, n, bs):
    """[B][n] rows of a rank's flat pool of local tokens 0 .. n-1."""
    t = torch.arange(n, device=table.device)
    return table.long()[:, t // bs] * bs + t % bs


def _plain_decode(s):
    case = s["case"]
    W, B, q, hk, d = case["dcp"], case["batch"], case["qlen"], case["kv_heads"], case["dim"]
    group, ML = case["heads"] // hk, _bound(case)
    rows = _pool_rows(s["table"], ML, case["block"])
    k = _decode(s["k"].view(W, -1, hk, d)[:, rows], case).permute(1, 3, 0, 2, 4).reshape(B, hk, W * ML, d)
    v = _decode(s["v"].view(W, -1, hk, d)[:, rows], case).permute(1, 3, 0, 2, 4).reshape(B, hk, W * ML, d)
    qq = s["q"].float().view(B, q, hk, group, d).permute(0, 2, 1, 3, 4).reshape(B, hk, q * group, d)
    x = (qq @ k.transpose(2, 3)) * (d ** -0.5 * _scale_of(s))
    seen = _visible(s).permute(1, 3, 0, 2).reshape(B, 1, q, 1, W * ML)
    x = x.view(B, hk, q, group, W * ML).masked_fill_(~seen, -math.inf)
    top = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(top == -math.inf, 0.0, top))
    total = p.sum(-1, keepdim=True)
    o = (p.view(B, hk, q * group, W * ML) @ v).view(B, hk, q, group, d) * (0.75 * _scale_of(s) if case["dtype"] == "fp8" else 1.0)
    o = torch.where(total > 0, o / total, 0.0).permute(0, 2, 1, 3, 4).reshape(B * q, case["heads"], d)
    lse = (top + torch.log(total)).squeeze(-1).permute(0, 2, 1, 3).reshape(B * q, case["heads"])
    return dict(out=o.bfloat16(), lse=lse)


def _plain_rows(x, scale, case):
    """New rows as the pool holds them."""
    if case["dtype"] == "bf16":
        return x
    return (x.float() / scale).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)


def _as_values(pool, case):
    return pool.view(torch.float8_e4m3fn) if case["dtype"] == "fp8" else pool


def _plain_write(s):
    case = s["case"]
    W, hk, d = case["dcp"], case["kv_heads"], case["dim"]
    rank, row = torch.nonzero(s["slots"] >= 0, as_tuple=True)
    at = s["slots"][rank, row].long()
    s["k"].view(W, -1, hk, d)[rank, at] = _plain_rows(s["k_new"][row], s["scale"], case)
    s["v"].view(W, -1, hk, d)[rank, at] = _plain_rows(s["v_new"][row], s["v_scale"], case)
    return dict(k=_as_values(s["k"], case), v=_as_values(s["v"], case))


def _plain_weights(s):
    case = s["case"]
    W, B, q, H, ML = case["dcp"], case["batch"], case["qlen"], case["heads"], _bound(case)
    rows = _pool_rows(s["table"], ML, case["block"])
    key = _decode(s["kv"].view(W, -1, D_LATENT)[:, rows], case)                      # [W][B][ML][576]
    qq = s["q"].float().view(B, q * H, D_LATENT).transpose(1, 2)
    x = (key @ qq) * (SOFTMAX_SCALE * _scale_of(s)) - s["lse"].view(B, 1, q * H)    # [W][B][ML][q*H]
    p = x.exp_().view(W, B, ML, q, H).sum(-1)
    p = torch.where(_visible(s), p, 0.0).sum(-1)
    t = torch.arange(ML, device="cuda")
    old = _local_lens(s["seq_lens"].long() - q, case)[:, :, None]
    return torch.where(t < old, case["decay"] * s["history"], 0.0) + p


def _plain_select(s):
    case = s["case"]
    span = case["dcp"] * case["interleave"]
    L = s["seq_lens"].long()
    cut = torch.where(L > case["budget"], (L - case["budget"] + span - 1) // span * span, 0)
    n, k = _local_lens(L, case)[:, :, None], _local_lens(L - cut, case)[:, :, None]
    t = torch.arange(_bound(case), device="cuda")
    ends = (t < case["sink"]) | (t >= n - case["recent"])
    free = ~ends & (t < n)
    w = torch.where(torch.isnan(s["weights"]), -math.inf, s["weights"]) + 0.0
    order = w.sort(dim=-1, descending=True, stable=True).indices
    # the free tokens first, in the order of their weights; equal ones in their own order
    order = order.gather(-1, free.gather(-1, order).sort(dim=-1, descending=True, stable=True).indices)
    place = torch.empty_like(order).scatter_(-1, order, t.expand_as(order).contiguous())
    ends_n = (ends & (t < n)).sum(-1, keepdim=True)
    keep = torch.where(n == k, t < n, (ends & (t < n)) | (free & (place < k - ends_n)))
    at = torch.where(keep, keep.long().cumsum(-1) - 1, _max_keep(case))
    idx = torch.full((*keep.shape[:2], _max_keep(case) + 1), -1, dtype=torch.int64, device="cuda")
    idx.scatter_(-1, at, torch.where(keep, t, -1))
    return (idx[..., :-1].to(torch.int32).contiguous(), k[:, :, 0].to(torch.int32).contiguous(),
            (L - cut).to(torch.int32))


def _plain_compact(s):
    case = s["case"]
    bs, i = case["block"], torch.arange(s["keep_idx"].shape[2], device="cuda")
    rank, b, i = torch.nonzero(i < s["keep_count"][:, :, None], as_tuple=True)
    t = s["keep_idx"][rank, b, i].long()
    src = s["table"][b, t // bs].long() * bs + t % bs
    dst = s["to"][b, i // bs].long() * bs + i % bs
    flat = s["pool"].view(case["dcp"], -1, case["row"])
    flat[rank, dst] = flat[rank, src]
    s["weights"][rank, b, i] = s["weights"][rank, b, t]
    return dict(pool=_as_values(s["pool"], case), weights=s["weights"])


# ------------------------------------------------------------------ the framework's calls


def _handle(s):
    """What a program builds once for its shapes and keeps: dims, plan and buffers."""
    import decode_context_mla_causal_gb300 as dm

    if "handle" not in s:
        case = s["case"]
        dims = dm.make_dims(batch=case["batch"], qlen=case.get("qlen", 1), num_heads=case.get("heads", 1),
                            dcp=case["dcp"], interleave=case["interleave"], block_size=case["block"],
                            max_blocks_per_seq=s["blocks"], max_local_len=_bound(case),
                            num_blocks=s["num_blocks"], num_splits=1)
        kv = dm.KV_FP8_E4M3 if case.get("dtype") == "fp8" else dm.KV_BF16
        if case["op"] == "decode":
            h = dm.GqaDecode(dims, case["kv_heads"], case["dim"], kv)
        elif case["op"] == "write":
            h = torch.zeros(1, dtype=torch.int32, device="cuda")  # the status word
        else:
            h = dm.KvEviction(dims, case.get("budget"), sink=case.get("sink", 0),
                              recent=case.get("recent", 0), decay=case.get("decay", 1.0))
        s["handle"] = (dm, dims, kv, h)
    return s["handle"]


def _own(s):
    dm, dims, kv, h = _handle(s)
    case = s["case"]
    op = case["op"]
    if op == "decode":
        out, lse = h(s["q"], s["k"], s["v"], s["scale"], s["v_scale"], case["dim"] ** -0.5, s["seq_lens"], s["table"])
        return dict(out=out, lse=lse)
    if op == "write":
        dm.dcp_gqa_kv_write(dims, case["kv_heads"], case["dim"], s["slots"], s["k_new"], s["v_new"], kv,
                            s["scale"], s["v_scale"], case["dcp"], s["k"], s["v"], h)
        return dict(k=_as_values(s["k"], case), v=_as_values(s["v"], case))
    if op == "weights":
        return h.accumulate(s["q"], s["kv"], kv, s["scale"], SOFTMAX_SCALE, s["lse"], s["seq_lens"], s["table"],
                            history=s["history"])
    if op == "select":
        return h.select(s["seq_lens"], weights=s["weights"])
    h.compact(s["pool"], s["table"], None if case["in_place"] else s["to"], keep_idx=s["keep_idx"],
              keep_count=s["keep_count"], weights=s["weights"])
    return dict(pool=_as_values(s["pool"], case), weights=s["weights"])


def run(state):
    if own:
        return _own(state)
    return {"decode": _plain_decode, "write": _plain_write, "weights": _plain_weights,
            "select": _plain_select, "compact": _plain_compact}[state["case"]["op"]](state)


# ------------------------------------------------------------------ 64-bit values


def _tokens_of(s, b, pool, case):
    """Rows of sequence b's tokens in global order, in 64 bits: each token is looked up by its position."""
    p = torch.arange(int(s["seq_lens"][b]), device="cuda")
    inter, W, bs = case["interleave"], case["dcp"], case["block"]
    chunk = p // inter
    local = chunk // W * inter + p % inter
    x = pool[chunk % W, s["table"][b].long()[local // bs], local % bs]
    return (x.view(torch.float8_e4m3fn) if case["dtype"] == "fp8" else x).double(), chunk % W, local


def exact(case, seed):
    if case["op"] in ("select", "compact"):
        return None  # whole numbers, and rows that are moved
    s = prepare(case, seed)
    if case["op"] == "write":
        return _exact_write(s)
    B, q, H = case["batch"], case["qlen"], case["heads"]
    if case["op"] == "weights":
        done = torch.zeros(case["dcp"], B, _bound(case), dtype=torch.float64, device="cuda")
        for b in range(B):
            key, rank, local = _tokens_of(s, b, s["kv"], case)
            n = key.shape[0]
            got = torch.zeros(n, dtype=torch.float64, device="cuda")
            for j in range(q):
                end = n - q + 1 + j
                row = s["q"][b * q + j].double()
                lse = s["lse"][b * q + j].double()
                x = (key[:end] @ row.T).mul_(SOFTMAX_SCALE * (float(s["scale"]) if s["scale"] is not None else 1.0))
                got[:end] += x.sub_(lse).exp_().sum(1)
            first = s["history"][rank, b, local].double()
            first[max(0, n - q):] = 0.0
            done[rank, b, local] = got + case["decay"] * first
        return done
    hk, d = case["kv_heads"], case["dim"]
    out = torch.zeros(B * q, H, d, dtype=torch.float64, device="cuda")
    lse = torch.full((B * q, H), -math.inf, dtype=torch.float64, device="cuda")
    ks, vs = (1.0 if s[n] is None else float(s[n]) for n in ("scale", "v_scale"))
    for b in range(B):
        key, val = _tokens_of(s, b, s["k"], case)[0], _tokens_of(s, b, s["v"], case)[0]
        for j in range(q):
            end = key.shape[0] - q + 1 + j
            if end < 1:
                continue
            for g in range(hk):
                of = slice(g * (H // hk), (g + 1) * (H // hk))
                x = (s["q"][b * q + j, of].double() @ key[:end, g].T) * (ks * d ** -0.5)
                lse[b * q + j, of] = x.logsumexp(1)
                out[b * q + j, of] = x.softmax(1) @ val[:end, g] * vs
    return dict(out=out, lse=lse)


def _exact_write(s):
    """Each new value over its scale at the nearest value the pool can hold, ties to an even last bit."""
    case = s["case"]
    held = [c / 8 * 2.0 ** -6 if c < 8 else (1 + c % 8 / 8) * 2.0 ** (c // 8 - 7) for c in range(127)]
    held = torch.tensor(held, dtype=torch.float64, device="cuda")
    done = {}
    for name, scale in (("k", s["scale"]), ("v", s["v_scale"])):
        pool = _as_values(s[name], case).double()
        new = s[name + "_new"]
        if case["dtype"] == "fp8":
            x = (new.float() / scale).double()  # the definition divides in 32 bits
            mag = x.abs().clamp(max=448.0)
            hi = torch.searchsorted(held, mag).clamp(max=126)
            lo = (hi - 1).clamp(min=0)
            up, down = held[hi] - mag, mag - held[lo]
            pick = torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
            new = held[pick] * x.sign()
        new = new.double()
        flat = pool.view(case["dcp"], -1, case["kv_heads"], case["dim"])
        for r in range(case["dcp"]):
            mine = s["slots"][r] >= 0
            flat[r, s["slots"][r][mine].long()] = new[mine]
        done[name] = pool
    return done
