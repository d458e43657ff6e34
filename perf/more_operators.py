"""Cases of the operators that bring prompts into the rank pools, and their plain forms.

Five operators around the paged, interleaved rank pools (token p of a sequence lives on rank
(p // S) % dcp at local index (p // (S*dcp))*S + p % S; block_table[b] names its blocks):

* ``plan``:   block tables, slot maps, positions and row offsets from the lengths that the
  requests have and those they are to have; blocks come from a free list and return to it.
* ``rope``:   rotary positions of query and key heads, interleaved or half layout, the first
  part of each head, frequencies scaled for long contexts.
* ``prompt``: causal attention over packed prompts with grouped heads, with or without a
  context in front of the new rows.
* ``cache``:  K and V rows into pools held in 4 bits (E2M1 codes, an E4M3 scale for every 16)
  and back out as packed rows.
* ``decode``: attention of the newest tokens over such pools.

``run`` computes the plain form with elementary torch operations where ``own`` is
false, and calls this package where it is true.
"""

import math
import random

import torch

own = False

MID = 0.75  # the value scale of V beside K's


# ------------------------------------------------------------------ the cases


def listed():
    return [
        # a decode step's bookkeeping: every request takes one more token, two have finished
        dict(name="plan decode step", op="plan", batch=64, lo=512, hi=131072, grow_lo=1, grow_hi=1, finish=2,
             dcp=8, interleave=1, block=64, room=1.0, len_seed=1),
        # admission: new prompts beside running requests, more than the pool has blocks for
        dict(name="plan admission", op="plan", batch=192, lo=0, hi=32768, grow_lo=1, grow_hi=4096, finish=24,
             dcp=4, interleave=16, block=32, room=0.97, len_seed=2),
        # a decode step's grouped heads: latency counts
        dict(name="rope one step", op="rope", rows=32, heads=64, kv_heads=8, dim=128, rot=128, interleaved=False,
             base=1e6, factor=1.0, reach=131072),
        # a prompt's latent heads: the 64 rotary dims out of rows of 192 into rows of 576,
        # frequencies scaled for the long-context workload's positions
        dict(name="rope latent prompt", op="rope", rows=8192, heads=128, kv_heads=1, dim=64, rot=64,
             interleaved=True, base=10000.0, factor=32.0, reach=1048576, latent=True),
        # one short request
        dict(name="prompt one request", op="prompt", batch=1, lo=200, hi=200, ctx=0, heads=32, kv_heads=8, dim=128,
             vdim=128, causal=True, len_seed=3),
        # a batch of ragged requests, an odd number of heads in a group
        dict(name="prompt ragged", op="prompt", batch=24, lo=100, hi=4096, ctx=0, heads=40, kv_heads=8, dim=128,
             vdim=128, causal=True, len_seed=4),
        # prompts of the latent workloads: keys of 192, values of 128, every head its own
        dict(name="prompt latent heads", op="prompt", batch=4, lo=1000, hi=5000, ctx=0, heads=128, kv_heads=128,
             dim=192, vdim=128, causal=True, len_seed=5),
        # a chunk of a long prompt behind what is cached already
        dict(name="prompt chunk of a long context", op="prompt", batch=1, lo=2048, hi=2048, ctx=32768, heads=64,
             kv_heads=8, dim=128, vdim=128, causal=True, len_seed=6),
        # one decode step's rows, and the same rows read back
        dict(name="cache one step", op="cache", batch=32, qlen=1, lo=32, hi=4096, kv_heads=8, dim=128, dcp=8,
             interleave=1, block=64, len_seed=7),
        # a prompt chunk of a few sequences
        dict(name="cache prompt chunk", op="cache", batch=5, qlen=4000, lo=4000, hi=16384, kv_heads=8, dim=128,
             dcp=4, interleave=16, block=64, len_seed=8),
        # one short request over the 4-bit cache
        dict(name="decode one request", op="decode", batch=1, qlen=1, lo=200, hi=200, heads=32, kv_heads=8, dim=128,
             dcp=2, interleave=1, block=16, len_seed=9),
        # the single-token decode workload's lengths: bandwidth counts
        dict(name="decode batch", op="decode", batch=32, qlen=1, lo=32768, hi=32768, heads=64, kv_heads=8, dim=128,
             dcp=8, interleave=1, block=64, len_seed=10),
    ]


def _log_int(rng, lo, hi):
    return lo if lo >= hi else int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """One more case of the same ranges; no drawn case costs more than the largest listed."""
    op = rng.choice(["plan", "rope", "prompt", "prompt", "cache", "decode", "decode"])
    case = dict(op=op, len_seed=rng.randrange(1 << 30))
    if op in ("plan", "cache", "decode"):
        block = rng.choice([8, 16, 24, 32, 64, 96, 128])
        case.update(block=block, dcp=rng.choice([1, 2, 3, 4, 8]), interleave=rng.choice([1, 1, block, block // 2]))
    if op == "plan":
        batch = _log_int(rng, 1, 400)
        case.update(batch=batch, lo=0, hi=_log_int(rng, 64, 131072), grow_lo=1,
                    grow_hi=_log_int(rng, 1, max(2, 200000 // batch)), finish=rng.randrange(0, batch // 3 + 1),
                    room=rng.choice([1.0, 0.6, 1.5]))
        case["grow_hi"] = min(case["grow_hi"], 8192)
    elif op == "rope":
        dim = rng.choice([64, 80, 128, 192, 256])
        case.update(rows=_log_int(rng, 1, 16384), kv_heads=rng.choice([1, 2, 4, 8]), dim=dim,
                    rot=rng.choice([dim, dim // 2 // 16 * 16, 32]), interleaved=rng.random() < 0.5,
                    base=rng.choice([10000.0, 500000.0]), factor=rng.choice([1.0, 4.0, 40.0]),
                    reach=_log_int(rng, 1000, 1 << 24))
        case["heads"] = case["kv_heads"] * rng.choice([1, 4, 5, 8, 16])
        del case["len_seed"]
    elif op == "prompt":
        hi = _log_int(rng, 1, 16384)
        dim, vdim = rng.choice([(64, 64), (128, 128), (128, 128), (192, 128)])
        kv_heads = rng.choice([1, 2, 4, 8, 16])
        case.update(batch=_log_int(rng, 1, max(1, min(64, 32768 // hi))), hi=hi,
                    lo=max(1, hi // rng.choice([1, 2, 16])), ctx=rng.choice([0, 0, _log_int(rng, 1, 16384)]),
                    kv_heads=kv_heads, heads=kv_heads * rng.choice([1, 2, 4, 5, 7, 8, 16]), dim=dim, vdim=vdim,
                    causal=rng.random() < 0.8)
    elif op == "cache":
        qlen = _log_int(rng, 1, 4000)
        batch = min(64, _log_int(rng, 1, max(1, 20000 // qlen)))
        case.update(batch=batch, qlen=qlen, lo=qlen, hi=qlen + rng.randrange(1, 4096),
                    kv_heads=rng.choice([1, 2, 4, 8]), dim=rng.choice([64, 128]))
    else:
        hi = _log_int(rng, 64, 65536)
        kv_heads = rng.choice([1, 2, 4, 8, 16])
        case.update(batch=_log_int(rng, 1, max(1, min(64, (1 << 20) // hi))), qlen=rng.choice([1, 1, 2, 4]), hi=hi,
                    lo=max(4, hi // rng.choice([1, 2, 16])), kv_heads=kv_heads,
                    heads=kv_heads * rng.choice([1, 2, 4, 5, 8, 16]), dim=rng.choice([64, 128]))
    most = [work(c) for c in listed() if c["op"] == op]
    while any(work(case)[n] > max(w[n] for w in most) for n in ("bytes", "flops")):
        if case.get("batch", 1) > 1:
            case["batch"] = (case["batch"] + 1) // 2
            case["finish"] = min(case.get("finish", 0), case["batch"])
        elif op == "rope":
            case["rows"] = (case["rows"] + 1) // 2
        elif case.get("ctx"):
            case["ctx"] //= 2
        else:
            case["hi"] = max(1, case["hi"] // 2)
            case["lo"] = min(case["lo"], case["hi"])
            if "grow_hi" in case:
                case["grow_hi"] = max(1, case["grow_hi"] // 2)
    return case


# ------------------------------------------------------------------ sizes that follow from a case


def _lengths(case):
    """Tokens of each sequence: before the step (plan), new (prompt), with the new ones (else)."""
    r, lo, hi = random.Random(case["len_seed"]), case["lo"], case["hi"]
    return [min(hi, max(lo, _log_int(r, max(lo, 1), hi))) if r.random() < 0.95 else lo for _ in range(case["batch"])]


def _targets(case):
    """Lengths that a plan's requests are to have; the first `finish` of a shuffle have finished."""
    r = random.Random(case["len_seed"] + 1)
    done = set(r.sample(range(case["batch"]), case["finish"]))
    return [0 if b in done else n + _log_int(r, case["grow_lo"], case["grow_hi"])
            for b, n in enumerate(_lengths(case))]


def _local(g, rank, dcp, inter):
    """Local length on a rank of a sequence of g tokens."""
    span = dcp * inter
    return g // span * inter + min(max(g % span - rank * inter, 0), inter)


def _blocks(g, case):
    return -(-_local(g, 0, case["dcp"], case["interleave"]) // case["block"])


def _bound(case):
    top = case["hi"] + (case["grow_hi"] if case["op"] == "plan" else 0)
    return max(1, _local(top, 0, case["dcp"], case["interleave"]))


def _row_bytes(case):
    n = case["kv_heads"] * case["dim"]
    return (n // 2 + n // 16 + 15) // 16 * 16


def _pairs(case):
    """(query, key) pairs that a prompt's rows see, per head."""
    c = case["ctx"]
    return sum(n * c + n * (n + 1) // 2 if case["causal"] else n * (n + c) for n in _lengths(case))


def work(case):
    op = case["op"]
    if op == "plan":
        old, new = _lengths(case), _targets(case)
        rows = sum(max(0, b - a) for a, b in zip(old, new))
        moved = sum(abs(_blocks(b, case) - _blocks(a, case)) for a, b in zip(old, new))
        return dict(bytes=4 * ((case["dcp"] + 1) * rows + 2 * moved + 4 * case["batch"]), flops=0)
    if op == "rope":
        n = case["rows"] * (case["heads"] + case["kv_heads"])
        return dict(bytes=n * case["dim"] * 4 + 4 * case["rows"], flops=3 * n * case["rot"])
    if op == "prompt":
        rows = sum(_lengths(case))
        keys = rows + case["batch"] * case["ctx"]
        d, v = case["dim"], case["vdim"]
        return dict(bytes=rows * case["heads"] * (2 * d + 2 * v + 4) + keys * case["kv_heads"] * 2 * (d + v),
                    flops=2 * (d + v) * case["heads"] * _pairs(case))
    n = case["kv_heads"] * case["dim"]
    rows = case["batch"] * case["qlen"]
    if op == "cache":
        return dict(bytes=rows * 2 * (4 * n + 2 * (n // 2 + n // 16)), flops=0)
    tokens = sum(_lengths(case))
    return dict(bytes=tokens * 2 * (n // 2 + n // 16) + rows * case["heads"] * (4 * case["dim"] + 4),
                flops=4 * case["qlen"] * tokens * case["heads"] * case["dim"])


# ------------------------------------------------------------------ inputs


def _normal(shape, gen):
    return torch.randn(*shape, generator=gen, device="cuda").bfloat16()


def _key_scale():
    return 6.0 / (448.0 * 6.0)  # six standard deviations reach the largest code of the largest block scale


def _tables(case, gen):
    """Shuffled blocks of every sequence, at the bound: [batch][blocks]."""
    per = -(-_bound(case) // case["block"])
    total = case["batch"] * per + 8
    perm = torch.randperm(total, generator=gen, device="cuda").to(torch.int32)
    return per, total, perm[:case["batch"] * per].view(case["batch"], per).contiguous()


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = dict(case=case)
    return {"plan": _prepare_plan, "rope": _prepare_rope, "prompt": _prepare_prompt,
            "cache": _prepare_pools, "decode": _prepare_pools}[case["op"]](case, s, gen)


def _prepare_plan(case, s, gen):
    old, new = _lengths(case), _targets(case)
    held = [_blocks(n, case) for n in old]
    need = sum(max(0, _blocks(b, case) - h) for b, h in zip(new, held))
    freed = sum(max(0, h - _blocks(b, case)) for b, h in zip(new, held))
    free = max(0, math.ceil(need * case["room"]) - freed) + (8 if case["room"] >= 1 else 0)
    per = -(-_bound(case) // case["block"])
    total = sum(held) + free
    perm = torch.randperm(max(total, 1), generator=gen, device="cuda").to(torch.int32)
    count = torch.tensor(held, device="cuda")
    at = torch.arange(per, device="cuda") < count[:, None]
    first = (count.cumsum(0) - count)[:, None] + torch.arange(per, device="cuda")
    s["table"] = torch.where(at, perm[first.clamp(max=max(total, 1) - 1)], -1).contiguous()
    s["free"] = torch.full((max(total, 1),), -1, dtype=torch.int32, device="cuda")
    s["free"][:free] = perm[sum(held):]
    s["count"] = torch.tensor([free], dtype=torch.int32, device="cuda")
    s["lens"] = torch.tensor(old, dtype=torch.int32, device="cuda")
    s["targets"] = torch.tensor(new, dtype=torch.int32, device="cuda")
    rows = sum(max(0, b - a) for a, b in zip(old, new))
    # the static bound on a step's rows, which a captured graph is made for
    s.update(blocks=per, num_blocks=max(total, 1), rows=rows + rows // 16 + 1)
    return s


def _prepare_rope(case, s, gen):
    T, H, K, d = case["rows"], case["heads"], case["kv_heads"], case["dim"]
    if case.get("latent"):
        # q's rotary part stands behind 128 other dims of a projection's rows, k's behind the
        # latent's 512; q goes to the rows that the absorbed attention reads
        s["q"] = _normal((T, H, 192), gen)[..., 128:]
        s["k"] = _normal((T, K, 576), gen)[..., 512:]
        s["q_out"] = torch.zeros(T, H, 576, dtype=torch.bfloat16, device="cuda")[..., 512:]
    else:
        s["q"], s["k"] = _normal((T, H, d), gen), _normal((T, K, d), gen)
        s["q_out"] = torch.empty_like(s["q"])
    s["k_out"] = torch.empty(T, K, d, dtype=torch.bfloat16, device="cuda")
    s["positions"] = torch.randint(0, case["reach"], (T,), generator=gen, device="cuda", dtype=torch.int32)
    return s


def _prepare_prompt(case, s, gen):
    lens, H, K = _lengths(case), case["heads"], case["kv_heads"]
    keys = [n + case["ctx"] for n in lens]
    s["q"] = _normal((sum(lens), H, case["dim"]), gen)
    if case["dim"] != case["vdim"]:
        # a latent projection's rows: 128 dims of k beside v's, and k put together with its rotary part
        both = _normal((sum(keys), K, 128 + case["vdim"]), gen)
        rot = _normal((sum(keys), 1, case["dim"] - 128), gen).expand(-1, K, -1)
        s["k"], s["v"] = torch.cat([both[..., :128], rot], -1), both[..., 128:]
    else:
        s["k"], s["v"] = _normal((sum(keys), K, case["dim"]), gen), _normal((sum(keys), K, case["vdim"]), gen)
    for name, n in (("cu_q", lens), ("cu_k", keys)):
        at = [0]
        for x in n:
            at.append(at[-1] + x)
        s[name + "_host"] = at
        s[name] = torch.tensor(at, dtype=torch.int32, device="cuda")
    s["scale"] = case["dim"] ** -0.5
    return s


def _prepare_pools(case, s, gen):
    W, bs, B, K, d = case["dcp"], case["block"], case["batch"], case["kv_heads"], case["dim"]
    per, NB, table = _tables(case, gen)
    s.update(blocks=per, num_blocks=NB, table=table,
             lens=torch.tensor(_lengths(case), dtype=torch.int32, device="cuda"),
             k_scale=torch.tensor([_key_scale()], device="cuda"),
             v_scale=torch.tensor([MID * _key_scale()], device="cuda"))
    rows = W * NB * bs
    for name in ("k", "v"):
        pool = torch.empty(rows, _row_bytes(case), dtype=torch.uint8, device="cuda")
        step = max(1, (1 << 26) // (K * d))
        for i in range(0, rows, step):
            n = min(step, rows - i)
            x = torch.randn(n, K * d, generator=gen, device="cuda").bfloat16()
            pool[i:i + n] = _encode(x, s[name + "_scale"], _row_bytes(case))
        s[name] = pool.view(W, NB, bs, -1)
    R = B * case["qlen"]
    if case["op"] == "decode":
        s["q"] = _normal((R, case["heads"], d), gen)
        return s
    s["k_new"], s["v_new"] = _normal((R, K, d), gen), _normal((R, K, d), gen)
    # the step's plan: slots (one rank's row, -1 on the others), first positions, row offsets
    s["begins"] = (s["lens"] - case["qlen"]).contiguous()
    s["cu"] = torch.arange(B + 1, dtype=torch.int32, device="cuda") * case["qlen"]
    pos = s["begins"].long()[:, None] + torch.arange(case["qlen"], device="cuda")
    rank, local = _place(pos, case)
    slot = table.long().gather(1, local // bs) * bs + local % bs
    mine = rank[None] == torch.arange(W, device="cuda")[:, None, None]
    s["slots"] = torch.where(mine, slot[None], -1).to(torch.int32).view(W, R).contiguous()
    return s


# ------------------------------------------------------------------ the plain forms


def _place(pos, case):
    """(rank, local index) of global positions."""
    inter, W = case["interleave"], case["dcp"]
    return pos // inter % W, pos // (inter * W) * inter + pos % inter


def _local0(g, case):
    inter = case["interleave"]
    span = case["dcp"] * inter
    return g // span * inter + (g % span).clamp(max=inter)


def _plain_plan(s):
    case, bs, ML = s["case"], s["case"]["block"], _bound(s["case"])
    B, MB, W = case["batch"], s["blocks"], case["dcp"]
    old, new = s["lens"].long(), s["targets"].long()
    dev = old.device
    ok = (new >= 0) & (old >= 0) & (_local0(new.clamp(min=0), case) <= ML) & (_local0(old.clamp(min=0), case) <= ML)
    held, want = -(-_local0(old, case) // bs), -(-_local0(new.clamp(min=0), case) // bs)
    rows = torch.where(ok, (new - old).clamp(min=0), 0)
    need = torch.where(ok, (want - held).clamp(min=0), 0)
    freed = torch.where(ok, (held - want).clamp(min=0), 0)
    F, count = freed.sum(), s["count"].long()[0]
    fits = (need.cumsum(0) <= count + F) & (rows.cumsum(0) <= s["rows"])
    grant = (rows > 0) & fits
    lens = torch.where(ok & (grant | (new <= old)), new, old)
    rows, need = torch.where(grant, rows, 0), torch.where(grant, need, 0)
    used = need.sum()
    # freed blocks, in the order of their requests: the first ones are handed out first
    NB = s["num_blocks"]
    i = torch.arange(NB, device=dev)
    freed_end = freed.cumsum(0)
    b = torch.searchsorted(freed_end, i, right=True).clamp(max=B - 1)
    back = s["table"].view(-1)[(b * MB + want[b] + i - (freed_end - freed)[b]).clamp(0, B * MB - 1)]
    # the blocks of the growing requests: freed ones, then the free list's from its end
    need_end = need.cumsum(0)
    j = torch.arange(MB, device=dev)
    nth = (need_end - need)[:, None] + j - held[:, None]
    given = torch.where(nth < F, back[nth.clamp(0, NB - 1)], s["free"][(count - 1 - (nth - F)).clamp(0, NB - 1)])
    takes = grant[:, None] & (j >= held[:, None]) & (j < want[:, None])
    table = torch.where(takes, given, s["table"])
    left = F - used  # what is not handed out goes on top of the list, the last first
    free = torch.where((i >= count) & (i < count + left), back[(F - 1 - (i - count)).clamp(0, NB - 1)], s["free"])
    # rows of the step
    ends = rows.cumsum(0)
    t = torch.arange(s["rows"], device=dev)
    b = torch.searchsorted(ends, t, right=True).clamp(max=B - 1)
    live = t < ends[-1]
    pos = torch.where(live, old[b] + t - (ends - rows)[b], 0)
    rank, local = _place(pos, case)
    slot = table.view(-1)[(b * MB + (local // bs).clamp(max=MB - 1))].long() * bs + local % bs
    mine = live & (rank == torch.arange(W, device=dev)[:, None])
    s["table"].copy_(table)
    s["free"].copy_(free)
    return dict(lens=lens.to(torch.int32), count=(count + left).to(torch.int32).view(1), table=s["table"],
                free=s["free"], slots=torch.where(mine, slot, -1).to(torch.int32), positions=pos.to(torch.int32),
                cu=torch.cat([ends.new_zeros(1), ends]).to(torch.int32))


def _frequencies(case):
    """Radians per position of each pair, in 64 bits, and the factor on cosine and sine."""
    n, factor = case["rot"] // 2, case["factor"]
    plain = [case["base"] ** (-i / n) for i in range(n)]
    if factor == 1.0:
        return plain, 1.0
    # scaled by parts: pairs that turn often within the original 4096 positions stay, slow ones
    # are stretched, a ramp between 32 turns and one
    def turn_pair(turns):
        return n * math.log(4096 / (turns * 2 * math.pi)) / math.log(case["base"])
    lo, hi = max(0.0, math.floor(turn_pair(32.0))), min(n - 1.0, math.ceil(turn_pair(1.0)))
    ramp = [min(1.0, max(0.0, (i - lo) / max(hi - lo, 0.001))) for i in range(n)]
    return [f * (1 - r) + f / factor * r for f, r in zip(plain, ramp)], 0.1 * math.log(factor) + 1.0


def _plain_rope(s):
    case = s["case"]
    rot, n = case["rot"], case["rot"] // 2
    freq, amp = _frequencies(case)
    angle = s["positions"].double()[:, None] * torch.tensor(freq, dtype=torch.float64, device="cuda")
    cos, sin = (amp * angle.cos()).float()[:, None], (amp * angle.sin()).float()[:, None]
    done = []
    for x, out in ((s["q"], s["q_out"]), (s["k"], s["k_out"])):
        y = x.float()
        a, b = (y[..., 0:rot:2], y[..., 1:rot:2]) if case["interleaved"] else (y[..., :n], y[..., n:rot])
        turned = (a * cos - b * sin, b * cos + a * sin)
        part = torch.stack(turned, -1).flatten(-2) if case["interleaved"] else torch.cat(turned, -1)
        out.copy_(torch.cat([part, y[..., rot:]], -1))
        done.append(out)
    return tuple(done)


def _plain_prompt(s):
    case = s["case"]
    H, K, d, v = case["heads"], case["kv_heads"], case["dim"], case["vdim"]
    group = H // K
    out = torch.zeros(s["q"].shape[0], H, v, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((s["q"].shape[0], H), -math.inf, device="cuda")
    for b in range(case["batch"]):
        q0, q1, k0, k1 = *s["cu_q_host"][b:b + 2], *s["cu_k_host"][b:b + 2]
        n, m = q1 - q0, k1 - k0
        heads = max(1, min(K, (1 << 29) // (group * m * min(n, 512))))
        for r0 in range(0, n, 512):
            r1 = min(n, r0 + 512)
            end = m - n + r1 if case["causal"] else m
            seen = torch.arange(end, device="cuda") <= (
                torch.arange(r0, r1, device="cuda")[:, None] + (m - n) if case["causal"] else m)
            for h in range(0, K, heads):
                of = slice(h, min(K, h + heads))
                k = s["k"][k0:k0 + end, of].float().permute(1, 2, 0)
                val = s["v"][k0:k0 + end, of].float().permute(1, 0, 2)
                q = s["q"][q0 + r0:q0 + r1, h * group:of.stop * group].float()
                q = q.view(r1 - r0, -1, group, d).permute(1, 2, 0, 3).reshape(-1, group * (r1 - r0), d)
                x = ((q @ k) * s["scale"]).view(-1, group, r1 - r0, end)
                x.masked_fill_(~seen, -math.inf)
                top = x.amax(-1, keepdim=True)
                x.sub_(top).exp_()
                total = x.sum(-1, keepdim=True)
                o = (x.view(q.shape[0], -1, end) @ val).view(-1, group, r1 - r0, v) / total
                at = slice(q0 + r0, q0 + r1)
                out[at, h * group:of.stop * group] = o.permute(2, 0, 1, 3).reshape(r1 - r0, -1, v).bfloat16()
                lse[at, h * group:of.stop * group] = (top + total.log()).squeeze(-1).permute(2, 0, 1).reshape(r1 - r0, -1)
    return dict(out=out, lse=lse)


_STEPS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _encode(x, scale, row_bytes):
    """Rows of the pool: two codes to a byte, the first in the low half; then the block scales."""
    x = x.float().view(x.shape[0], -1, 16)
    block = (x.abs().amax(-1) / (6.0 * scale)).clamp(max=448.0).to(torch.float8_e4m3fn)
    step = scale * block.float()
    y = torch.where(step[..., None] > 0, x / torch.where(step > 0, step, 1.0)[..., None], 0.0).abs()
    # to the nearest of eight magnitudes, ties to the even code
    code = sum((y >= t if up else y > t).to(torch.uint8) for t, up in
               ((0.25, 0), (0.75, 1), (1.25, 0), (1.75, 1), (2.5, 0), (3.5, 1), (5.0, 0)))
    code = (code | (torch.signbit(x).to(torch.uint8) << 3)).view(x.shape[0], -1, 2)
    out = torch.zeros(x.shape[0], row_bytes, dtype=torch.uint8, device=x.device)
    n = code.shape[1]
    out[:, :n] = code[..., 0] | (code[..., 1] << 4)
    out[:, n:n + block.shape[1]] = block.view(torch.uint8)
    return out


def _decoded(rows, n, scale):
    """Values of pool rows [..., row_bytes] -> float [..., n]."""
    code = torch.stack([rows[..., :n // 2] & 15, rows[..., :n // 2] >> 4], -1).flatten(-2)
    value = torch.tensor(_STEPS + tuple(-x for x in _STEPS), device=rows.device)[code.int()]
    block = rows[..., n // 2:n // 2 + n // 16].contiguous().view(torch.float8_e4m3fn).float()
    return (value.unflatten(-1, (-1, 16)) * block[..., None]).flatten(-2) * scale


def _plain_cache(s):
    case = s["case"]
    W, K, d, bs = case["dcp"], case["kv_heads"], case["dim"], case["block"]
    rank, row = torch.nonzero(s["slots"] >= 0, as_tuple=True)
    at = s["slots"][rank, row].long()
    pos = s["begins"].long()[:, None] + torch.arange(case["qlen"], device="cuda")
    r, local = _place(pos, case)
    slot = s["table"].long().gather(1, local // bs) * bs + local % bs
    done = []
    for name in ("k", "v"):
        scale = s[name + "_scale"]
        pool = s[name].view(W, -1, _row_bytes(case))
        pool[rank, at] = _encode(s[name + "_new"][row].flatten(1), scale, _row_bytes(case))
        done.append(_decoded(pool[r, slot], K * d, scale).bfloat16().view(-1, K, d))
    return tuple(done)


def _plain_decode(s):
    case = s["case"]
    W, B, n, K, d = case["dcp"], case["batch"], case["qlen"], case["kv_heads"], case["dim"]
    group, ML, bs = case["heads"] // K, _bound(case), case["block"]
    t = torch.arange(ML, device="cuda")
    rank = torch.arange(W, device="cuda")[:, None]
    inter = case["interleave"]
    # global position of every (rank, local index): what the rows see is decided by it
    pos = (t // inter * W + rank) * inter + t % inter  # [W][ML]
    out = torch.zeros(B * n, case["heads"], d, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(B * n, case["heads"], device="cuda")
    for b in range(B):
        rows = s["table"][b].long()[t // bs] * bs + t % bs
        k, v = (_decoded(s[x].view(W, -1, _row_bytes(case))[:, rows], K * d, s[x + "_scale"]).view(W * ML, K, d)
                .permute(1, 0, 2) for x in ("k", "v"))
        q = s["q"][b * n:(b + 1) * n].float().view(n, K, group, d).permute(1, 0, 2, 3).reshape(K, n * group, d)
        x = ((q @ k.transpose(1, 2)) * d ** -0.5).view(K, n, group, W * ML)
        end = s["lens"][b].long() - n + 1 + torch.arange(n, device="cuda")
        x.masked_fill_(~(pos.view(-1) < end[:, None])[:, None], -math.inf)
        top = x.amax(-1, keepdim=True)
        x = torch.exp(x - torch.where(top == -math.inf, 0.0, top))
        total = x.sum(-1, keepdim=True)
        o = (x.view(K, n * group, -1) @ v).view(K, n, group, d)
        o = torch.where(total > 0, o / total, 0.0)
        out[b * n:(b + 1) * n] = o.permute(1, 0, 2, 3).reshape(n, -1, d).bfloat16()
        lse[b * n:(b + 1) * n] = (top + torch.log(total)).squeeze(-1).permute(1, 0, 2).reshape(n, -1)
    return dict(out=out, lse=lse)


# ------------------------------------------------------------------ the framework's calls


def _handle(s):
    """What a program builds once for its shapes and keeps: dims, plans and buffers."""
    import decode_context_mla_causal_gb300 as dm

    if "handle" in s:
        return s["handle"]
    case = s["case"]
    op = case["op"]
    if op == "rope":
        scaling = None if case["factor"] == 1.0 else dict(kind="yarn", factor=case["factor"], original_len=4096)
        h, dims = dm.Rope(case["rot"], base=case["base"], interleaved=case["interleaved"], scaling=scaling), None
    elif op == "prompt":
        h = dm.PromptAttention(case["heads"], case["kv_heads"], case["dim"], case["vdim"],
                               max_rows=s["q"].shape[0], max_seqs=case["batch"], causal=case["causal"])
        dims = None
    else:
        dims = dm.make_dims(batch=case["batch"], qlen=case.get("qlen", 1), num_heads=case.get("heads", 1),
                            dcp=case["dcp"], interleave=case["interleave"], block_size=case["block"],
                            max_blocks_per_seq=s["blocks"], max_local_len=_bound(case),
                            num_blocks=s["num_blocks"], num_splits=1)
        if op == "plan":
            h = dm.PagePlan(dims, s["rows"])
        elif op == "cache":
            h = dict(status=torch.zeros(1, dtype=torch.int32, device="cuda"),
                     k=torch.empty_like(s["k_new"]), v=torch.empty_like(s["v_new"]))
        else:
            h = dm.GqaDecode(dims, case["kv_heads"], case["dim"], dm.KV_NVFP4)
    s["handle"] = (dm, dims, h)
    return s["handle"]


def _own(s):
    dm, dims, h = _handle(s)
    case = s["case"]
    op = case["op"]
    if op == "plan":
        h(s["targets"], s["lens"], s["table"], s["free"], s["count"], new_lens=h.new_lens, new_count=h.new_count)
        return dict(lens=h.new_lens, count=h.new_count, table=s["table"], free=s["free"], slots=h.slot_mapping,
                    positions=h.positions, cu=h.cu_rows)
    if op == "rope":
        return h(s["positions"], s["q"], s["k"], out_q=s["q_out"], out_k=s["k_out"])
    if op == "prompt":
        out, lse = h(s["q"], s["k"], s["v"], s["cu_q"], s["cu_k"], s["scale"])
        return dict(out=out, lse=lse)
    if op == "cache":
        dm.dcp_gqa_kv_write(dims, case["kv_heads"], case["dim"], s["slots"], s["k_new"], s["v_new"], dm.KV_NVFP4,
                            s["k_scale"], s["v_scale"], case["dcp"], s["k"], s["v"], h["status"])
        dm.dcp_gqa_kv_gather(dims, case["kv_heads"], case["dim"], s["begins"], s["cu"], s["table"], s["k"], s["v"],
                             dm.KV_NVFP4, s["k_scale"], s["v_scale"], 0, case["dcp"], h["k"], h["v"], h["status"])
        return h["k"], h["v"]
    out, lse = h(s["q"], s["k"], s["v"], s["k_scale"], s["v_scale"], case["dim"] ** -0.5, s["lens"], s["table"])
    return dict(out=out, lse=lse)


def run(state):
    if own:
        return _own(state)
    return {"plan": _plain_plan, "rope": _plain_rope, "prompt": _plain_prompt, "cache": _plain_cache,
            "decode": _plain_decode}[state["case"]["op"]](state)


# ------------------------------------------------------------------ 64-bit values


def exact(case, seed):
    if case["op"] == "plan":
        return None  # whole numbers
    if case["op"] in ("prompt", "decode") and work(case)["flops"] > 3e12:
        return None
    s = prepare(case, seed)
    return {"rope": _exact_rope, "prompt": _exact_prompt, "cache": _exact_cache, "decode": _exact_decode}[case["op"]](s)


def _exact_rope(s):
    """Each pair as a complex number times e^(i angle)."""
    case = s["case"]
    rot = case["rot"]
    freq, amp = _frequencies(case)
    turn = torch.polar(torch.tensor(amp, dtype=torch.float64, device="cuda"), s["positions"].double()[:, None, None]
                       * torch.tensor(freq, dtype=torch.float64, device="cuda"))
    done = []
    for x in (s["q"], s["k"]):
        y = x.double().clone()
        pairs = (y[..., :rot].unflatten(-1, (-1, 2)) if case["interleaved"]
                 else y[..., :rot].unflatten(-1, (2, -1)).transpose(-1, -2))
        z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
        y[..., :rot] = (z if case["interleaved"] else z.transpose(-1, -2)).flatten(-2)
        done.append(y)
    return tuple(done)


def _exact_prompt(s):
    case = s["case"]
    group = case["heads"] // case["kv_heads"]
    T = s["q"].shape[0]
    out = torch.zeros(T, case["heads"], case["vdim"], dtype=torch.float64, device="cuda")
    lse = torch.full((T, case["heads"]), -math.inf, dtype=torch.float64, device="cuda")
    for b in range(case["batch"]):
        q0, q1 = s["cu_q_host"][b], s["cu_q_host"][b + 1]
        k0, k1 = s["cu_k_host"][b], s["cu_k_host"][b + 1]
        n, m = q1 - q0, k1 - k0
        for h in range(case["heads"]):
            k, v = s["k"][k0:k1, h // group].double(), s["v"][k0:k1, h // group].double()
            for r0 in range(0, n, 4096):
                r1 = min(n, r0 + 4096)
                end = r1 + m - n if case["causal"] else m
                x = (s["q"][q0 + r0:q0 + r1, h].double() @ k[:end].T) * s["scale"]
                if case["causal"]:
                    x.masked_fill_(torch.ones_like(x, dtype=torch.bool).triu_(r0 + m - n + 1), -math.inf)
                lse[q0 + r0:q0 + r1, h] = x.logsumexp(1)
                out[q0 + r0:q0 + r1, h] = x.softmax(1) @ v[:end]
    return dict(out=out, lse=lse)


def _e4m3_values():
    held = [c / 8 * 2.0 ** -6 if c < 8 else (1 + c % 8 / 8) * 2.0 ** (c // 8 - 7) for c in range(127)]
    return torch.tensor(held, dtype=torch.float64, device="cuda")


def _nearest(x, held):
    """The nearest of ascending magnitudes, ties to an even index; beyond the last, the last."""
    mag = x.abs().clamp(max=float(held[-1]))
    hi = torch.searchsorted(held, mag).clamp(max=len(held) - 1)
    lo = (hi - 1).clamp(min=0)
    up, down = held[hi] - mag, mag - held[lo]
    return held[torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)] * x.sign()


def _exact_cache(s):
    case = s["case"]
    done = []
    for name in ("k", "v"):
        x = s[name + "_new"].double().unflatten(-1, (-1, 16))
        scale = s[name + "_scale"]
        # the definition divides in 32 bits
        most = (x.abs().amax(-1, keepdim=True).float() / (6.0 * scale)).double()
        step = (_nearest(most, _e4m3_values()).float() * scale)
        code = torch.where(step > 0, x.float() / step, 0.0).double()
        value = _nearest(code, torch.tensor(_STEPS, dtype=torch.float64, device="cuda"))
        done.append((value * _nearest(most, _e4m3_values()) * scale.double()).flatten(-2).view(-1, case["kv_heads"], case["dim"]))
    return tuple(done)


def _exact_decode(s):
    case = s["case"]
    W, bs, K, d, H, n = case["dcp"], case["block"], case["kv_heads"], case["dim"], case["heads"], case["qlen"]
    out = torch.zeros(case["batch"] * n, H, d, dtype=torch.float64, device="cuda")
    lse = torch.full((case["batch"] * n, H), -math.inf, dtype=torch.float64, device="cuda")
    e4m3 = torch.cat([_e4m3_values(), torch.full((1,), math.nan, dtype=torch.float64, device="cuda")])
    magnitude = torch.tensor(_STEPS, dtype=torch.float64, device="cuda")
    for b in range(case["batch"]):
        p = torch.arange(int(s["lens"][b]), device="cuda")
        chunk = p // case["interleave"]
        local = chunk // W * case["interleave"] + p % case["interleave"]
        got = []
        for name in ("k", "v"):
            row = s[name][chunk % W, s["table"][b].long()[local // bs], local % bs].int()
            i = torch.arange(K * d, device="cuda")
            code = row[:, i // 2] >> (4 * (i % 2)) & 15
            got.append((magnitude[code & 7] * (1.0 - 2.0 * (code >> 3)) * e4m3[row[:, K * d // 2 + i // 16]]
                        * float(s[name + "_scale"])).view(-1, K, d))
        for j in range(n):
            end = len(p) - n + 1 + j
            if end < 1:
                continue
            for g in range(K):
                of = slice(g * (H // K), (g + 1) * (H // K))
                x = (s["q"][b * n + j, of].double() @ got[0][:end, g].T) * d ** -0.5
                lse[b * n + j, of] = x.logsumexp(1)
                out[b * n + j, of] = x.softmax(1) @ got[1][:end, g]
    return dict(out=out, lse=lse)
