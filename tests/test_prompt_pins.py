"""Pins of the page, rotary, prompt and 4-bit oracles against something other than themselves:
complex numbers, plain softmax, counting, closed forms and invariants."""

import random

import numpy as np
import pytest

from oracle import evict, fp4, fp8, gqa, kv_write, metadata, pages, prompt

RNG = np.random.default_rng


def _bits(x):
    return (np.asarray(x, np.float32).view(np.uint32) >> 16).astype(np.uint16)


# ------------------------------------------------------------------ 4 bits


def test_e2m1_codes_are_their_values():
    for code in range(16):
        x = fp4.MAGNITUDES[code & 7] * (-1 if code & 8 else 1)
        assert fp4.encode_e2m1(np.array([x]))[0] == code or x == 0
    # halfway goes to the even code, beyond the largest to it
    ties = {0.25: 0, 0.75: 2, 1.25: 2, 1.75: 4, 2.5: 4, 3.5: 6, 5.0: 6, 5.0001: 7, 1e30: 7}
    for x, code in ties.items():
        assert fp4.encode_e2m1(np.array([x, -x])).tolist() == [code, code | 8], x


def test_a_row_of_exact_values_survives():
    # values that are scale * block * code exactly come back as they are
    rng = RNG(1)
    code = rng.integers(0, 16, (5, 64))
    code[:, ::16] = 7  # the largest of each block, so that the block scale is found again
    block = rng.choice([0.5, 1.0, 2.0, 16.0], (5, 4))
    x = fp4.MAGNITUDES[code & 7] * np.where(code & 8, -1.0, 1.0) * np.repeat(block, 16, 1) * 0.25
    rows = fp4.quantize_rows(_bits(x), 0.25)
    assert rows.shape == (5, fp4.row_bytes(64)) == (5, 48)
    assert np.array_equal(0.25 * fp4.decode_rows(rows, 64), x)
    assert np.array_equal(fp8.decode_e4m3(rows[:, 32:36]), block)


def test_quantised_values_are_near():
    # a step of E2M1 is at most a third of the value above half of the block's largest: within a
    # sixth, and the block scale within 2^-4 of the one asked for
    x = RNG(2).standard_normal((50, 128))
    x = fp8.decode_bf16(_bits(x))
    got = fp4.decode_rows(fp4.quantize_rows(_bits(x), 0.003), 128) * np.float32(0.003)
    most = np.abs(x).reshape(50, 8, 16).max(-1).repeat(16).reshape(50, 128)
    assert (np.abs(got - x) <= most / 6 * (1 + 2.0 ** -4) + np.abs(x) * 2.0 ** -4).all()


# ------------------------------------------------------------------ pages


def _pool(lens, W, S, bs, bound, spare, seed):
    ML = evict.local_count(bound, 0, W, S)
    held = [-(-evict.local_count(n, 0, W, S) // bs) for n in lens]
    NB = sum(held) + spare
    perm = list(range(NB))
    random.Random(seed).shuffle(perm)
    table = np.full((len(lens), max(1, -(-ML // bs))), -1)
    for b, n in enumerate(held):
        table[b, :n], perm = perm[:n], perm[n:]
    free = np.full(NB, -1)
    free[:spare] = perm
    return dict(seq_lens=lens, block_table=table, free_list=free, free_count=spare, dcp=W, interleave=S, block_size=bs,
                max_local_len=ML, num_blocks=NB)


def test_slots_are_those_of_the_verify_write():
    # with the same number of new tokens for each, slots are the slot mapping's
    p = _pool([20, 33, 5], 3, 2, 4, 60, 30, 1)
    got = pages.plan(targets=[24, 37, 9], max_rows=12, **p)
    want, status = kv_write.slot_mapping(seq_lens=[24, 37, 9], block_table=got["block_table"], qlen=4, dcp=3,
                                         interleave=2, block_size=4, max_blocks_per_seq=got["block_table"].shape[1],
                                         num_blocks=p["num_blocks"])
    assert status == 0 and got["status"] == 0 and np.array_equal(got["slot_mapping"], want)
    assert got["positions"].tolist() == [20, 21, 22, 23, 33, 34, 35, 36, 5, 6, 7, 8]


def test_blocks_are_neither_lost_nor_given_twice():
    rng = random.Random(4)
    p = _pool([0] * 9, 2, 1, 4, 100, 60, 2)
    for _ in range(200):
        targets = [rng.choice([0, n, n + 1, rng.randrange(101)]) for n in p["seq_lens"]]
        targets = [min(t, 100) for t in targets]
        got = pages.plan(targets=targets, max_rows=rng.choice([5, 500]), **p)
        p.update(seq_lens=got["new_lens"].tolist(), block_table=got["block_table"], free_list=got["free_list"],
                 free_count=got["free_count"])
        held = [int(x) for b, n in enumerate(p["seq_lens"])
                for x in p["block_table"][b, : -(-evict.local_count(n, 0, 2, 1) // 4)]]
        assert sorted(held + p["free_list"][: p["free_count"]].tolist()) == list(range(60))


def test_growth_stops_at_the_first_that_does_not_fit():
    p = _pool([0, 0, 0, 8], 1, 1, 4, 40, 3, 3)
    got = pages.plan(targets=[8, 20, 4, 0], max_rows=100, **p)  # two blocks of 3 + 2, then five, then one
    assert got["new_lens"].tolist() == [8, 0, 0, 0] and got["status"] == pages.STATUS_HELD_BACK
    assert got["free_count"] == 3 and got["cu_rows"].tolist() == [0, 8, 8, 8, 8]


# ------------------------------------------------------------------ rotary positions and prompts


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_is_a_product_of_complex_numbers(interleaved):
    rng = RNG(5)
    x, pos = rng.standard_normal((6, 2, 40)), rng.integers(-1000, 1 << 20, 6)
    freq, amp = prompt.frequencies(32, 500.0, kind="yarn", factor=8.0, original_len=300)
    got = prompt.rotate(x, pos, freq, amp, interleaved)
    a, b = (x[..., 0:32:2], x[..., 1:32:2]) if interleaved else (x[..., :16], x[..., 16:32])
    z = (a + 1j * b) * amp * np.exp(1j * pos[:, None, None] * freq)
    want = np.stack([z.real, z.imag], -1).reshape(6, 2, 32) if interleaved else np.concatenate([z.real, z.imag], -1)
    assert np.allclose(got[..., :32], want) and np.array_equal(got[..., 32:], x[..., 32:])


def test_scores_depend_on_distance_alone():
    rng = RNG(6)
    freq, amp = prompt.frequencies(64, 10000.0)
    q, k = rng.standard_normal((1, 1, 64)), rng.standard_normal((1, 1, 64))
    def score(i, j):
        return float((prompt.rotate(q, [i], freq, amp, False) * prompt.rotate(k, [j], freq, amp, False)).sum())
    assert np.isclose(score(70, 20), score(5050, 5000)) and not np.isclose(score(70, 20), score(70, 21))


def test_scaled_by_parts_keeps_fast_pairs_and_stretches_slow_ones():
    plain, _ = prompt.frequencies(128, 10000.0)
    got, amp = prompt.frequencies(128, 10000.0, kind="yarn", factor=16.0, original_len=4096)
    turns = plain * 4096 / (2 * np.pi)
    assert np.allclose(got[turns > 40], plain[turns > 40]) and np.allclose(got[turns < 0.8], plain[turns < 0.8] / 16)
    assert (got <= plain * (1 + 1e-12)).all() and (np.diff(got) < 0).all() and np.isclose(amp, 0.1 * np.log(16) + 1)


def test_prompt_is_causal_softmax():
    rng = RNG(7)
    q, k, v = rng.standard_normal((9, 4, 8)), rng.standard_normal((14, 2, 8)), rng.standard_normal((14, 2, 6))
    got = prompt.attend(q=q, k=k, v=v, cu_q=[0, 5, 9], cu_k=[0, 3, 14], softmax_scale=0.3)
    # five rows over three keys: the first two see none; four rows behind seven keys
    assert np.isneginf(got["lse"][:2]).all() and (got["out"][:2] == 0).all()
    for row, first, seen in ((2, 0, 1), (4, 0, 3), (5, 3, 8), (8, 3, 11)):
        for h in range(4):
            s = 0.3 * k[first:first + seen, h // 2] @ q[row, h]
            assert np.isclose(got["lse"][row, h], np.log(np.exp(s).sum()))
            assert np.allclose(got["out"][row, h], np.exp(s) @ v[first:first + seen, h // 2] / np.exp(s).sum())


def test_a_prompt_s_last_row_is_its_decode():
    # the newest token's row over the cache is the prompt's last row
    rng = RNG(8)
    n, W, S, bs = 23, 2, 1, 4
    k, v = (fp8.decode_bf16(_bits(rng.standard_normal((n, 2, 64)))) for _ in range(2))
    table = rng.permutation(6)[:4][None]
    pools = [np.zeros((W, 6, bs, 2, 64)) for _ in range(2)]
    p = np.arange(n)
    li = metadata.local_index(p, W, S)
    for pool, x in zip(pools, (k, v)):
        pool[metadata.owner(p, W, S), table[0][li // bs], li % bs] = x
    q = rng.standard_normal((n, 6, 64))
    whole = prompt.attend(q=q, k=k, v=v, cu_q=[0, n], cu_k=[0, n], softmax_scale=0.2)
    last = gqa.decode(q=q[-1:], k_pools=pools[0], v_pools=pools[1], block_table=table, seq_lens=[n], qlen=1, dcp=W,
                      interleave=S, block_size=bs, kv_dtype="values", k_scale=1.0, v_scale=1.0, softmax_scale=0.2)
    assert np.allclose(whole["out"][-1:], last["out"]) and np.allclose(whole["lse"][-1:], last["lse"])


SLOW_ENDS = [  # rot_dim, base, original_len, beta_fast, beta_slow, ramp's ends worked out by hand
    # 32 ln(131072 / 64 pi) / ln 1e4 = 22.5 and 32 ln(131072 / 2 pi) / ln 1e4 = 34.6
    (64, 1e4, 131072.0, 32.0, 1.0, 22, 35),
    # 64 ln(65536 / 64 pi) / ln 1e4 = 40.2 and 64 ln(65536 / 2 pi) / ln 1e4 = 64.3
    (128, 1e4, 65536.0, 32.0, 1.0, 40, 65),
    # 8 ln(1e6 / 2e5 pi) / ln 100 = 0.8 and 8 ln(1e6 / 2 pi) / ln 100 = 20.8, beyond the last dim
    (16, 100.0, 1e6, 1e5, 1.0, 0, 15),
    # both ends behind the last pair: nothing is stretched
    (16, 10.0, 1e9, 32.0, 1.0, 53, 15),
]


@pytest.mark.parametrize("case", SLOW_ENDS, ids=str)
def test_scaled_by_parts_with_the_slow_end_behind_the_last_pair(case):
    rot, base, original, fast, slow, lo, hi = case
    got, _ = prompt.frequencies(rot, base, kind="yarn", factor=4.0, original_len=original, beta_fast=fast, beta_slow=slow)
    for i in range(rot // 2):
        plain = base ** (-2 * i / rot)
        r = 0.0 if i <= lo else (i - lo) / (hi - lo)  # never reaches 1
        assert 0.0 <= r < 1.0 and np.isclose(got[i], plain * (1 - r) + plain / 4 * r, rtol=1e-12), i


def test_a_block_with_an_infinity_or_nan_reads_as_nan():
    x = RNG(3).standard_normal((4, 48))
    bits = _bits(x)
    clean = fp4.quantize_rows(bits, 0.01)
    for row, (at, value) in enumerate(((0, 0x7F80), (17, 0xFF80), (47, 0x7FC1))):  # inf, -inf, nan
        bits[row, at] = value
    rows = fp4.quantize_rows(bits, 0.01)
    got, want = fp4.decode_rows(rows, 48).reshape(4, 3, 16), fp4.decode_rows(clean, 48).reshape(4, 3, 16)
    hit = np.zeros((4, 3), bool)
    hit[[0, 1, 2], [0, 1, 2]] = True
    assert np.isnan(got[hit]).all() and np.array_equal(got[~hit], want[~hit])
    assert (rows[0, 24:27] == [0x7F, *clean[0, 25:27]]).all() and not rows[0, :8].any()


def test_bad_ids_that_go_onto_the_list_are_noticed():
    for bad in (-1, 99):
        p = _pool([9, 5], 1, 1, 4, 40, 3, 3)
        p["block_table"][0, 2] = bad
        got = pages.plan(targets=[0, 6], max_rows=4, **p)
        assert got["status"] == metadata.STATUS_BAD_BLOCK_ID and bad in got["free_list"][: got["free_count"]]
        # an id that stays in its table is not looked at
        assert pages.plan(targets=[9, 6], max_rows=4, **p)["status"] == 0
