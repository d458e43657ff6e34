"""Pins of the grouped-head and eviction oracles against something other than themselves:
closed forms, the latent-cache oracle, counting, and invariants."""

import numpy as np
import pytest

from oracle import attention, evict, fp8, gqa

RNG = np.random.default_rng


def _pools(rng, W, NB, bs, *tail):
    return (rng.standard_normal((W, NB, bs, *tail)).astype(np.float32).view(np.uint32) >> 16).astype(np.uint16)


def _table(rng, B, MB, NB):
    return rng.permutation(NB)[: B * MB].reshape(B, MB)


def test_gqa_of_one_visible_token_is_its_value():
    rng = RNG(1)
    k, v = _pools(rng, 2, 6, 4, 2, 64), _pools(rng, 2, 6, 4, 2, 64)
    table = _table(rng, 1, 3, 6)
    q = rng.standard_normal((1, 6, 64))
    got = gqa.decode(q=q, k_pools=k, v_pools=v, block_table=table, seq_lens=[1], qlen=1, dcp=2,
                     interleave=1, block_size=4, kv_dtype="bf16", k_scale=1, v_scale=1, softmax_scale=0.3)
    for h in range(6):
        row = fp8.decode_bf16(v[0, table[0][0], 0, h // 3])
        assert np.allclose(got["out"][0, h], row)
        assert np.isclose(got["lse"][0, h], 0.3 * fp8.decode_bf16(k[0, table[0][0], 0, h // 3]) @ q[0, h])


def test_gqa_with_equal_keys_averages_the_values():
    rng = RNG(2)
    k = np.zeros((3, 9, 4, 1, 64), np.uint16)
    v = _pools(rng, 3, 9, 4, 1, 64)
    table = _table(rng, 1, 3, 9)
    got = gqa.decode(q=rng.standard_normal((2, 2, 64)), k_pools=k, v_pools=v, block_table=table,
                     seq_lens=[25], qlen=2, dcp=3, interleave=2, block_size=4, kv_dtype="bf16",
                     k_scale=1, v_scale=1, softmax_scale=1.0)
    rows, _, _ = gqa.token_rows(v, table[0], np.arange(25), dcp=3, interleave=2, block_size=4)
    vals = fp8.decode_bf16(rows)[:, 0]
    assert np.allclose(got["out"][0], vals[:24].mean(0)) and np.allclose(got["out"][1], vals.mean(0))
    assert np.allclose(got["lse"][:, 0], np.log([24, 25]))


def test_gqa_rank_results_merge_to_the_whole():
    rng = RNG(3)
    W = 4
    k, v = _pools(rng, W, 12, 8, 2, 64), _pools(rng, W, 12, 8, 2, 64)
    table = _table(rng, 2, 5, 12)
    args = dict(q=rng.standard_normal((4, 4, 64)), k_pools=k, v_pools=v, block_table=table,
                seq_lens=[3, 77], qlen=2, dcp=W, interleave=4, block_size=8, kv_dtype="bf16",
                k_scale=0.7, v_scale=1.1, softmax_scale=0.2)
    whole = gqa.decode(**args)
    parts = [gqa.decode(**args, ranks=[r]) for r in range(W)]
    w = np.exp(np.array([p["lse"] for p in parts]) - whole["lse"])
    assert np.allclose(w.sum(0), 1.0)
    assert np.allclose(sum(x[..., None] * p["out"] for x, p in zip(w, parts)), whole["out"])


def test_gqa_equals_the_latent_oracle_on_a_latent_cache():
    # one K/V head of 576 dims whose V is K: the latent oracle's output is the first 512 dims
    rng = RNG(4)
    pools = _pools(rng, 2, 10, 8, 576)
    table = _table(rng, 1, 4, 10)
    q = rng.standard_normal((3, 2, 576))
    got = gqa.decode(q=q, k_pools=pools[:, :, :, None], v_pools=pools[:, :, :, None],
                     block_table=table, seq_lens=[50], qlen=3, dcp=2, interleave=1, block_size=8,
                     kv_dtype="bf16", k_scale=1, v_scale=1, softmax_scale=0.05)
    K = attention.gather_sequence(pools, table[0], 50, dcp=2, interleave=1, block_size=8,
                                  kv_dtype="bf16", kv_scale=1.0)
    for j in range(3):
        o, lse = attention.attend(q[j], K, [48 + j] * 2, 0.05)
        assert np.allclose(got["out"][j, :, :512], o) and np.allclose(got["lse"][j], lse)


def test_key_weights_of_a_step_sum_to_its_rows():
    # each row's probabilities add to one over all ranks' tokens
    rng = RNG(5)
    W, B, ML = 3, 2, 20
    pools = _pools(rng, W, 12, 4, 576)
    table = _table(rng, B, 5, 12)
    lens = [7, 41]
    q = rng.standard_normal((B * 2, 4, 576)) * 0.3
    lse = np.zeros((B * 2, 4))
    for b in range(B):
        K = attention.gather_sequence(pools, table[b], lens[b], dcp=W, interleave=2, block_size=4,
                                      kv_dtype="bf16", kv_scale=1.0)
        for j in range(2):
            lse[2 * b + j] = attention.attend(q[2 * b + j], K, [lens[b] - 1 + j] * 4, 0.1)[1]
    args = dict(q=q, pools=pools, block_table=table, seq_lens=lens, qlen=2, dcp=W, interleave=2,
                block_size=4, kv_dtype="bf16", kv_scale=1.0, softmax_scale=0.1, lse=lse)
    w, added, _ = evict.key_weights(**args, decay=0.0, history=np.full((W, B, ML), 9.0))
    assert np.allclose(added.sum(axis=(0, 2)), 8.0)
    # history counts for the tokens before the step's own, and stays where no token is
    w2, _, _ = evict.key_weights(**args, decay=0.5, history=np.full((W, B, ML), 9.0))
    assert np.isclose((w2 - w).sum(), 0.5 * 9.0 * sum(n - 2 for n in lens))
    assert (w == 9.0).sum() == W * B * ML - sum(lens)


@pytest.mark.parametrize("W,S", [(1, 1), (2, 1), (3, 4), (8, 2)])
def test_new_length_keeps_owners_and_shares(W, S):
    for L in range(1, 200, 7):
        n = evict.new_length(L, 60, W, S)
        assert n <= max(60, 0) and (L <= 60) == (n == L) and (L - n) % (W * S) == 0
        assert L <= 60 or n > 60 - W * S
        gone = [evict.local_count(L, r, W, S) - evict.local_count(n, r, W, S) for r in range(W)]
        assert gone == [(L - n) // W] * W


def test_select_by_hand():
    w = np.array([[[5, 1, 3, 3, 3, 0, 9, 2.0]]])
    kept, lens = evict.select(weights=w, seq_lens=[8], budget=5, sink=1, recent=1, dcp=1, interleave=1)
    assert lens == [5] and kept[0][0] == [0, 2, 3, 6, 7]     # 9, then the first two threes
    w[0, 0, 6] = np.nan
    kept, _ = evict.select(weights=w, seq_lens=[8], budget=5, sink=1, recent=1, dcp=1, interleave=1)
    assert kept[0][0] == [0, 2, 3, 4, 7]
    kept, _ = evict.select(weights=w, seq_lens=[5], budget=5, sink=1, recent=1, dcp=1, interleave=1)
    assert kept[0][0] == [0, 1, 2, 3, 4]


def test_compact_moves_rows_in_order_and_nothing_else():
    pools = np.arange(2 * 4 * 2 * 3).reshape(2, 4, 2, 3)
    table = np.array([[2, 0]])
    out = evict.compact(pools, [[[0, 2, 3]], [[1]]], table, table, 2)
    assert (out[0, 2, 0] == pools[0, 2, 0]).all() and (out[0, 2, 1] == pools[0, 0, 0]).all()
    assert (out[0, 0, 0] == pools[0, 0, 1]).all() and (out[1, 2, 0] == pools[1, 2, 1]).all()
    assert (out[0, [1, 3]] == pools[0, [1, 3]]).all() and (out[0, 0, 1] == pools[0, 0, 1]).all()
