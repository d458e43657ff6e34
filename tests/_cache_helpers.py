"""Inputs and tolerances of the grouped-head and eviction tests."""

from __future__ import annotations

import math

import numpy as np
import torch

import oracle

NAN_CODE = 0x7F


def raw(t):
    """Host bits of a BF16 (uint16) or E4M3 (uint8) tensor."""
    t = t.detach().cpu().contiguous()
    return t.numpy() if t.dtype == torch.uint8 else t.view(torch.int16).numpy().view(np.uint16)


def f64(t):
    return t.detach().double().cpu().numpy()


class Cache:
    """Shuffled pools of one layer. Slots that hold no token of a sequence hold NaN, so that
    anything read behind a length, or in a spare block, shows."""

    def __init__(self, lens, *, dcp, interleave, block, tails, dtype, seed, scale=0.02, bound=None,
                 spare=0):
        self.lens, self.W, self.S, self.bs, self.dtype = list(lens), dcp, interleave, block, dtype
        self.B = len(self.lens)
        longest = max(oracle.evict.local_count(n, 0, dcp, interleave) for n in self.lens)
        self.ML = max(1, longest if bound is None else bound)
        self.MB = -(-self.ML // block)
        self.NB = self.B * self.MB * (2 if spare else 1) + 3
        g = torch.Generator().manual_seed(seed)
        perm = torch.randperm(self.NB, generator=g).to(torch.int32)
        self.table = perm[: self.B * self.MB].view(self.B, self.MB).contiguous()
        self.other = perm[self.B * self.MB: 2 * self.B * self.MB].view(self.B, self.MB).contiguous() if spare else None
        self.scale = scale if dtype == "fp8" else 1.0
        self.pools = []
        for tail in tails:
            x = torch.randn(dcp, self.NB, block, *tail, generator=g)
            if dtype == "fp8":
                x = (x / scale).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
                full = torch.full_like(x, NAN_CODE)
            else:
                x = x.bfloat16()
                full = torch.full_like(x, math.nan)
            for b, n in enumerate(self.lens):
                p = np.arange(max(n, 0))
                r = oracle.metadata.owner(p, dcp, interleave)
                li = oracle.metadata.local_index(p, dcp, interleave)
                ok = li < self.ML
                r, li = torch.as_tensor(r[ok]), torch.as_tensor(li[ok])
                at = (r, self.table[b].long()[li // block], li % block)
                full[at] = x[at]
            self.pools.append(full)

    def dims(self, dm, qlen=1, heads=8, splits=1, causal=True):
        return dm.make_dims(batch=self.B, qlen=qlen, num_heads=heads, dcp=self.W,
                            interleave=self.S, block_size=self.bs, max_blocks_per_seq=self.MB,
                            max_local_len=self.ML, num_blocks=self.NB, num_splits=splits,
                            causal=causal)

    @property
    def geometry(self):
        return dict(dcp=self.W, interleave=self.S, block_size=self.bs)

    def kv_dtype(self, dm):
        return dm.KV_FP8_E4M3 if self.dtype == "fp8" else dm.KV_BF16

    def dev_scale(self, factor=1.0):
        return torch.tensor([self.scale * factor], device="cuda") if self.dtype == "fp8" else None

    def lens_dev(self):
        return torch.tensor(self.lens, dtype=torch.int32, device="cuda")


def gqa_tolerance(ref, dim):
    """out: each weight is rounded to 16 bits before the second product (half a BF16 step,
    2^-8, covers both types), the result once more to BF16, and a score that is off by ds
    moves a weight by a factor e^ds; ds: `dim` products and their sums in 32 bits, each off by
    at most 2^-23 of the sum of magnitudes (a product's rounding, and a sum that drops bits),
    then four roundings of the score. lse: ds, the exponential and logarithm (2^-20 together)
    and two roundings of its own size."""
    fin = np.isfinite(ref["lse"])
    ds = (dim + 4) * 2.0 ** -23 * ref["abss"] + 2.0 ** -20
    tol_o = 2.0 ** -8 * (ref["absv"] + np.abs(ref["out"])) + 2 * ds[..., None] * ref["absv"]
    tol_l = ds + 2.0 ** -22 * np.where(fin, np.abs(ref["lse"]), 0.0)
    return tol_o, tol_l


def assert_gqa(out, lse, ref, dim, what=""):
    tol_o, tol_l = gqa_tolerance(ref, dim)
    o, s = f64(out), f64(lse)
    assert np.array_equal(np.isneginf(s), np.isneginf(ref["lse"])), what
    fin = np.isfinite(ref["lse"])
    assert (np.abs(s[fin] - ref["lse"][fin]) <= tol_l[fin]).all(), what
    assert np.isfinite(o).all() and (np.abs(o - ref["out"]) <= tol_o).all(), what
    assert (o[~fin] == 0).all(), what


def assert_key_weights(got, ref, added, slack, lse, decay, what=""):
    """A row's weight is e^(s - lse): s is off by at most 580 * 2^-23 of its sum of magnitudes
    (576 products and sums in 32 bits, and the scales), lse and the difference by 2^-22 of
    their size, q's two terms (FP8) together by 2^-20 of its largest element (within the 2^-17 of the
    sum of magnitudes), the exponential by 2^-21; sums of up to a few
    hundred positive terms by 2^-23 each."""
    fin = np.abs(lse[np.isfinite(lse)]).max() if np.isfinite(lse).any() else 0.0
    tol = (580 * 2.0 ** -23 + 2.0 ** -17) * slack + (2.0 ** -20 * (fin + 2) + 2.0 ** -14) * added + 2.0 ** -22 * np.abs(ref)
    bad = ~(np.abs(f64(got) - ref) <= tol) & ~(np.isnan(ref) & np.isnan(f64(got)))
    assert not bad.any(), (what, int(bad.sum()), np.argwhere(bad)[:3])
    # and together far closer: the errors above are of random sign
    d, n = (f64(got) - ref)[np.isfinite(ref)], np.linalg.norm(ref[np.isfinite(ref)])
    assert np.linalg.norm(d) <= 2e-5 * max(n, 1e-30), (what, np.linalg.norm(d) / n)
