"""Inputs and rounding bounds shared by the tests of rotary positions, chunk
attention, attention weights and eviction.

A rounding to bf16 is off by at most HALF = 2^-8 of the value, to fp32 by 2^-24.
"""
import math

import numpy as np
import torch

HALF = 2.0 ** -8
SCALE = 1 / math.sqrt(192)


def f64(t):
    return t.detach().cpu().double().numpy()


def paged(lens, seed, extra_blocks=3, width=0):
    """Shuffled block table over the sequences' blocks plus some unused ones."""
    g = torch.Generator().manual_seed(seed)
    nblk = [(n + 63) // 64 for n in lens]
    NB = sum(nblk) + extra_blocks
    mb = max(max(nblk), 1, width)
    perm = torch.randperm(NB, generator=g)
    table = torch.full((len(lens), mb), -1, dtype=torch.int32)
    at = 0
    for b, k in enumerate(nblk):
        table[b, :k] = perm[at:at + k].to(torch.int32)
        at += k
    return table, NB


class Chunk:
    """A ragged chunk call: n[b] new tokens of a sequence of lens[b] cached rows."""

    def __init__(self, n, lens, H, seed, q_std=1.0, before=0, after=0, poison=False, width=0):
        g = torch.Generator().manual_seed(seed)
        self.n, self.H, self.B = list(n), H, len(n)
        self.table, NB = paged(lens, seed, width=width)
        self.lens = torch.tensor(lens, dtype=torch.int32)
        offs = np.concatenate([[0], np.cumsum(n)]) + before
        self.offs = torch.tensor(offs, dtype=torch.int32)
        self.T = int(offs[-1]) + after
        self.q = (torch.randn(self.T, H, 576, generator=g) * q_std).bfloat16()
        self.cache = (torch.randn(NB, 64, 576, generator=g) / math.sqrt(512)).bfloat16()
        if poison:  # rows that no token may see
            live = torch.zeros(NB, 64, dtype=torch.bool)
            for b, L in enumerate(lens):
                s = torch.arange(L)
                live[self.table[b, s // 64].long(), s % 64] = True
            bad = torch.tensor([float("nan"), float("inf"), -float("inf"), 3e38])
            self.cache[~live] = bad[torch.arange(576) % 4].bfloat16()
            owned = torch.zeros(self.T, dtype=torch.bool)
            owned[int(offs[0]):int(offs[-1])] = True
            self.q[~owned] = float("nan")

    def cuda(self):
        return tuple(t.cuda() for t in (self.q, self.offs, self.cache, self.table, self.lens))

    def np(self):
        return (f64(self.q), self.offs.numpy(), f64(self.cache), self.table.numpy(), self.lens.numpy())


def score_slack(mag):
    """Error of a score of 576 products accumulated in fp32, relative 2^-23 a step (a step
    may truncate): at most 576 * 2^-23 of the sum of magnitudes, and the scale's rounding."""
    return (576 * 2.0 ** -23 + 2.0 ** -23) * mag


def check_attention(got, glse, ref, rlse, mass, mag, longest, what=""):
    """out: every probability is off by twice its score's error (its own and the sum's) and
    one bf16 rounding, the result by another; lse by a score's error, its own fp32 rounding
    (2^-22 covers log2 -> ln) and that of a sum of `longest` terms."""
    assert np.array_equal(np.isnan(ref), np.isnan(got)), f"{what}: rows written differ"
    live = ~np.isnan(ref)
    ds = score_slack(mag)[..., None]
    tol = HALF * (mass + np.abs(ref)) * (1 + HALF) + mass * (2 * ds + 2.0 ** -18 + longest * 2.0 ** -23)
    bad = np.abs(got - ref)[live] > np.broadcast_to(tol, ref.shape)[live]
    assert not bad.any(), f"{what}: out off in {bad.sum()} of {bad.size}, worst {np.nanmax(np.abs(got - ref) - tol):.3e}"
    fin = np.isfinite(rlse)
    assert np.array_equal(glse[~fin & ~np.isnan(rlse)], rlse[~fin & ~np.isnan(rlse)]), f"{what}: empty rows' lse"
    off = np.abs(glse[fin] - rlse[fin])
    ltol = (score_slack(mag) + 2.0 ** -22 * (1 + np.abs(rlse)) + longest * 2.0 ** -23)[fin]
    assert (off <= ltol).all(), f"{what}: lse off by {off.max():.3e}, bound {ltol[off.argmax()]:.3e}"
