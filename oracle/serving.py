"""Rotary positions, chunk attention, attention weights and eviction in plain FP64 numpy.

TEST INFRASTRUCTURE ONLY: the tests are the only callers; nothing here is
shared with, or called by, the CUDA path.

Every function takes numpy arrays (bf16 values already widened to float64)
and loops over the definition.  Beside results it returns the magnitudes that
rounding bounds are stated in.
"""
from __future__ import annotations

import math

import numpy as np

BLOCK, D_C, D_ROW = 64, 512, 576


def rope_freqs(rot, base=10000.0, scaling="none", factor=1.0, orig_len=4096.0, beta_fast=32.0, beta_slow=1.0):
    """Angle per position of every pair, one pair at a time."""
    out = []
    for i in range(rot // 2):
        theta = math.exp(-2.0 * i / rot * math.log(base))
        if scaling == "none":
            f = theta
        elif scaling == "linear":
            f = theta / factor
        elif scaling == "ntk":
            # the slowest pair (i = rot/2 - 1) turns `factor` times slower, the fastest as before
            f = theta * factor ** (-2.0 * i / (rot - 2.0))
        else:
            turns_to_pair = lambda n: rot * math.log(orig_len / (2 * math.pi * n)) / (2 * math.log(base))  # noqa: E731
            lo = max(0, math.floor(turns_to_pair(beta_fast)))
            hi = min(rot - 1, math.ceil(turns_to_pair(beta_slow)))
            share = (i - lo) / max(hi - lo, 1e-3)
            share = min(1.0, max(0.0, share))
            f = theta / factor * share + theta * (1 - share)
        out.append(f)
    return np.array(out)


def rope(x, pos, freqs, mscale=1.0, half=False, inverse=False):
    """x [T, ..., rot] rotated by pos[t] * freqs, as a product of complex numbers."""
    x = np.asarray(x, np.float64)
    r = x.shape[-1] // 2
    z = x[..., :r] + 1j * x[..., r:] if half else x[..., 0::2] + 1j * x[..., 1::2]
    ang = np.asarray(pos, np.float64).reshape((-1,) + (1,) * (x.ndim - 1)) * freqs
    z = z * mscale * np.exp((-1j if inverse else 1j) * ang)
    out = np.empty_like(x)
    if half:
        out[..., :r], out[..., r:] = z.real, z.imag
    else:
        out[..., 0::2], out[..., 1::2] = z.real, z.imag
    return out


def rows_of(cache, table, b, n):
    """The first n cached rows of sequence b, in slot order."""
    slots = np.arange(n)
    return cache[table[b, slots // BLOCK], slots % BLOCK]


def _chunks(q_offsets, seq_lens):
    for b in range(len(seq_lens)):
        n = int(q_offsets[b + 1] - q_offsets[b])
        for j in range(n):
            yield b, int(q_offsets[b]) + j, max(0, int(seq_lens[b]) - (n - 1 - j))


def chunk_attend(q, q_offsets, cache, table, seq_lens, scale):
    """(out [T,H,512], lse [T,H], sum of p|v| [T,H,512], largest scale * sum |q k| [T,H]);
    tokens of no sequence stay NaN."""
    T, H = q.shape[:2]
    out = np.full((T, H, D_C), np.nan)
    lse = np.full((T, H), np.nan)
    mass = np.full((T, H, D_C), np.nan)
    mag = np.full((T, H), np.nan)
    for b, t, sees in _chunks(q_offsets, seq_lens):
        if sees == 0:
            out[t], lse[t], mass[t], mag[t] = 0.0, -np.inf, 0.0, 0.0
            continue
        k = rows_of(cache, table, b, sees)
        s = (q[t] @ k.T) * scale
        mag[t] = (np.abs(q[t]) @ np.abs(k).T).max(1) * abs(scale)
        m = s.max(1, keepdims=True)
        e = np.exp(s - m)
        z = e.sum(1, keepdims=True)
        lse[t] = (m + np.log(z))[:, 0]
        out[t] = (e / z) @ k[:, :D_C]
        mass[t] = (e / z) @ np.abs(k[:, :D_C])
    return out, lse, mass, mag


def weigh(q, q_offsets, lse, cache, table, seq_lens, scale):
    """(added weight [B, S], largest scale * sum |q k| and largest |argument| of exp per sequence)."""
    S = table.shape[1] * BLOCK
    add = np.zeros((len(seq_lens), S))
    mag = np.zeros(len(seq_lens))
    arg = np.zeros(len(seq_lens))
    for b, t, sees in _chunks(q_offsets, seq_lens):
        if sees == 0:
            continue
        k = rows_of(cache, table, b, sees)
        s = (q[t] @ k.T) * scale
        a = s - np.asarray(lse[t], np.float64)[:, None]
        add[b, :sees] += np.exp(a).sum(0)
        mag[b] = max(mag[b], ((np.abs(q[t]) @ np.abs(k).T) * abs(scale)).max())
        fin = np.isfinite(lse[t])
        if fin.any():
            arg[b] = max(arg[b], np.abs(s[fin]).max() + np.abs(lse[t][fin]).max())
    return add, mag, arg


def evict(weight, slot_pos, seq_lens, keep, n_first, n_recent):
    """Per sequence (kept slots in new slot order): list of int arrays."""
    result = []
    for b, L in enumerate(int(v) for v in seq_lens):
        n = min(max(int(keep[b]), 0), L)
        newest = max((int(slot_pos[b, s]) for s in range(L)), default=0)

        def order(s):
            p = int(slot_pos[b, s])
            w = float(weight[b, s])
            w = -math.inf if math.isnan(w) else w
            return (0 if p < n_first or p > newest - n_recent else 1, -w, s)

        kept = set(sorted(range(L), key=order)[:n])
        movers = sorted(s for s in kept if s >= n)
        slots = []
        for s in range(n):
            slots.append(s if s in kept else movers.pop(0))
        assert not movers
        result.append(np.array(slots, np.int64))
    return result
