"""Pins of oracle/serving.py against library routines and closed forms."""
import math

import numpy as np
import torch

from oracle import naive, serving
from tests._serving import Chunk, SCALE


def test_rope_matches_the_plain_rotation_and_both_layouts_agree():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((7, 3, 64))
    pos = np.array([0, 1, 5, 77, 4095, 131071, 2 ** 31 - 1])
    f = serving.rope_freqs(64)
    ref = np.stack([naive.rope(x[i], np.full(3, pos[i])) for i in range(7)])
    tol = 1e-12 * (1 + pos[:, None, None])  # theta from exp/log against a power: relative 1e-15 of the angle
    assert (np.abs(serving.rope(x, pos, f) - ref) <= tol).all()
    perm = np.concatenate([np.arange(0, 64, 2), np.arange(1, 64, 2)])
    assert np.allclose(serving.rope(x[..., perm], pos, f, half=True), serving.rope(x, pos, f)[..., perm], atol=1e-13)
    back = serving.rope(serving.rope(x, pos, f), pos, f, inverse=True)
    assert np.allclose(back, x, atol=1e-12)


def test_scaled_frequencies_closed_forms():
    plain = serving.rope_freqs(64)
    assert np.allclose(serving.rope_freqs(64, scaling="linear", factor=8.0), plain / 8)
    ntk = serving.rope_freqs(64, scaling="ntk", factor=8.0)
    assert ntk[0] == plain[0] and math.isclose(ntk[-1], plain[-1] / 8, rel_tol=1e-12)
    yarn = serving.rope_freqs(64, scaling="yarn", factor=40.0)
    turns = plain * 4096 / (2 * math.pi)
    assert np.allclose(yarn[turns > 40], plain[turns > 40]) and np.allclose(yarn[turns < 0.7], plain[turns < 0.7] / 40)
    assert np.all(np.diff(yarn) < 0)


def test_chunk_attention_matches_library_attention():
    c = Chunk([5, 0, 3], [70, 10, 3], 16, seed=1)
    q, offs, cache, table, lens = c.np()
    out, lse, mass, _ = serving.chunk_attend(q, offs, cache, table, lens, SCALE)
    for b in range(3):
        n, L = c.n[b], int(lens[b])
        if n == 0:
            continue
        k = torch.from_numpy(serving.rows_of(cache, table, b, L))
        qb = torch.from_numpy(q[offs[b]:offs[b + 1]]).permute(1, 0, 2)
        mask = torch.arange(L)[None] < (L - n + 1 + torch.arange(n))[:, None]
        ref = torch.nn.functional.scaled_dot_product_attention(
            qb, k.expand(16, -1, -1), k[:, :512].expand(16, -1, -1), attn_mask=mask, scale=SCALE)
        assert np.allclose(out[offs[b]:offs[b + 1]], ref.permute(1, 0, 2).numpy(), atol=1e-12)
    assert (mass >= np.abs(out) - 1e-12).all()


def test_weights_sum_to_the_number_of_queries():
    c = Chunk([4, 1], [100, 65], 16, seed=2)
    q, offs, cache, table, lens = c.np()
    _, lse, _, _ = serving.chunk_attend(q, offs, cache, table, lens, SCALE)
    add, _, _ = serving.weigh(q, offs, lse, cache, table, lens, SCALE)
    assert np.allclose(add.sum(1), [4 * 16, 16])
    assert (add[0, 100:] == 0).all() and (add[1, 65:] == 0).all()


def test_eviction_order():
    w = np.array([[5, 1, 9, 9, 0, 9, np.nan, 2.0]])
    pos = np.arange(8)[None]
    # no protection: the 9s (slots 2, 3, 5), then 5 (slot 0); slot 5 moves into the first free slot
    assert serving.evict(w, pos, [8], [4], 0, 0)[0].tolist() == [0, 5, 2, 3]
    # ties go to the lower slot
    assert serving.evict(w, pos, [8], [2], 0, 0)[0].tolist() == [2, 3]
    # the first one and the last two are protected, NaN counts as the smallest
    assert serving.evict(w, pos, [8], [4], 1, 2)[0].tolist() == [0, 6, 2, 7]
    assert serving.evict(w, pos, [8], [1], 1, 2)[0].tolist() == [0]
    assert serving.evict(w, pos, [8], [99], 0, 0)[0].tolist() == list(range(8))
    assert serving.evict(w, pos, [8], [-1], 0, 0)[0].tolist() == []
