"""Caches, queries and outputs whose element offsets pass 32 bits."""
import numpy as np
import pytest
import torch

from mla_latent_kv_25_b200 import binding
from oracle import serving
from tests._serving import SCALE, Chunk, check_attention, f64
from tests.test_chunk_gpu import check_weights

pytestmark = pytest.mark.gpu

FAR = 130000 * 64 * 576          # elements of a cache of 130000 blocks: 4.8e9


def test_blocks_at_the_end_of_a_large_cache():
    """Append, attend, weigh and evict on the last blocks of 9.6 GB."""
    c = Chunk([5, 3], [300, 70], 32, seed=1)
    NB, small = FAR // (64 * 576), c.cache.shape[0]
    big = torch.empty(NB, 64, 576, dtype=torch.bfloat16, device="cuda")
    big[NB - small:] = c.cache.cuda()
    far = torch.where(c.table >= 0, c.table + (NB - small), c.table)
    q, offs, _, table, lens = c.cuda()
    table = far.cuda()
    out, lse = torch.empty(8, 32, 512, dtype=torch.bfloat16, device="cuda"), torch.empty(8, 32, device="cuda")
    ws = binding.alloc_chunk_workspace(8, 2, 32)
    binding.mla_chunk_attend(q, offs, big, table, lens, SCALE, out, lse, ws)
    assert binding.mla_get_device_error(ws) == 0
    check_attention(f64(out), f64(lse), *serving.chunk_attend(*c.np(), SCALE), 300, "far blocks")
    w = torch.full((2, table.shape[1] * 64), -7.0, device="cuda")
    binding.mla_cache_weigh(q, offs, lse, big, table, lens, SCALE, None, w)
    check_weights(w, c, lse.cpu(), None, what="far blocks")
    # the last row of the first sequence again, through append
    row = torch.randn(1, 576, generator=torch.Generator().manual_seed(2)).bfloat16().cuda()
    i32 = lambda v: torch.tensor([v], dtype=torch.int32, device="cuda")  # noqa: E731
    binding.mla_cache_append_rope(row[:, :512], row[:, 512:], i32(0), i32(299), i32(0), binding.mla_rope_freqs(), table, big)
    assert binding.mla_cache_get_error() == 0
    assert torch.equal(big[int(far[0, 4]), 299 % 64], row[0])
    # eviction
    pos = torch.arange(w.shape[1], dtype=torch.int32, device="cuda").repeat(2, 1)
    keep = torch.tensor([120, 40], dtype=torch.int32, device="cuda")
    kept = serving.evict(f64(w), pos.cpu().numpy(), c.lens.numpy(), keep.cpu().numpy(), 4, 8)
    before = big[NB - small:].cpu()
    binding.mla_cache_evict(w, pos, lens, keep, 4, 8, table, big, w, pos, lens, (ew := binding.alloc_evict_workspace(2, table.shape[1])))
    assert binding.mla_get_device_error(ew) == 0
    after = big[NB - small:].cpu()
    for b, s in enumerate(kept):
        to = np.arange(len(s))
        assert torch.equal(after[c.table[b, to // 64].long(), to % 64], before[c.table[b, s // 64].long(), s % 64])


def test_rows_at_the_end_of_many_queries():
    """70000 tokens of 128 heads, of which the last ten have a sequence: rows past the 2^32-th element
    of q and out are rotated, attended and weighed."""
    T, H, n, L = 70000, 128, 10, 200
    assert T * H * 512 > 2 ** 32
    c = Chunk([n], [L], H, seed=3, before=0)
    q = torch.empty(T, H, 576, dtype=torch.bfloat16, device="cuda")
    q[T - n:] = c.q.cuda()
    pos = torch.zeros(T, dtype=torch.int32, device="cuda")
    pos[T - n:] = torch.arange(n, dtype=torch.int32, device="cuda") + 1000
    freqs = binding.mla_rope_freqs()
    binding.mla_rope(q[..., 512:], pos, freqs, q[..., 512:])
    ref = serving.rope(f64(c.q[..., 512:]), np.arange(n) + 1000, f64(freqs))
    assert np.abs(f64(q[T - n:, :, 512:]) - ref).max() <= 2.0 ** -8 * np.abs(ref).max() + 2.0 ** -16
    c.q = q[T - n:].cpu()
    out = torch.empty(T, H, 512, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(T, H, device="cuda")
    out[T - n - 1].fill_(3.0)
    offs = torch.tensor([T - n, T], dtype=torch.int32, device="cuda")
    _, _, cache, table, lens = c.cuda()
    ws = binding.alloc_chunk_workspace(T, 1, H)
    binding.mla_chunk_attend(q, offs, cache, table, lens, SCALE, out, lse, ws)
    assert binding.mla_get_device_error(ws) == 0
    check_attention(f64(out[T - n:]), f64(lse[T - n:]), *serving.chunk_attend(*c.np(), SCALE), L, "far rows")
    assert bool((out[T - n - 1] == 3).all())
    w = torch.full((1, table.shape[1] * 64), -7.0, device="cuda")
    binding.mla_cache_weigh(q, offs, lse, cache, table, lens, SCALE, None, w)
    check_weights(w, c, lse[T - n:].cpu(), None, what="far rows")
