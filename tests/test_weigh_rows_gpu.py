"""Attention weights of query rows that do not fill the tensor cores' step of 32 rows."""
import numpy as np
import pytest
import torch

from mla_latent_kv_25_b200 import binding
from oracle import serving
from tests._serving import SCALE, Chunk
from tests.test_chunk_gpu import check_weights, weigh

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n,H", [(1, 16), (3, 16), (1, 48), (1, 80), (1, 112), (17, 16), (33, 16), (7, 48), (3, 112), (5, 80)])
def test_rows_behind_the_tile_are_not_looked_at(n, H):
    """The next sequence's queries, whose rows lie behind this one's, are NaN."""
    c = Chunk([n, 2], [200, 70], H, seed=n * H)
    good = torch.from_numpy(serving.chunk_attend(*c.np(), SCALE)[1]).float()
    w = torch.rand(2, c.table.shape[1] * 64, generator=torch.Generator().manual_seed(1))
    whole = weigh(c, good, w.cuda())
    check_weights(whole, c, good, w, what="finite")
    c.q[n:] = float("nan")
    got = weigh(c, good, w.cuda())
    assert torch.equal(got[0], whole[0])
    assert bool(got[1, :69].isnan().all()) and np.all(got[1, 70:].cpu().numpy() == -7.0)


@pytest.mark.parametrize("n,lens,H", [([1] * 40, [3000] * 40, 128), ([32], [1024], 128), ([40, 3], [9000, 500], 64)])
def test_slots_of_a_call_that_gave_up(n, lens, H):
    """Every slot holds its old weight or the right new one, in place too; the next call is right."""
    c = Chunk(n, lens, H, seed=7)
    t = c.cuda()
    lse = torch.full((c.T, H), 6.0, device="cuda")
    w = torch.rand(c.B, c.table.shape[1] * 64, generator=torch.Generator().manual_seed(1)).cuda()
    right = w.clone()
    binding.mla_cache_weigh(t[0], t[1], lse, t[2], t[3], t[4], SCALE, w, right)
    assert binding.mla_cache_get_error() == 0
    some = 0
    for limit in (1, 1000, 20000):
        got = w.clone()
        binding.mla_set_wait_limit(limit)
        try:
            binding.mla_cache_weigh(t[0], t[1], lse, t[2], t[3], t[4], SCALE, got, got)
            bits = binding.mla_cache_get_error()
        finally:
            binding.mla_set_wait_limit(0)
        old, new = got == w, got == right
        assert bool((old | new).all())
        left = int((~new).sum())
        assert bits == binding.DEVERR_TIMEOUT if left else bits in (0, binding.DEVERR_TIMEOUT)
        some += left
    assert some > 0, "no wait ran out"
    got = w.clone()
    binding.mla_cache_weigh(t[0], t[1], lse, t[2], t[3], t[4], SCALE, got, got)
    assert binding.mla_cache_get_error() == 0 and torch.equal(got, right)
