"""Attention weights of query rows that do not fill the tensor cores' step of 32 rows."""
import numpy as np
import pytest
import torch

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
