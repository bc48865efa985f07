"""Chunk attention over a cached row with one infinite element, for either sign of its score."""
import numpy as np
import pytest
import torch

from oracle import serving
from tests._serving import SCALE, Chunk, check_attention, f64
from tests.test_chunk_gpu import attend

pytestmark = pytest.mark.gpu

COL = 7


@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("col", [COL, 570])
@pytest.mark.parametrize("at", ["all", "some"])
@pytest.mark.parametrize("H,splits", [(16, 1), (48, 0), (128, 1), (128, 5)])
def test_one_infinite_element(H, splits, at, col, sign):
    """The row is seen by every token of every tile, or by the last four of nine tokens; the element
    is in the latent (part of the values) or in the rotated key (part of the scores alone)."""
    n, L = 9, 300
    c = Chunk([n], [L], H, seed=H)
    c.q[..., col] = sign * c.q[..., col].abs().clamp(min=0.25)
    where = 70 if at == "all" else L - n + 5
    clean = f64(c.cache).copy()
    c.cache[int(c.table[0, where // 64]), where % 64, col] = float("inf")
    out, lse, err = attend(c, splits)
    assert err == 0
    got, glse, q, table = f64(out), f64(lse), f64(c.q), c.table.numpy()
    for j in range(n):
        sees = L - (n - 1 - j)
        rows = serving.rows_of(clean, table, 0, sees)
        if where < sees and sign > 0:
            assert np.isnan(got[j]).all() and np.isnan(glse[j]).all()
            continue
        if where < sees:
            rows = np.delete(rows, where, 0)
        flat = np.zeros(((len(rows) + 63) // 64, 64, 576))
        flat.reshape(-1, 576)[:len(rows)] = rows
        ref, rlse, mass, mag = serving.chunk_attend(q[j:j + 1], np.array([0, 1]), flat, np.arange(len(flat))[None],
                                                    np.array([len(rows)]), SCALE)
        mine = got[j:j + 1].copy()
        if where < sees and col < 512:
            nan = np.isnan(mine[..., col])
            mine[..., col][nan] = ref[..., col][nan]
        check_attention(mine, glse[j:j + 1], ref, rlse, mass, mag, L, f"token {j}")
