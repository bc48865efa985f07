"""Calls above the sizes of one round of a planning loop: more sequences and more tiles than the chunk
plan has threads, tiles cut into more pieces than a warp has lanes, more sequences than a grid has rows."""
import numpy as np
import pytest
import torch

from mla_latent_kv_25_b200 import binding
from oracle import serving
from tests._serving import SCALE, Chunk, check_attention, f64
from tests.test_chunk_gpu import attend, check, check_weights, weigh
from tests.test_evict_gpu import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("num_splits", [0, 7, 200])
@pytest.mark.parametrize("H", [16, 128])
def test_chunk_of_more_sequences_than_the_plan_has_threads(H, num_splits):
    """1500 sequences of 0 to 2 tokens over 0 to 100 rows: two rounds of sequences and, at 16 heads
    and at 128, two of tiles."""
    g = torch.Generator().manual_seed(H + num_splits)
    lens = torch.randint(0, 101, (1500,), generator=g).tolist()
    n = torch.randint(0, 3, (1500,), generator=g).tolist()
    n[1000:1100] = [2] * 100
    lens[1023:1026] = [100, 0, 65]
    assert sum(k > 0 for k in n) > 1000
    if H == 128:       # shorter, for the definition's sake
        lens = [min(L, 40) for L in lens]
    c = Chunk(n, lens, H, seed=H, before=1, after=2)
    out, lse = check(c, num_splits, what=f"1500 sequences, splits={num_splits}")
    if num_splits == 0:
        check_weights(weigh(c, lse.cpu(), None), c, lse.cpu(), None, what="1500 sequences")


def test_chunk_of_more_tiles_than_the_plan_has_threads():
    """A prompt of 2500 tokens of 128 heads over 2600 rows: 1250 tiles of two tokens, all with rows to
    read, before another sequence."""
    T, H, L = 2500, 128, 2600
    c = Chunk([0, 0], [L, 70], H, seed=1)
    c.n, c.T, c.offs = [T, 3], T + 3, torch.tensor([0, T, T + 3], dtype=torch.int32)
    g = torch.Generator(device="cuda").manual_seed(2)
    q = torch.randn(c.T, H, 576, generator=g, device="cuda").bfloat16()
    out = torch.full((c.T, H, 512), float("nan"), dtype=torch.bfloat16, device="cuda")
    lse = torch.full((c.T, H), float("nan"), device="cuda")
    ws = binding.alloc_chunk_workspace(c.T, 2, H)
    args = (c.offs.cuda(), c.cache.cuda(), c.table.cuda(), c.lens.cuda(), SCALE)
    binding.mla_chunk_attend(q, *args, out, lse, ws)
    assert binding.mla_get_device_error(ws) == 0
    assert not bool(out.isnan().any()) and bool(lse.isfinite().all())
    cache, table = f64(c.cache), c.table.numpy()
    # tiles on both sides of the 1024th, the first, the last, and some between
    tokens = [0, 1, 511, 1000, 2046, 2047, 2048, 2049, 2050, 2499, T, T + 1, T + 2]
    for t in tokens:
        b, j, n, rows = (0, t, T, L) if t < T else (1, t - T, 3, 70)
        one = (f64(q[t:t + 1]), np.array([0, 1]), cache, table[b:b + 1], np.array([rows - (n - 1 - j)]), SCALE)
        ref, rlse, mass, mag = serving.chunk_attend(*one)
        check_attention(f64(out[t:t + 1]), f64(lse[t:t + 1]), ref, rlse, mass, mag, L, f"token {t}")


@pytest.mark.parametrize("n,L,H,num_splits", [(1, 40000, 16, 64), (3, 45000, 16, 64), (1, 90000, 48, 130)])
def test_chunk_tiles_in_more_pieces_than_a_warp_has_lanes(n, L, H, num_splits):
    check(Chunk([n], [L], H, seed=num_splits), num_splits, what=f"{L} rows, splits={num_splits}")


def test_chunk_repeats_bit_for_bit():
    """Cut tiles, whole tiles and the order in which engines finish leave no trace."""
    c = Chunk([40, 3, 1, 17], [3000, 500, 7000, 64], 128, seed=63)
    a, la, _ = attend(c)
    for _ in range(10):
        b, lb, _ = attend(c)
        assert torch.equal(a.view(torch.int16), b.view(torch.int16)) and torch.equal(la, lb)


def test_evict_of_more_sequences_than_a_grid_has_rows():
    """65600 sequences, most of them empty; those at and past the 65536th have pointers of their own."""
    B = 65600
    lens = [0] * B
    for b in list(range(0, B, 1000)) + list(range(65530, B)):
        lens[b] = 1 + (7 * b) % 64
    Case(lens, [1 + b % 40 for b in range(B)], seed=12, shuffled_pos=False).check(2, 5)
