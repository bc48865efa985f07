"""What an eviction leaves of tokens that it could not move: beside bad block ids and after waits that ran out."""
import numpy as np
import pytest
import torch

from mla_latent_kv_25_b200 import binding
from oracle import serving
from tests.test_evict_gpu import Case

pytestmark = pytest.mark.gpu


def check_state(c, nw, np_, nl, ca, moved, first, recent):
    """Every kept token is in its new slot with row, weight and position, or (moved(b, src, dst, arrived)
    false) still in its old one with all three, and the slot that waited for it is marked empty and keeps
    its row.  Returns how many moves were made and how many were not."""
    kept = serving.evict(c.weight.numpy(), c.pos.numpy(), c.lens.numpy(), c.keep.numpy(), first, recent)
    made = left = 0
    rows = c.cache.clone()
    NB = c.cache.shape[0]

    def row(b, s):
        k = int(c.table[b, s // 64])
        return (k, s % 64) if 0 <= k < NB else None

    for b, slots in enumerate(kept):
        n, L = len(slots), int(c.lens[b])
        assert int(nl[b]) == n
        w, p = torch.zeros(L), torch.full((L,), -1, dtype=torch.int32)
        for dst, src in enumerate(slots.tolist()):
            if src == dst:
                w[dst], p[dst] = c.weight[b, dst], c.pos[b, dst]
                continue
            if moved(b, src, dst, int(np_[b, dst]) != -1):
                w[dst], p[dst] = c.weight[b, src], c.pos[b, src]
                rows[row(b, dst)] = c.cache[row(b, src)]
                made += 1
            else:
                w[src], p[src] = c.weight[b, src], c.pos[b, src]
                left += 1
        assert torch.equal(np_[b, :L], p), f"sequence {b}: positions"
        assert torch.equal(nw[b, :L], w), f"sequence {b}: weights"
    assert torch.equal(ca.view(torch.int16), rows.view(torch.int16))
    return made, left


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("block,bad", [(3, 10 ** 6), (3, -1), (0, 10 ** 6), (0, -1)])
def test_a_row_that_cannot_move_keeps_its_weight_and_position(block, bad, in_place):
    """Block 3 holds sources only, block 0 destinations only."""
    c = Case([256, 256], [128, 100], seed=9)
    c.table[0, block] = bad
    nw, np_, nl, ca, err, _ = c.run(0, 0, in_place)
    assert err == binding.DEVERR_BAD_BLOCK
    side = (lambda src, dst: src // 64) if block == 3 else (lambda src, dst: dst // 64)
    made, left = check_state(c, nw, np_, nl, ca, lambda b, s, d, _: b == 1 or side(s, d) != block, 0, 0)
    assert made > 0 and left > 0


@pytest.mark.parametrize("in_place", [False, True])
def test_moves_whose_waits_ran_out(in_place):
    """With a wait limit of one cycle and rows that come from DRAM, every move is made whole or not at
    all, and the next call is right."""
    c = Case([40000, 700, 64], [20000, 350, 64], seed=10, shuffled_pos=True)
    w, p, ln, kp, tb, ca = (t.cuda() for t in (c.weight, c.pos, c.lens, c.keep, c.table, c.cache))
    nw, np_, nl = (w, p, ln) if in_place else (torch.full_like(w, -3.0), torch.full_like(p, -3), torch.full_like(ln, -3))
    ws = binding.alloc_evict_workspace(3, tb.shape[1])
    torch.empty(1 << 29, dtype=torch.uint8, device="cuda").fill_(1)     # larger than L2
    old = binding.mla_set_wait_limit(1)
    try:
        binding.mla_cache_evict(w, p, ln, kp, 4, 32, tb, ca, nw, np_, nl, ws)
        err = binding.mla_get_device_error(ws)
    finally:
        binding.mla_set_wait_limit(0)
    assert old > 1
    made, left = check_state(c, nw.cpu(), np_.cpu(), nl.cpu(), ca.cpu(), lambda b, s, d, arrived: arrived, 4, 32)
    assert err == (binding.DEVERR_TIMEOUT if left else 0)
    assert left > 0, "no wait ran out"
    Case([9000, 700, 64], [4500, 350, 64], seed=10, shuffled_pos=True).check(4, 32, in_place)
