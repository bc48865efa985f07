"""Calls of the chunk, weight, eviction and rotation operators that go wrong easily: values that
are not finite where a mask hides them, waits that run out, several streams, shared workspaces."""
import numpy as np
import pytest
import torch

from mla_latent_kv_25_b200 import binding
from oracle import serving
from tests._serving import SCALE, Chunk, check_attention, f64
from tests.test_chunk_gpu import attend, check_weights, weigh
from tests.test_evict_gpu import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("H", [16, 48, 128])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_a_row_that_is_not_finite_reaches_only_the_tokens_that_see_it(H, bad):
    """Tokens of one tile see different lengths: the last rows belong to some of them only."""
    n, L = 9, 133
    c = Chunk([n], [L], H, seed=H)
    clean = f64(c.cache).copy()
    first = L - n + 5                       # seen by tokens 5.. alone
    for s in (first, first + 1):
        c.cache[int(c.table[0, s // 64]), s % 64, :] = bad
    out, lse, err = attend(c)
    assert err == 0
    q, offs, _, table, lens = c.np()
    ref, rlse, mass, mag = serving.chunk_attend(q, offs, clean, table, lens, SCALE)
    check_attention(f64(out)[:5], f64(lse)[:5], ref[:5], rlse[:5], mass[:5], mag[:5], L, "tokens that do not see it")
    if np.isnan(bad):
        assert bool(out[5:].isnan().all()) and bool(lse[5:].isnan().all())
    # its own weight alone is spoilt
    rl = torch.from_numpy(rlse).float()
    got = weigh(c, rl, None)
    good = Chunk([n], [L], H, seed=H)
    want = weigh(good, rl, None)
    rest = [s for s in range(L) if s not in (first, first + 1)]
    assert torch.equal(got[0, rest], want[0, rest])


def test_query_rows_that_are_not_finite_stay_alone():
    c = Chunk([6], [200], 32, seed=3)
    c.q[2, 7] = float("nan")
    c.q[4, 0, 100] = float("inf")
    out, lse, err = attend(c)
    good = Chunk([6], [200], 32, seed=3)
    ref, rlse, mass, mag = serving.chunk_attend(*good.np(), SCALE)
    ok = np.ones((6, 32), bool)
    ok[2, 7] = ok[4, 0] = False
    for t, h in zip(*np.nonzero(ok)):
        check_attention(f64(out)[t, h][None], f64(lse)[t, h][None], ref[t, h][None], rlse[t, h][None],
                        mass[t, h][None], mag[t, h][None], 200)
    assert bool(out[2, 7].isnan().all())


def test_waits_that_run_out():
    """A wait limit of a microsecond: the calls end, say so and leave the next call right."""
    c = Chunk([40, 3], [3000, 500], 128, seed=5)
    rlse = serving.chunk_attend(*c.np(), SCALE)
    q, offs, cache, table, lens = c.cuda()
    out = torch.empty(c.T, 128, 512, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(c.T, 128, device="cuda")
    ws = binding.alloc_chunk_workspace(c.T, 2, 128)
    w = torch.zeros(2, table.shape[1] * 64, device="cuda")
    binding.mla_cache_get_error()
    old = binding.mla_set_wait_limit(1000)
    try:
        binding.mla_chunk_attend(q, offs, cache, table, lens, SCALE, out, lse, ws)
        torch.cuda.synchronize()
        given_up = bool(lse.isnan().all()) and bool((out == 0).all())
        binding.mla_chunk_attend(q, offs, cache, table, lens, SCALE, out, lse, ws)
        torch.cuda.synchronize()
        still = bool(lse.isnan().all()) and bool((out == 0).all())
        bits = binding.mla_get_device_error(ws)
        binding.mla_cache_weigh(q, offs, torch.zeros(c.T, 128, device="cuda"), cache, table, lens, SCALE, None, w)
        wbits = binding.mla_cache_get_error()
    finally:
        binding.mla_set_wait_limit(0 if old <= 0 else old)
    assert bits == binding.DEVERR_TIMEOUT and given_up and still
    assert wbits == binding.DEVERR_TIMEOUT
    binding.mla_chunk_attend(q, offs, cache, table, lens, SCALE, out, lse, ws)
    assert binding.mla_get_device_error(ws) == 0
    check_attention(f64(out), f64(lse), *rlse, 3000, "after a call that gave up")
    binding.mla_cache_weigh(q, offs, lse, cache, table, lens, SCALE, None, w)
    assert binding.mla_cache_get_error() == 0
    check_weights(w, c, lse.cpu(), None, what="after a call that gave up", untouched=0.0)


def test_two_streams_with_workspaces_of_their_own():
    a, b = Chunk([30, 5], [700, 64], 64, seed=6), Chunk([7], [2000], 128, seed=7)
    runs = []
    for c in (a, b):
        t = c.cuda()
        out = torch.empty(c.T, c.H, 512, dtype=torch.bfloat16, device="cuda")
        lse = torch.empty(c.T, c.H, device="cuda")
        w = torch.zeros(c.B, c.table.shape[1] * 64, device="cuda")
        runs.append((c, t, out, lse, binding.alloc_chunk_workspace(c.T, c.B, c.H), w, torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(5):
        for c, t, out, lse, ws, w, st in runs:
            binding.mla_chunk_attend(t[0], t[1], t[2], t[3], t[4], SCALE, out, lse, ws, stream=st)
            binding.mla_cache_weigh(t[0], t[1], lse, t[2], t[3], t[4], SCALE, None, w, stream=st)
    torch.cuda.synchronize()
    for c, t, out, lse, ws, w, st in runs:
        assert binding.mla_get_device_error(ws) == 0
        check_attention(f64(out), f64(lse), *serving.chunk_attend(*c.np(), SCALE), int(c.lens.max()))
        check_weights(w, c, lse.cpu(), None, untouched=0.0)


def test_two_graphs_share_a_workspace():
    """Replayed one after the other, in either order; nothing is carried from one to the next."""
    a, b = Chunk([30, 5], [700, 64], 64, seed=8), Chunk([12], [500], 128, seed=9)
    ws = binding.alloc_chunk_workspace(64, 2, 128)
    graphs = []
    for c in (a, b):
        t = c.cuda()
        out = torch.zeros(c.T, c.H, 512, dtype=torch.bfloat16, device="cuda")
        lse = torch.zeros(c.T, c.H, device="cuda")
        binding.mla_chunk_attend(*t, SCALE, out, lse, ws)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            binding.mla_chunk_attend(*t, SCALE, out, lse, ws)
        graphs.append((c, t, out, lse, g))
    for order in ((0, 1), (1, 0), (0, 0), (1, 1)):
        for k in order:
            graphs[k][2].zero_()
            graphs[k][4].replay()
    torch.cuda.synchronize()
    for c, _, out, lse, _ in graphs:
        check_attention(f64(out), f64(lse), *serving.chunk_attend(*c.np(), SCALE), int(c.lens.max()))
    assert binding.mla_get_device_error(ws) == 0


def test_many_short_sequences_and_many_heads_of_one():
    """More sequences than engines, lengths from 1, chunks of 0 to 3 tokens; and one long prompt."""
    g = torch.Generator().manual_seed(10)
    lens = torch.randint(1, 150, (200,), generator=g).tolist()
    n = [min(int(k), L) for k, L in zip(torch.randint(0, 4, (200,), generator=g), lens)]
    c = Chunk(n, lens, 16, seed=11, poison=True)
    out, lse, err = attend(c)
    assert err == 0
    ref = serving.chunk_attend(*c.np(), SCALE)
    check_attention(f64(out), f64(lse), *ref, 150, "many sequences")
    rl = torch.from_numpy(ref[1]).float()
    check_weights(weigh(c, rl, None), c, rl, None, what="many sequences")
    c = Chunk([300], [300], 16, seed=12)
    out, lse, err = attend(c)
    assert err == 0
    check_attention(f64(out), f64(lse), *serving.chunk_attend(*c.np(), SCALE), 300, "one prompt")


def test_a_padded_batch():
    """Sequences of length 0 between others, a table wider than any of them, rows of q past the last."""
    c = Chunk([3, 0, 0, 5, 0], [70, 0, 0, 64, 0], 128, seed=13, before=4, after=6, poison=True, width=40)
    out, lse, err = attend(c)
    assert err == 0
    ref = serving.chunk_attend(*c.np(), SCALE)
    check_attention(f64(out), f64(lse), *ref, 70, "padded")
    rl = torch.from_numpy(ref[1]).float()
    check_weights(weigh(c, rl, None), c, rl, None, what="padded")


def test_evicting_again_and_again_in_one_workspace():
    """Four evictions in place, each on what the one before left."""
    c = Case([1500, 333], [1200, 300], seed=14)
    w, p, ln, tb, ca = (t.cuda() for t in (c.weight, c.pos, c.lens, c.table, c.cache))
    ws = binding.alloc_evict_workspace(2, tb.shape[1])
    weight, pos, lens = c.weight.numpy().copy(), c.pos.numpy().copy(), c.lens.numpy().copy()
    rows = [serving.rows_of(f64(c.cache), c.table.numpy(), b, int(lens[b])) for b in range(2)]
    for keep in ([1200, 300], [700, 290], [64, 63], [1, 0]):
        kept = serving.evict(weight, pos, lens, keep, 3, 20)
        binding.mla_cache_evict(w, p, ln, torch.tensor(keep, dtype=torch.int32, device="cuda"), 3, 20, tb, ca, w, p, ln, ws)
        assert binding.mla_get_device_error(ws) == 0
        for b, s in enumerate(kept):
            rows[b] = rows[b][s]
            weight[b, :len(s)], pos[b, :len(s)] = weight[b, s], pos[b, s]
            lens[b] = len(s)
            assert int(ln[b]) == len(s)
            assert np.array_equal(w[b, :len(s)].cpu().numpy(), weight[b, :len(s)])
            assert np.array_equal(p[b, :len(s)].cpu().numpy(), pos[b, :len(s)])
            assert np.array_equal(serving.rows_of(f64(ca), c.table.numpy(), b, len(s)), rows[b])


def test_operands_on_another_device_or_layout_are_refused():
    c = Chunk([2], [70], 16, seed=15)
    q, offs, cache, table, lens = c.cuda()
    out, lse = torch.empty(2, 16, 512, dtype=torch.bfloat16, device="cuda"), torch.empty(2, 16, device="cuda")
    ws = binding.alloc_chunk_workspace(2, 1, 16)
    with pytest.raises(ValueError):
        binding.mla_chunk_attend(q.transpose(0, 1).contiguous().transpose(0, 1), offs, cache, table, lens, SCALE, out, lse, ws)
    with pytest.raises(ValueError):
        binding.mla_chunk_attend(q, offs.cpu(), cache, table, lens, SCALE, out, lse, ws)
    with pytest.raises(binding.MLAError):            # a workspace that is not 256-byte aligned
        binding.mla_chunk_attend(q, offs, cache, table, lens, SCALE, out, lse, torch.zeros(ws.numel() + 64, dtype=torch.uint8, device="cuda")[16:])
