"""GPU tests of mla_cache_evict (exact) and of a whole serving run over the operators."""
import numpy as np
import pytest
import torch

from mla_latent_kv_25_b200 import binding
from oracle import serving
from tests._serving import SCALE, check_attention, f64, paged

pytestmark = pytest.mark.gpu


class Case:
    def __init__(self, lens, keep, seed, kind="random", width=0, shuffled_pos=False):
        g = torch.Generator().manual_seed(seed)
        self.lens = torch.tensor(lens, dtype=torch.int32)
        self.keep = torch.tensor(keep, dtype=torch.int32)
        self.table, NB = paged(lens, seed, width=width)
        B, S = len(lens), self.table.shape[1] * 64
        w = torch.randn(B, S, generator=g)
        if kind == "ties":
            w = torch.randint(0, 3, (B, S), generator=g).float()
        elif kind == "equal":
            w = torch.full((B, S), 0.25)
        elif kind == "special":
            pick = torch.tensor([float("nan"), float("inf"), -float("inf"), 0.0, -0.0, 1e-45, -1e-45, 3e38, -3e38, 1.0])
            w = pick[torch.randint(0, 10, (B, S), generator=g)]
        elif kind == "close":  # differences in the last bits only
            w = (torch.full((B, S), 1.5).view(torch.int32) + torch.randint(0, 300, (B, S), generator=g).int()).view(torch.float32)
        self.weight = w
        self.pos = torch.arange(S, dtype=torch.int32).repeat(B, 1) + 5
        if shuffled_pos:
            self.pos = torch.stack([torch.randperm(S, generator=g).to(torch.int32) for _ in range(B)])
        self.cache = torch.randn(NB, 64, 576, generator=g).bfloat16()

    def run(self, n_first, n_recent, in_place):
        d = [t.cuda() for t in (self.weight, self.pos, self.lens, self.keep, self.table, self.cache)]
        w, p, ln, kp, tb, ca = d
        nw, np_, nl = (w, p, ln) if in_place else (torch.full_like(w, -3.0), torch.full_like(p, -3), torch.full_like(ln, -3))
        ws = binding.alloc_evict_workspace(len(self.lens), tb.shape[1])
        binding.mla_cache_evict(w, p, ln, kp, n_first, n_recent, tb, ca, nw, np_, nl, ws)
        return nw.cpu(), np_.cpu(), nl.cpu(), ca.cpu(), binding.mla_get_device_error(ws), (w, p, ln, kp, tb)

    def check(self, n_first=4, n_recent=32, in_place=False):
        nw, np_, nl, ca, err, given = self.run(n_first, n_recent, in_place)
        assert err == 0
        kept = serving.evict(self.weight.numpy(), self.pos.numpy(), self.lens.numpy(), self.keep.numpy(), n_first, n_recent)
        bits = lambda t: t.contiguous().view(torch.int32)  # noqa: E731
        want = self.cache.clone()
        for b, slots in enumerate(kept):
            n, L = len(slots), int(self.lens[b])
            s = torch.from_numpy(slots)
            assert int(nl[b]) == n
            assert torch.equal(bits(nw[b, :n]), bits(self.weight[b][s])) and torch.equal(np_[b, :n], self.pos[b][s])
            assert bool((nw[b, n:L] == 0).all()) and bool((np_[b, n:L] == -1).all())
            rest_w, rest_p = (self.weight[b, L:], self.pos[b, L:]) if in_place else (torch.full_like(self.weight[b, L:], -3.0),
                                                                                     torch.full_like(self.pos[b, L:], -3))
            assert torch.equal(bits(nw[b, L:]), bits(rest_w)) and torch.equal(np_[b, L:], rest_p)
            to = torch.arange(n)
            want[self.table[b, to // 64].long(), to % 64] = self.cache[self.table[b, s // 64].long(), s % 64]
        assert torch.equal(ca.view(torch.int16), want.view(torch.int16))   # every other row as it was
        if not in_place:
            for t, was in zip(given, (self.weight, self.pos, self.lens, self.keep, self.table)):
                assert torch.equal(t.cpu().view(torch.int32), was.view(torch.int32))


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("lens,keep", [
    ([1], [1]), ([1], [0]), ([300], [128]), ([63, 64, 65, 128, 129], [32, 63, 64, 65, 1]), ([5, 0, 70], [9, 3, 70]),
    ([100, 100], [-4, 2 ** 31 - 1]), ([2000, 1, 1025, 4097], [1000, 1, 1024, 40]), ([40], [20]), ([37], [36])])
def test_evict_lengths_and_budgets(lens, keep, in_place):
    Case(lens, keep, seed=sum(lens)).check(in_place=in_place)


@pytest.mark.parametrize("kind", ["ties", "equal", "special", "close"])
@pytest.mark.parametrize("first,recent", [(0, 0), (4, 32), (200, 200), (0, 10 ** 9), (2 ** 31 - 1, 0)])
def test_evict_orders(kind, first, recent):
    Case([700, 130, 1500], [300, 64, 700], seed=3, kind=kind).check(first, recent)


@pytest.mark.parametrize("in_place", [False, True])
def test_evict_after_positions_were_shuffled(in_place):
    """After an earlier eviction positions no longer follow the slots."""
    Case([900, 400], [450, 100], seed=4, shuffled_pos=True).check(16, 100, in_place)


def test_evict_a_long_sequence():
    Case([40000, 20], [17000, 10], seed=5).check(4, 128)
    Case([140001], [70001], seed=6, kind="ties").check(4, 128)


@pytest.mark.parametrize("width", [300, 1100, 8000])
def test_evict_in_wide_tables(width):
    """The table's width, not the lengths, sets how a sequence is shared out: few CTAs, many,
    and too wide for the keys to stay in shared memory."""
    Case([700, 19000], [300, 9000], seed=21, kind="ties", width=width).check(4, 32)
    Case([5000], [1], seed=22, width=width, shuffled_pos=True).check(0, 7, in_place=True)


@pytest.mark.parametrize("first,recent", [(4, 32), (0, 10 ** 9)])
@pytest.mark.parametrize("kind", ["random", "ties", "equal", "special", "close"])
@pytest.mark.parametrize("width", [300, 8000])
def test_evict_orders_in_wide_tables(width, kind, first, recent):
    """Clusters with the keys kept (300 blocks) and read again (8000), in place: protected slots
    that compete, ties cut between CTAs, moves whose weights follow with the rows."""
    Case([5000, 19100], [2501, 9001], seed=31, kind=kind, width=width, shuffled_pos=True).check(first, recent, in_place=True)


@pytest.mark.parametrize("weights_in_place", [False, True])
def test_evict_with_one_array_in_place(weights_in_place):
    c = Case([700, 64, 3001], [300, 64, 1500], seed=33, shuffled_pos=True)
    w, p, ln, kp, tb, ca = [t.cuda() for t in (c.weight, c.pos, c.lens, c.keep, c.table, c.cache)]
    nw, np_ = (w, torch.full_like(p, -3)) if weights_in_place else (torch.full_like(w, -3.0), p)
    ws = binding.alloc_evict_workspace(3, tb.shape[1])
    binding.mla_cache_evict(w, p, ln, kp, 4, 32, tb, ca, nw, np_, ln, ws)
    assert binding.mla_get_device_error(ws) == 0
    kept = serving.evict(c.weight.numpy(), c.pos.numpy(), c.lens.numpy(), c.keep.numpy(), 4, 32)
    for b, slots in enumerate(kept):
        n, L, s = len(slots), int(c.lens[b]), torch.from_numpy(slots)
        assert int(ln[b]) == n
        assert torch.equal(nw[b, :n].cpu(), c.weight[b][s]) and torch.equal(np_[b, :n].cpu(), c.pos[b][s])
        assert bool((nw[b, n:L] == 0).all()) and bool((np_[b, n:L] == -1).all())


def test_evict_many_sequences():
    g = torch.Generator().manual_seed(7)
    lens = torch.randint(0, 200, (300,), generator=g).tolist()
    keep = torch.randint(0, 200, (300,), generator=g).tolist()
    Case(lens, keep, seed=8, width=5).check(2, 5)


def test_evict_bad_blocks_and_lengths():
    c = Case([256, 256], [128, 128], seed=9)
    c.table[0, 3] = 10 ** 6
    nw, np_, nl, ca, err, _ = c.run(0, 0, False)
    assert err == binding.DEVERR_BAD_BLOCK
    kept = serving.evict(c.weight.numpy(), c.pos.numpy(), c.lens.numpy(), c.keep.numpy(), 0, 0)
    want = c.cache.clone()
    for b, slots in enumerate(kept):
        for to, s in enumerate(slots.tolist()):
            if c.table[b, s // 64] < c.cache.shape[0]:
                want[int(c.table[b, to // 64]), to % 64] = c.cache[int(c.table[b, s // 64]), s % 64]
    assert torch.equal(ca, want)
    c = Case([64, 64], [10, 10], seed=10)
    c.lens[0] = 65
    nw, np_, nl, ca, err, _ = c.run(0, 0, False)
    assert err == binding.DEVERR_SEQ_TOO_LONG and nl.tolist() == [10, 10]


def test_evict_in_a_graph():
    c = Case([500, 90], [200, 64], seed=11)
    w, p, ln, kp, tb, ca = (t.cuda() for t in (c.weight, c.pos, c.lens, c.keep, c.table, c.cache))
    nw, np_, nl = torch.zeros_like(w), torch.zeros_like(p), torch.zeros_like(ln)
    ws = binding.alloc_evict_workspace(2, tb.shape[1])
    binding.mla_cache_evict(w, p, ln, kp, 4, 32, tb, ca, nw, np_, nl, ws)
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        binding.mla_cache_evict(w, p, ln, kp, 4, 32, tb, ca, nw, np_, nl, ws)
    d = Case([400, 128], [150, 20], seed=12, width=tb.shape[1])
    w.copy_(d.weight.cuda())
    ln.copy_(d.lens.cuda())
    kp.copy_(d.keep.cuda())
    g.replay()
    torch.cuda.synchronize()
    kept = serving.evict(d.weight.numpy(), d.pos.numpy(), d.lens.numpy(), d.keep.numpy(), 4, 32)
    for b, s in enumerate(kept):
        assert int(nl[b]) == len(s) and torch.equal(np_[b, :len(s)].cpu(), d.pos[b][torch.from_numpy(s)])


def test_a_request_from_prompt_to_decode_after_eviction():
    """Rotate and append two prompts in chunks, attend, accumulate weights, evict, append one
    more token at a slot that is not its position, decode: against FP64 at every step."""
    H, chunks, B = 32, [40, 33, 60], 2
    rng = np.random.default_rng(20)
    freqs = binding.mla_rope_freqs(64, scaling="yarn", factor=8.0)
    fnp = f64(freqs)
    table = torch.tensor([[3, 0, 5], [1, 4, 2]], dtype=torch.int32)
    cache = torch.zeros(7, 64, 576, dtype=torch.bfloat16, device="cuda")
    tb = table.cuda()
    weight, slot_pos = torch.zeros(B, 192, device="cuda"), torch.full((B, 192), -1, dtype=torch.int32, device="cuda")
    ws = binding.alloc_chunk_workspace(B * max(chunks), B, H)
    done = 0

    def tokens(n):
        """Projections of n new tokens per sequence: latent rows and queries, bf16."""
        rows = torch.from_numpy(rng.standard_normal((B * n, 576)) * np.r_[np.full(512, 0.05), np.ones(64)]).bfloat16()
        q = torch.from_numpy(rng.standard_normal((B * n, H, 576))).bfloat16()
        return rows.cuda(), q.cuda()

    def step(n, slots, positions):
        rows, q = tokens(n)
        seq = torch.arange(B, dtype=torch.int32).repeat_interleave(n).cuda()
        binding.mla_cache_append_rope(rows[:, :512], rows[:, 512:], seq, slots, positions, freqs, tb, cache,
                                      slot_pos=slot_pos)
        raw = f64(q[..., 512:])
        binding.mla_rope(q[..., 512:], positions, freqs, q[..., 512:])
        ref = serving.rope(raw, positions.cpu().numpy(), fnp)
        assert np.abs(f64(q[..., 512:]) - ref).max() <= 2.0 ** -8 * np.abs(ref).max() + 2.0 ** -16
        return q

    for n in chunks:
        at = (torch.arange(n, dtype=torch.int32) + done).repeat(B).cuda()
        q = step(n, at, at)
        done += n
        lens = torch.full((B,), done, dtype=torch.int32, device="cuda")
        offs = torch.arange(B + 1, dtype=torch.int32, device="cuda") * n
        out, lse = torch.empty(B * n, H, 512, dtype=torch.bfloat16, device="cuda"), torch.empty(B * n, H, device="cuda")
        binding.mla_chunk_attend(q, offs, cache, tb, lens, SCALE, out, lse, ws)
        args = (f64(q), offs.cpu().numpy(), f64(cache), table.numpy(), lens.cpu().numpy())
        ref, rlse, mass, mag = serving.chunk_attend(*args, SCALE)
        check_attention(f64(out), f64(lse), ref, rlse, mass, mag, done, f"chunk of {n}")
        before = f64(weight)
        binding.mla_cache_weigh(q, offs, lse, cache, tb, lens, SCALE, weight, weight)
        add, _, _ = serving.weigh(args[0], args[1], f64(lse), *args[2:], SCALE)
        assert np.allclose(f64(weight), before + add, rtol=2e-4, atol=1e-6)
    assert binding.mla_get_device_error(ws) == 0 and binding.mla_cache_get_error() == 0

    keep = torch.tensor([64, 50], dtype=torch.int32, device="cuda")
    kept = serving.evict(f64(weight), slot_pos.cpu().numpy(), lens.cpu().numpy(), keep.cpu().numpy(), 4, 16)
    old = f64(cache)
    ew = binding.alloc_evict_workspace(B, 3)
    binding.mla_cache_evict(weight, slot_pos, lens, keep, 4, 16, tb, cache, weight, slot_pos, lens, ew)
    assert binding.mla_get_device_error(ew) == 0 and lens.tolist() == [64, 50]
    for b, s in enumerate(kept):
        assert slot_pos[b, :len(s)].tolist() == s.tolist()      # position = slot before the first eviction
        assert np.array_equal(serving.rows_of(f64(cache), table.numpy(), b, len(s)), old[table.numpy()[b, s // 64], s % 64])

    q = step(1, lens.clone(), torch.full((B,), done, dtype=torch.int32, device="cuda"))
    lens += 1
    assert slot_pos[0, 64].item() == done and slot_pos[1, 50].item() == done
    out, lse = torch.empty(B, H, 512, dtype=torch.bfloat16, device="cuda"), torch.empty(B, H, device="cuda")
    dw = binding.alloc_workspace(B, H)
    binding.mla_decode(q, cache, tb, lens, SCALE, out, lse, dw)
    assert binding.mla_get_device_error(dw) == 0
    args = (f64(q), np.arange(B + 1), f64(cache), table.numpy(), lens.cpu().numpy())
    check_attention(f64(out), f64(lse), *serving.chunk_attend(*args, SCALE), 65, "decode after eviction")
