"""GPU parity of mla_chunk_attend and mla_cache_weigh against the FP64 definition."""
import numpy as np
import pytest
import torch

from mla_latent_kv_25_b200 import binding
from oracle import serving
from tests._serving import SCALE, Chunk, check_attention, f64, score_slack

pytestmark = pytest.mark.gpu

# tokens per sequence, cached rows per sequence, heads
SHAPES = {
    "one token": ([1], [1], 16),
    "tiny": ([5], [261], 16),
    "block edges": ([1, 2, 3, 4, 5], [63, 64, 65, 127, 129], 128),
    "pass edges": ([3, 2, 1], [255, 256, 257], 128),
    "empty sequences": ([0, 3, 0, 2, 0], [40, 70, 0, 2, 5], 64),
    "whole prompt": ([130], [130], 32),
    "odd heads": ([7, 1, 12], [300, 33, 64], 48),
    "112 heads": ([5, 3], [90, 700], 112),
    "80 heads, many tokens": ([40, 9], [100, 1000], 80),
    "more tokens than rows": ([6, 4], [2, 0], 128),
    "long": ([3], [5000], 128),
}


def attend(c, num_splits=0, scale=SCALE, stream=None):
    q, offs, cache, table, lens = c.cuda()
    out = torch.full((c.T, c.H, 512), float("nan"), dtype=torch.bfloat16, device="cuda")
    lse = torch.full((c.T, c.H), float("nan"), device="cuda")
    ws = binding.alloc_chunk_workspace(c.T, c.B, c.H, num_splits)
    binding.mla_chunk_attend(q, offs, cache, table, lens, scale, out, lse, ws, num_splits=num_splits)
    return out, lse, binding.mla_get_device_error(ws)


def check(c, num_splits=0, scale=SCALE, what=""):
    out, lse, err = attend(c, num_splits, scale)
    assert err == 0, f"device error bits {err:#x}"
    q, offs, cache, table, lens = c.np()
    ref, rlse, mass, mag = serving.chunk_attend(q, offs, cache, table, lens, scale)
    check_attention(f64(out), f64(lse), ref, rlse, mass, mag, int(lens.max()), what)
    return out, lse


@pytest.mark.parametrize("name", SHAPES)
def test_chunk_matches_the_definition(name):
    n, lens, H = SHAPES[name]
    check(Chunk(n, lens, H, seed=len(name), before=2, after=3, poison=True), what=name)


@pytest.mark.parametrize("num_splits", [1, 2, 3, 5, 36, 64, 200])
def test_chunk_split_counts(num_splits):
    check(Chunk([9, 1, 4], [1000, 63, 300], 64, seed=4), num_splits, what=f"splits={num_splits}")


@pytest.mark.parametrize("num_splits", [0, 1, 13, 37, 64, 65])
@pytest.mark.parametrize("name", ["equal", "ragged", "one_long", "empty"])
def test_chunk_tiles_that_stay_whole(name, num_splits):
    """Several tiles to an engine: cuts that move to the ends of tiles, all of them or some, empty
    ranges, more engines than that is done for, sequences without queries or without a cache."""
    g = torch.Generator().manual_seed(17)
    n, lens = {"equal": ([4] * 40, [250] * 40),
               "ragged": (torch.randint(1, 7, (48,), generator=g).tolist(), torch.randint(8, 700, (48,), generator=g).tolist()),
               "one_long": ([2] * 30, [5000] + [130] * 29),
               "empty": ([2, 0, 3, 1, 0] * 8, [100, 50, 0, 300, 0] * 8)}[name]
    lens = [max(a, b) if b else 0 for a, b in zip(n, lens)]
    check(Chunk(n, lens, 128, seed=num_splits), num_splits, what=f"{name}, splits={num_splits}")


@pytest.mark.parametrize("scale", [0.0, -0.3, 3.0])
def test_chunk_scales(scale):
    """Uniform, inverted and sharp softmax."""
    check(Chunk([4, 6], [200, 77], 32, seed=5, q_std=2.0), scale=scale, what=f"scale={scale}")


def test_chunk_rows_do_not_depend_on_placement_or_company():
    """Another physical placement gives the same bits."""
    c = Chunk([5, 8], [400, 90], 128, seed=6)
    a, la, _ = attend(c, num_splits=3)
    perm = torch.randperm(c.cache.shape[0], generator=torch.Generator().manual_seed(1))
    moved = torch.empty_like(c.cache)
    moved[perm] = c.cache
    c.cache = moved
    c.table = torch.where(c.table >= 0, perm[c.table.clamp(min=0).long()].to(torch.int32), c.table)
    b, lb, _ = attend(c, num_splits=3)
    assert torch.equal(a, b) and torch.equal(la, lb)


def test_chunk_of_one_token_is_decode():
    c = Chunk([1] * 5, [64, 100, 1, 513, 30], 128, seed=7)
    out, lse = check(c, what="decode")
    q, offs, cache, table, lens = c.cuda()
    o2, l2 = torch.empty_like(out), torch.empty_like(lse)
    ws = binding.alloc_workspace(5, 128)
    binding.mla_decode(q, cache, table, lens, SCALE, o2, l2, ws)
    ref, rlse, mass, mag = serving.chunk_attend(*c.np(), SCALE)
    check_attention(f64(o2), f64(l2), ref, rlse, mass, mag, 513, "mla_decode on the same rows")


def test_chunk_reports_bad_ids_lengths_and_offsets():
    c = Chunk([2, 2, 2], [100, 70, 90], 16, seed=8)
    c.table[1, 1] = 10 ** 6
    out, lse, err = attend(c)
    assert err == binding.DEVERR_BAD_BLOCK
    good = Chunk([2, 2, 2], [100, 70, 90], 16, seed=8)
    ref, rlse, mass, mag = serving.chunk_attend(*good.np(), SCALE)
    for t in (0, 1, 4, 5):      # the other sequences are right
        check_attention(f64(out)[t], f64(lse)[t], ref[t], rlse[t], mass[t], mag[t], 100, "beside a bad id")
    # its own tokens see the rows of the good block alone
    c.lens[1] = 64
    for j in range(2):
        s = f64(c.q)[2 + j] @ serving.rows_of(f64(c.cache), c.table.numpy(), 1, 64).T * SCALE
        z = np.exp(s).sum(1)
        assert np.allclose(f64(lse)[2 + j], np.log(z), atol=1e-3)
    long = Chunk([1, 1], [64, 64], 16, seed=9)
    long.lens[0] = 65
    assert attend(long)[2] == binding.DEVERR_SEQ_TOO_LONG
    back = Chunk([2, 2, 2], [100, 70, 90], 16, seed=8)
    back.offs = torch.tensor([0, 4, 2, 6], dtype=torch.int32)
    assert attend(back)[2] & binding.DEVERR_SEQ_TOO_LONG
    far = Chunk([2, 2], [100, 70], 16, seed=8)
    far.offs = torch.tensor([0, 2, 9], dtype=torch.int32)
    out, lse, err = attend(far)
    assert err & binding.DEVERR_SEQ_TOO_LONG and bool(torch.isfinite(out[:2]).all()) and bool(out[2:].isnan().all())


def test_chunk_over_an_fp8_cache():
    """Codes and block scales: the definition on bf16(code * scale), the value the widened row holds."""
    c = Chunk([5, 0, 40], [300, 64, 100], 48, seed=20, before=1, after=1)
    NB = c.cache.shape[0]
    codes = torch.zeros(NB, 64, 512, dtype=torch.uint8, device="cuda")
    k_rope = torch.zeros(NB, 64, 64, dtype=torch.bfloat16, device="cuda")
    scale = torch.zeros(NB, device="cuda")
    binding.mla_cache_quantize_fp8(c.cache.cuda(), torch.arange(NB, dtype=torch.int32, device="cuda"), codes, k_rope, scale)
    assert binding.mla_cache_get_error() == 0
    lat = codes.cpu().view(torch.float8_e4m3fn).float() * scale.cpu()[:, None, None]
    c.cache = torch.cat([lat.bfloat16(), k_rope.cpu()], -1)
    q, offs, _, table, lens = c.cuda()
    out = torch.full((c.T, c.H, 512), float("nan"), dtype=torch.bfloat16, device="cuda")
    lse = torch.full((c.T, c.H), float("nan"), device="cuda")
    ws = binding.alloc_chunk_workspace(c.T, c.B, c.H, fp8_max_blocks=table.shape[1])
    binding.mla_chunk_attend(q, offs, codes, table, lens, SCALE, out, lse, ws, k_rope=k_rope, block_scale=scale)
    assert binding.mla_get_device_error(ws) == 0
    check_attention(f64(out), f64(lse), *serving.chunk_attend(*c.np(), SCALE), 300, "fp8 cache")
    with pytest.raises(binding.MLAError):
        binding.mla_chunk_attend(q, offs, codes, table, lens, SCALE, out, lse, binding.alloc_chunk_workspace(c.T, c.B, c.H),
                                 k_rope=k_rope, block_scale=scale)
    bad = table.clone()
    bad[2, 0] = -1
    binding.mla_chunk_attend(q, offs, codes, bad, lens, SCALE, out, lse, ws, k_rope=k_rope, block_scale=scale)
    assert binding.mla_get_device_error(ws) == binding.DEVERR_BAD_BLOCK


def test_chunk_in_a_graph_and_on_another_stream():
    c = Chunk([6, 3], [300, 200], 64, seed=10)
    want, wlse, _ = attend(c)
    q, offs, cache, table, lens = c.cuda()
    out, lse = torch.zeros_like(want), torch.zeros_like(wlse)
    ws = binding.alloc_chunk_workspace(c.T, c.B, c.H)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    binding.mla_chunk_attend(q, offs, cache, table, lens, SCALE, out, lse, ws, stream=side)
    side.synchronize()
    assert torch.equal(out, want) and torch.equal(lse, wlse)
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        binding.mla_chunk_attend(q, offs, cache, table, lens, SCALE, out, lse, ws)
    d = Chunk([2, 7], [129, 290], 64, seed=11)     # other lengths and values in the same buffers
    assert d.T == c.T and d.cache.shape[0] <= c.cache.shape[0] and d.table.shape == c.table.shape
    for dst, src in zip((q, offs, cache[:d.cache.shape[0]], table, lens), d.cuda()):
        dst.copy_(src)
    for _ in range(2):
        out.fill_(float("nan"))
        g.replay()
    torch.cuda.synchronize()
    ref, rlse, mass, mag = serving.chunk_attend(*d.np(), SCALE)
    check_attention(f64(out), f64(lse), ref, rlse, mass, mag, 290, "replayed")


# ------------------------------------------------------------------------------------------ weigh

def weigh(c, lse, weight, out=None, scale=SCALE):
    q, offs, cache, table, lens = c.cuda()
    out = torch.full((c.B, table.shape[1] * 64), -7.0, device="cuda") if out is None else out
    binding.mla_cache_weigh(q, offs, lse.cuda(), cache, table, lens, scale, weight, out)
    return out


def check_weights(got, c, lse, weight, scale=SCALE, what="", untouched=-7.0):
    """exp's argument is off by its score's error and one rounding of its terms; exp2, the
    conversion to base 2 and the sum of n*H terms add 2^-22, 2^-23 |argument| and 2^-24 each."""
    q, offs, cache, table, lens = c.np()
    add, mag, arg = serving.weigh(q, offs, f64(lse), cache, table, lens, scale)
    w = np.zeros_like(add) if weight is None else f64(weight)
    live = np.arange(add.shape[1])[None] < lens[:, None]
    terms = (max(c.n) * c.H + 16) * 2.0 ** -24
    tol = add * (score_slack(mag) + 2.0 ** -21 * (1 + arg) + terms)[:, None] + 2.0 ** -23 * np.abs(w) + 1e-30
    off = np.abs(f64(got) - (w + add))
    assert (off <= tol)[live].all(), f"{what}: {np.max((off - tol)[live]):.3e} over the bound"
    assert (f64(got)[~live] == untouched).all(), f"{what}: slots past the sequences were written"


@pytest.mark.parametrize("name", SHAPES)
def test_weights_match_the_definition(name):
    n, lens, H = SHAPES[name]
    c = Chunk(n, lens, H, seed=len(name) + 50, before=1, after=2, poison=True)
    q, offs, cache, table, ln = c.np()
    rlse = serving.chunk_attend(q, offs, cache, table, ln, SCALE)[1]
    lse = torch.from_numpy(rlse).float()
    w = torch.rand(c.B, c.table.shape[1] * 64, generator=torch.Generator().manual_seed(1))
    check_weights(weigh(c, lse, w.cuda()), c, lse, w, what=name)
    check_weights(weigh(c, lse, None), c, lse, None, what=name + ", no input")


def test_weights_accumulate_in_place_and_skip_infinite_rows():
    c = Chunk([4, 2], [150, 64], 32, seed=60)
    lse = torch.from_numpy(serving.chunk_attend(*c.np(), SCALE)[1]).float()
    lse[1, 3:9] = float("inf")
    lse[5] = float("inf")
    w = torch.rand(c.B, c.table.shape[1] * 64, generator=torch.Generator().manual_seed(2))
    once = weigh(c, lse, w.cuda())
    buf = w.cuda()
    weigh(c, lse, buf, buf)
    live = torch.arange(w.shape[1])[None] < c.lens[:, None]
    assert torch.equal(buf.cpu()[live], once.cpu()[live]) and torch.equal(buf.cpu()[~live], w[~live])
    check_weights(once, c, lse, w, what="infinite lse")


def test_weights_of_no_queries_copy_the_input():
    c = Chunk([0, 0], [70, 10], 16, seed=61)
    w = torch.rand(2, c.table.shape[1] * 64, generator=torch.Generator().manual_seed(3))
    got = weigh(c, torch.zeros(c.T, 16), w.cuda())
    check_weights(got, c, torch.zeros(c.T, 16), w, what="no queries")


def test_weights_beside_a_bad_block():
    c = Chunk([1, 1], [130, 100], 16, seed=62)
    lse = torch.from_numpy(serving.chunk_attend(*c.np(), SCALE)[1]).float()
    w = torch.rand(2, c.table.shape[1] * 64, generator=torch.Generator().manual_seed(4))
    want = weigh(c, lse, w.cuda())
    assert binding.mla_cache_get_error() == 0
    c.table[0, 1] = -1
    got = weigh(c, lse, w.cuda())
    assert binding.mla_cache_get_error() == binding.DEVERR_BAD_BLOCK
    assert torch.equal(got.cpu()[0, 64:128], w[0, 64:128])
    assert torch.equal(got[1], want[1]) and torch.equal(got[0, :64], want[0, :64]) and torch.equal(got[0, 128:], want[0, 128:])


def test_weights_repeat_bit_for_bit():
    c = Chunk([40, 3], [3000, 500], 128, seed=63)
    lse = torch.zeros(c.T, 128) + 8.0
    a, b = weigh(c, lse, None), weigh(c, lse, None)
    assert torch.equal(a, b)


def test_refusals_of_the_binding():
    c = Chunk([2, 1], [70, 10], 16, seed=64)
    q, offs, cache, table, lens = c.cuda()
    out, lse = torch.empty(3, 16, 512, dtype=torch.bfloat16, device="cuda"), torch.empty(3, 16, device="cuda")
    ws = binding.alloc_chunk_workspace(3, 2, 16)
    ok = [q, offs, cache, table, lens, SCALE, out, lse, ws]
    for i, bad in [(0, q[:, :, :512]), (0, q.float()), (0, q.cpu()), (1, offs[:2]), (1, offs.long()), (2, cache[:, :32]),
                   (3, table[:1]), (4, lens[:1]), (6, out[:2]), (6, out.float()), (7, lse[:, :8]), (8, ws.float())]:
        with pytest.raises((TypeError, ValueError)):
            binding.mla_chunk_attend(*(ok[:i] + [bad] + ok[i + 1:]))
    with pytest.raises(binding.MLAError):
        binding.mla_chunk_attend(*(ok[:8] + [ws[:128]]))
    w = torch.zeros(2, table.shape[1] * 64, device="cuda")
    with pytest.raises(ValueError):
        binding.mla_cache_weigh(q, offs, lse, cache, table, lens, SCALE, w[:, :64], w)
    with pytest.raises(TypeError):
        binding.mla_cache_weigh(q, offs, lse, cache, table, lens, SCALE, w.double(), w)
