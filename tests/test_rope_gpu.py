"""GPU parity of mla_rope and mla_cache_append_rope against the FP64 rotation."""
import numpy as np
import pytest
import torch

from mla_latent_kv_25_b200 import binding
from oracle import serving
from tests._serving import HALF, f64, paged

pytestmark = pytest.mark.gpu


def check(got, x, pos, freqs, mscale, half, inverse=False, what=""):
    """Cosine and sine are within 2^-22 of the exact ones (argument rounded once, library
    function within 2 units), two products and a sum in fp32, one rounding to bf16."""
    ref = serving.rope(x, pos, freqs, mscale, half, inverse)
    r = x.shape[-1] // 2
    a, b = (x[..., :r], x[..., r:]) if half else (x[..., 0::2], x[..., 1::2])
    m = (np.abs(a) + np.abs(b)) * abs(mscale)
    mag = np.concatenate([m, m], -1) if half else np.stack([m, m], -1).reshape(x.shape)
    off = np.abs(got - ref)
    tol = HALF * np.abs(ref) + 2.0 ** -20 * mag + 1e-38
    assert (off <= tol).all(), f"{what}: {np.max(off - tol):.3e} over the bound"


def positions(T, seed):
    g = torch.Generator().manual_seed(seed)
    pos = torch.randint(0, 131072, (T,), generator=g, dtype=torch.int32)
    edge = torch.tensor([0, 1, 2 ** 31 - 1, -1, -131071], dtype=torch.int32)
    pos[:min(T, 5)] = edge[:min(T, 5)]
    return pos


@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("T,H,rot", [(1, 1, 64), (1, 128, 64), (7, 16, 64), (3, 5, 2), (5, 3, 6), (33, 128, 64),
                                     (4, 7, 96), (2, 3, 256), (300, 9, 48)])
def test_rope_dense(T, H, rot, half):
    g = torch.Generator().manual_seed(T * 1000 + H + rot)
    x = torch.randn(T, H, rot, generator=g).bfloat16()
    pos = positions(T, rot)
    freqs = binding.mla_rope_freqs(rot, scaling="yarn", factor=40.0)
    y = torch.full((T, H, rot), 7.0, dtype=torch.bfloat16, device="cuda")
    got = binding.mla_rope(x.cuda(), pos.cuda(), freqs, y, mscale=1.25, layout="half" if half else "interleaved")
    check(f64(got), f64(x), pos.numpy(), f64(freqs), 1.25, half)


@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("pad,off", [(128, 128), (1, 1), (3, 2), (8, 8), (10, 4)])
def test_rope_of_part_of_a_head(pad, off, half):
    """The rotated part anywhere in longer heads, aligned to 16 bytes or not; all else stays."""
    T, H, rot = 6, 11, 64
    g = torch.Generator().manual_seed(off)
    x = torch.randn(T, H, rot + pad, generator=g).bfloat16()
    pos = positions(T, off)
    freqs = binding.mla_rope_freqs(rot)
    xd = x.cuda()
    y = torch.randn(T, H, 576, generator=g).bfloat16()
    yd = y.cuda()
    binding.mla_rope(xd[..., off:off + rot], pos.cuda(), freqs, yd[..., 512:], layout="half" if half else "interleaved")
    check(f64(yd[..., 512:]), f64(x[..., off:off + rot]), pos.numpy(), f64(freqs), 1.0, half)
    assert torch.equal(yd[..., :512].cpu(), y[..., :512]) and torch.equal(xd.cpu(), x)
    # in place
    part = xd[..., off:off + rot]
    binding.mla_rope(part, pos.cuda(), freqs, part, layout="half" if half else "interleaved")
    check(f64(part), f64(x[..., off:off + rot]), pos.numpy(), f64(freqs), 1.0, half)
    rest = [i for i in range(rot + pad) if not off <= i < off + rot]
    assert torch.equal(xd.cpu()[..., rest], x[..., rest])


def test_rope_strides_head_major_and_shared_rows():
    T, H, rot = 9, 4, 64
    g = torch.Generator().manual_seed(3)
    x = torch.randn(H, T, rot, generator=g).bfloat16()
    pos, freqs = positions(T, 4), binding.mla_rope_freqs(rot)
    y = torch.empty(H, T, rot, dtype=torch.bfloat16, device="cuda")
    binding.mla_rope(x.cuda().transpose(0, 1), pos.cuda(), freqs, y.transpose(0, 1))
    check(f64(y.transpose(0, 1)), f64(x.transpose(0, 1)), pos.numpy(), f64(freqs), 1.0, False)
    one = x[:1].transpose(0, 1)                      # one key row for all heads: stride 0
    y2 = torch.empty(T, H, rot, dtype=torch.bfloat16, device="cuda")
    binding.mla_rope(one.cuda().expand(T, H, rot), pos.cuda(), freqs, y2)
    check(f64(y2), f64(one.expand(T, H, rot)), pos.numpy(), f64(freqs), 1.0, False)


@pytest.mark.parametrize("half", [False, True])
def test_inverse_rotation_is_the_gradient(half):
    """d(g . R x)/dx = R^-1 g for the same mscale: against the formula and against differences
    of the FP64 form (linear in x, so one difference is exact up to its rounding)."""
    T, H, rot = 4, 3, 64
    rng = np.random.default_rng(5)
    gr = torch.from_numpy(rng.standard_normal((T, H, rot))).bfloat16()
    pos, freqs = positions(T, 6), binding.mla_rope_freqs(rot, scaling="ntk", factor=4.0)
    y = torch.empty(T, H, rot, dtype=torch.bfloat16, device="cuda")
    lay = "half" if half else "interleaved"
    binding.mla_rope(gr.cuda(), pos.cuda(), freqs, y, mscale=0.75, layout=lay, inverse=True)
    check(f64(y), f64(gr), pos.numpy(), f64(freqs), 0.75, half, inverse=True)
    x = rng.standard_normal((T, H, rot))
    for t, h, r in [(0, 0, 0), (1, 2, 33), (2, 1, 63), (3, 0, 17)]:
        up, dn = x.copy(), x.copy()
        up[t, h, r] += 0.5
        dn[t, h, r] -= 0.5
        diff = (f64(gr) * (serving.rope(up, pos.numpy(), f64(freqs), 0.75, half)
                           - serving.rope(dn, pos.numpy(), f64(freqs), 0.75, half))).sum()
        big = np.abs(f64(gr)[t, h]).max() * 0.75 * 2
        assert abs(f64(y)[t, h, r] - diff) <= HALF * abs(diff) + 2.0 ** -20 * big + 1e-9


def test_rope_scores_depend_on_distance_only():
    g = torch.Generator().manual_seed(8)
    q, k = (torch.randn(1, 1, 64, generator=g).bfloat16().cuda().expand(200, 1, 64) for _ in range(2))
    pos = torch.arange(200, dtype=torch.int32, device="cuda") * 601
    freqs = binding.mla_rope_freqs(64, scaling="linear", factor=2.0)
    a, b = torch.empty(200, 1, 64, dtype=torch.bfloat16, device="cuda"), torch.empty(200, 1, 64, dtype=torch.bfloat16, device="cuda")
    binding.mla_rope(q, pos + 77, freqs, a)
    binding.mla_rope(k, pos, freqs, b)
    s = (a.double() * b.double()).sum(-1)
    # both sides rounded to bf16: 2 * 2^-8 of the sum of magnitudes, bounded by the norms
    bound = 2 * HALF * (1 + HALF) * float(a[0].double().norm() * b[0].double().norm()) * 1.01
    assert float(s.max() - s.min()) <= 2 * bound


# ------------------------------------------------------------------------------------- append

@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("joint", [False, True])
def test_append_rope_places_rows(half, joint):
    lens = [70, 1, 200]
    table, NB = paged(lens, 11)
    g = torch.Generator().manual_seed(12)
    cache = torch.randn(NB, 64, 576, generator=g).bfloat16()
    seq = torch.tensor([0, 0, 1, 2, 2, 2], dtype=torch.int32)
    slot = torch.tensor([69, 3, 0, 199, 64, 63], dtype=torch.int32)
    pos = torch.tensor([131071, 12, 2 ** 31 - 1, 0, 99999, -5], dtype=torch.int32)
    rows = torch.randn(6, 640 if joint else 576, generator=g).bfloat16()
    c_kv, k_r = rows[:, :512], rows[:, 512:576]
    dev = rows.cuda()
    ck, kr = (dev[:, :512], dev[:, 512:576]) if joint else (c_kv.contiguous().cuda(), k_r.contiguous().cuda())
    freqs = binding.mla_rope_freqs(64, scaling="yarn", factor=40.0)
    sp = torch.full((3, table.shape[1] * 64), -9, dtype=torch.int32, device="cuda")
    out = cache.cuda()
    binding.mla_cache_append_rope(ck, kr, seq.cuda(), slot.cuda(), pos.cuda(), freqs, table.cuda(), out, slot_pos=sp,
                                  mscale=1.5, layout="half" if half else "interleaved")
    assert binding.mla_cache_get_error() == 0
    want_sp = torch.full_like(sp, -9).cpu()
    touched = torch.zeros(NB, 64, dtype=torch.bool)
    for t in range(6):
        b, s = int(seq[t]), int(slot[t])
        blk = int(table[b, s // 64])
        touched[blk, s % 64] = True
        want_sp[b, s] = pos[t]
        assert torch.equal(out[blk, s % 64, :512].cpu(), c_kv[t])
        check(f64(out[blk, s % 64, 512:])[None, None], f64(k_r[t])[None, None], pos[t:t + 1].numpy(), f64(freqs), 1.5, half)
    assert torch.equal(out.cpu()[~touched], cache[~touched])
    assert torch.equal(sp.cpu(), want_sp)


def test_append_rope_equals_append_at_position_slot():
    """The plain rotation at position = slot is mla_cache_append's, up to one rounding."""
    lens = [150]
    table, NB = paged(lens, 13)
    g = torch.Generator().manual_seed(14)
    ck, kr = torch.randn(150, 512, generator=g).bfloat16().cuda(), torch.randn(150, 64, generator=g).bfloat16().cuda()
    seq = torch.zeros(150, dtype=torch.int32, device="cuda")
    at = torch.arange(150, dtype=torch.int32, device="cuda")
    a, b = torch.zeros(NB, 64, 576, dtype=torch.bfloat16, device="cuda"), torch.zeros(NB, 64, 576, dtype=torch.bfloat16, device="cuda")
    binding.mla_cache_append(ck, kr, seq, at, table.cuda(), a)
    binding.mla_cache_append_rope(ck, kr, seq, at, at, binding.mla_rope_freqs(), table.cuda(), b)
    assert torch.equal(a[..., :512], b[..., :512])
    assert ((a - b).double().abs() <= 2 * HALF * a.double().abs() + 2.0 ** -18 * 8).all()


def test_append_rope_reports_bad_targets_and_writes_nothing():
    table = torch.tensor([[2, -1], [7, 0]], dtype=torch.int32, device="cuda")
    cache = torch.ones(4, 64, 576, dtype=torch.bfloat16, device="cuda")
    sp = torch.full((2, 128), -9, dtype=torch.int32, device="cuda")
    ck, kr = torch.zeros(5, 512, dtype=torch.bfloat16, device="cuda"), torch.zeros(5, 64, dtype=torch.bfloat16, device="cuda")
    seq = torch.tensor([0, 1, 0, 2, -1], dtype=torch.int32, device="cuda")
    slot = torch.tensor([64, 10, 128, 0, 0], dtype=torch.int32, device="cuda")
    binding.mla_cache_append_rope(ck, kr, seq, slot, slot, binding.mla_rope_freqs(), table, cache, slot_pos=sp)
    assert binding.mla_cache_get_error() == binding.DEVERR_BAD_BLOCK | binding.DEVERR_SEQ_TOO_LONG
    assert bool((cache == 1).all()) and bool((sp == -9).all())


def test_refusals_of_the_binding():
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16, device="cuda")
    pos = torch.zeros(4, dtype=torch.int32, device="cuda")
    f = binding.mla_rope_freqs()
    y = torch.zeros_like(x)
    for args in [(x.float(), pos, f, y), (x, pos.long(), f, y), (x, pos, f.float(), y), (x.cpu(), pos, f, y)]:
        with pytest.raises((TypeError, ValueError)):
            binding.mla_rope(*args)
    for args in [(x, pos[:3], f, y), (x, pos, f[:31], y), (x, pos, f, y[:, :1]), (x.transpose(1, 2), pos, f, y),
                 (x[..., ::2], pos, f[:16], y[..., :32]), (x[0], pos, f, y)]:
        with pytest.raises(ValueError):
            binding.mla_rope(*args)
    with pytest.raises(binding.MLAError):           # y's rows on top of each other
        binding.mla_rope(x, pos, f, y[:1].expand(4, 2, 64))
    assert binding.mla_rope(x[:0], pos[:0], f, y[:0]).shape[0] == 0
