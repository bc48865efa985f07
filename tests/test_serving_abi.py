"""Host side of mla_rope*, mla_cache_append_rope, mla_chunk_attend, mla_cache_weigh
and mla_cache_evict: refusals before anything is launched, sizes, frequencies."""
import ctypes

import numpy as np
import pytest

from mla_latent_kv_25_b200 import binding
from oracle import serving

P = ctypes.c_void_p
G = P(4096)
INVALID, SMALL = 1, 3


def call(fn, good, **change):
    args = dict(good, **change)
    return getattr(binding.load(), fn)(*args.values())


ROPE = dict(x=G, x_ldt=8192, x_ldh=64, pos=G, freqs=G, m=1.0, flags=0, y=G, y_ldt=8192, y_ldh=64, T=4, H=128, rot=64,
            st=None)
APPEND = dict(c=G, ckv_ld=576, k=G, kr_ld=576, seq=G, slot=G, pos=G, T=4, freqs=G, m=1.0, flags=0, table=G, B=2, mb=4,
              NB=8, cache=G, slot_pos=G, st=None)
CHUNK = dict(q=G, offs=G, T=4, kind=0, cache=G, k_rope=None, scales=None, table=G, lens=G, B=2, H=128, NB=8, mb=4, scale=0.1, out=G, lse=G, ws=G,
             wsb=1 << 40, splits=4, st=None)
WEIGH = dict(q=G, offs=G, T=4, lse=G, cache=G, table=G, lens=G, B=2, H=128, NB=8, mb=4, scale=0.1, win=G, wout=G,
             st=None)
EVICT = dict(w=G, pos=G, lens=G, keep=G, first=4, recent=32, table=G, B=2, NB=8, mb=4, cache=G, nw=G, np=G, nl=G, ws=G,
             wsb=1 << 40, st=None)


@pytest.mark.parametrize("change", [
    dict(x=None), dict(pos=None), dict(freqs=None), dict(y=None), dict(T=-1), dict(T=(1 << 26) + 1), dict(H=0),
    dict(H=65536), dict(rot=63), dict(rot=0), dict(rot=258), dict(m=float("nan")), dict(m=float("inf")), dict(flags=4),
    dict(x_ldt=-1), dict(y_ldh=-64), dict(y_ldh=0), dict(y_ldt=32), dict(x=P(4097)), dict(pos=P(4098)),
    dict(freqs=P(4100))])
def test_rope_refuses(change):
    assert call("mla_rope", ROPE, **change) == INVALID


@pytest.mark.parametrize("change", [
    dict(c=None), dict(k=None), dict(seq=None), dict(slot=None), dict(pos=None), dict(freqs=None), dict(table=None),
    dict(cache=None), dict(T=-1), dict(B=0), dict(mb=0), dict(NB=0), dict(ckv_ld=504), dict(ckv_ld=580), dict(kr_ld=62),
    dict(kr_ld=65), dict(flags=8), dict(m=float("nan")), dict(c=P(4104)), dict(k=P(4098)), dict(cache=P(4104)),
    dict(slot_pos=P(4097))])
def test_append_refuses(change):
    assert call("mla_cache_append_rope", APPEND, **change) == INVALID


@pytest.mark.parametrize("change", [
    dict(q=None), dict(offs=None), dict(cache=None), dict(table=None), dict(lens=None), dict(out=None), dict(lse=None),
    dict(ws=None), dict(kind=2), dict(k_rope=G), dict(scales=G), dict(kind=1), dict(kind=1, k_rope=G), dict(kind=1, scales=G),
    dict(kind=1, k_rope=P(4104), scales=G), dict(kind=1, k_rope=G, scales=P(4098)),
    dict(T=-1), dict(B=0), dict(H=8), dict(H=144), dict(H=40), dict(NB=0), dict(mb=0),
    dict(mb=(1 << 24) + 1), dict(scale=float("nan")), dict(scale=float("inf")), dict(splits=-1), dict(splits=4097),
    dict(T=(1 << 23) + 1), dict(q=P(4104)), dict(cache=P(4104)), dict(out=P(4104)), dict(lse=P(4098)), dict(ws=P(4224))])
def test_chunk_refuses(change):
    assert call("mla_chunk_attend", CHUNK, **change) == INVALID


@pytest.mark.parametrize("change", [
    dict(q=None), dict(offs=None), dict(lse=None), dict(cache=None), dict(table=None), dict(lens=None), dict(wout=None),
    dict(T=-1), dict(B=0), dict(H=24), dict(NB=0), dict(mb=0), dict(scale=float("inf")), dict(q=P(4104)),
    dict(cache=P(4104)), dict(lse=P(4098)), dict(win=P(4098)), dict(wout=P(4098))])
def test_weigh_refuses(change):
    assert call("mla_cache_weigh", WEIGH, **change) == INVALID


@pytest.mark.parametrize("change", [
    dict(w=None), dict(pos=None), dict(lens=None), dict(keep=None), dict(table=None), dict(cache=None), dict(nw=None),
    dict(np=None), dict(nl=None), dict(ws=None), dict(B=0), dict(NB=0), dict(mb=0), dict(first=-1), dict(recent=-1),
    dict(cache=P(4104)), dict(w=P(4098)), dict(ws=P(4224))])
def test_evict_refuses(change):
    assert call("mla_cache_evict", EVICT, **change) == INVALID


def test_short_workspaces_are_refused():
    n = binding.mla_chunk_workspace_bytes(4, 2, 128, 4)
    assert n > 0 and call("mla_chunk_attend", CHUNK, wsb=n - 1) == SMALL
    n8 = binding.mla_chunk_fp8_workspace_bytes(4, 2, 128, 4, 4)
    assert n8 == -(-(-(-n // 256) * 256 + 4 * 8) // 256) * 256 + 8 * 64 * 576 * 2
    assert call("mla_chunk_attend", CHUNK, kind=1, k_rope=G, scales=G, wsb=n8 - 1) == SMALL
    assert call("mla_chunk_attend", CHUNK, kind=1, k_rope=G, scales=G, B=4096, mb=8192) == 2   # 2^25 blocks to widen
    assert binding.mla_chunk_fp8_workspace_bytes(4, 4096, 128, 8192, 4) == 0
    n = binding.mla_evict_workspace_bytes(2, 4)
    assert n >= 256 + 2 * 4 + 2 * 4 * 32 * 8 and call("mla_cache_evict", EVICT, wsb=n - 1) == SMALL
    assert binding.mla_chunk_workspace_bytes(4, 2, 24, 4) == 0
    assert binding.mla_chunk_workspace_bytes(-1, 2, 128, 4) == 0
    assert call("mla_cache_evict", EVICT, mb=65537) == 2 and binding.mla_evict_workspace_bytes(1, 65537) == 0
    assert binding.mla_evict_workspace_bytes(1, 65536) > 0
    assert binding.mla_evict_workspace_bytes(0, 4) == 0 and binding.mla_evict_workspace_bytes(1, 0) == 0


def test_no_tokens_is_no_work():
    assert call("mla_rope", ROPE, T=0, x=None, y=None, pos=None) == 0
    assert call("mla_cache_append_rope", APPEND, T=0, c=None, k=None) == 0
    assert call("mla_chunk_attend", CHUNK, T=0, q=None, out=None, lse=None) == 0


@pytest.mark.parametrize("rot", [2, 64, 96, 256])
@pytest.mark.parametrize("scaling,kw", [
    ("none", {}), ("linear", dict(factor=4.0)), ("ntk", dict(factor=16.0, base=500000.0)), ("yarn", dict(factor=40.0)),
    ("yarn", dict(factor=4.0, base=1e6, orig_len=32768.0, beta_fast=16.0, beta_slow=2.0)), ("yarn", dict(factor=1.0))])
def test_frequencies(rot, scaling, kw):
    if scaling == "ntk" and rot < 4:
        with pytest.raises(binding.MLAError):
            binding.mla_rope_freqs(rot, scaling=scaling, device="cpu", **kw)
        return
    got = binding.mla_rope_freqs(rot, scaling=scaling, device="cpu", **kw).numpy()
    # exp, log and pow are good to a few units of 2^-53; the exponents reach ln(1e6) = 14
    assert np.allclose(got, serving.rope_freqs(rot, scaling=scaling, **kw), rtol=64 * 2.0 ** -53, atol=0)


@pytest.mark.parametrize("kw", [
    dict(rot=63), dict(rot=0), dict(rot=258), dict(base=1.0), dict(base=float("nan")), dict(factor=0.5),
    dict(factor=float("inf")), dict(scaling="yarn", orig_len=0.0), dict(scaling="yarn", beta_fast=0.5),
    dict(scaling="yarn", beta_slow=0.0)])
def test_frequencies_refuse(kw):
    with pytest.raises(binding.MLAError):
        binding.mla_rope_freqs(device="cpu", **kw)


def test_unknown_names_are_refused():
    with pytest.raises(ValueError):
        binding.mla_rope_freqs(scaling="dynamic", device="cpu")
    with pytest.raises(ValueError):
        binding._rope_flags("split")
