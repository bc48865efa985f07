"""The error word that the cache writers and mla_cache_weigh share."""
import os
import subprocess
import sys

import pytest
import torch

from mla_latent_kv_25_b200 import binding
from tests._serving import SCALE, Chunk

pytestmark = pytest.mark.gpu


def bad_append(seq, block):
    """An append whose only token targets a sequence or a block that does not exist."""
    row = torch.zeros(1, 576, dtype=torch.bfloat16, device="cuda")
    i32 = lambda v: torch.tensor([v], dtype=torch.int32, device="cuda")  # noqa: E731
    binding.mla_cache_append_rope(row[:, :512], row[:, 512:], i32(seq), i32(0), i32(0), binding.mla_rope_freqs(),
                                  torch.tensor([[block]], dtype=torch.int32, device="cuda"),
                                  torch.zeros(2, 64, 576, dtype=torch.bfloat16, device="cuda"))


def bad_weigh():
    c = Chunk([1], [70], 16, seed=1)
    c.table[0, 1] = -1
    q, offs, cache, table, lens = c.cuda()
    binding.mla_cache_weigh(q, offs, torch.zeros(1, 16, device="cuda"), cache, table, lens, SCALE, None,
                            torch.zeros(1, 128, device="cuda"))


def test_bits_of_every_call_come_in_one_query_and_are_cleared():
    binding.mla_cache_get_error()
    bad_append(7, 0)
    bad_weigh()
    assert binding.mla_cache_get_error() == binding.DEVERR_SEQ_TOO_LONG | binding.DEVERR_BAD_BLOCK
    assert binding.mla_cache_get_error() == 0
    bad_append(0, 5)
    assert binding.mla_cache_get_error() == binding.DEVERR_BAD_BLOCK
    bad_weigh()
    assert binding.mla_cache_get_error() == binding.DEVERR_BAD_BLOCK
    assert binding.mla_cache_get_error() == 0


def test_a_query_is_one_copy_and_one_clear():
    """One device-to-host copy, one memset and no kernel: no bits are lost between two queries of one call."""
    binding.mla_cache_get_error()
    with torch.profiler.profile(activities=[torch.profiler.ProfilerActivity.CUDA]) as prof:
        for _ in range(4):
            binding.mla_cache_get_error()
        torch.cuda.synchronize()
    seen = [e.name for e in prof.events() if e.device_type == torch.profiler.DeviceType.CUDA]
    copies = [n for n in seen if n.startswith("Memcpy DtoH")]
    clears = [n for n in seen if n.startswith("Memset")]
    assert (len(copies), len(clears), len(seen)) == (4, 4, 8), seen


def test_the_first_call_of_a_process_may_be_captured():
    """mla_cache_weigh looks the word up on the current device, also while a stream is captured."""
    code = """
import torch
from mla_latent_kv_25_b200 import binding
from tests._serving import SCALE, Chunk
c = Chunk([3], [100], 16, seed=2)
q, offs, cache, table, lens = c.cuda()
lse, out = torch.zeros(3, 16, device="cuda"), torch.zeros(1, 128, device="cuda")
binding.load()
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    binding.mla_cache_weigh(q, offs, lse, cache, table, lens, SCALE, None, out)
assert not out.any()
g.replay()
again = torch.zeros_like(out)
binding.mla_cache_weigh(q, offs, lse, cache, table, lens, SCALE, None, again)
assert torch.equal(out, again) and bool((out[0, :100] > 0).all())
assert binding.mla_cache_get_error() == 0
print("ok")
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and r.stdout.strip().endswith("ok"), r.stdout + r.stderr
