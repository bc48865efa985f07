"""The first call of a process inside a stream capture, for every operator of a request."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

SET_UP = """
import torch
from mla_latent_kv_25_b200 import binding
from tests._serving import SCALE, Chunk
from tests.test_evict_gpu import Case
c = Chunk([3, 40], [100, 700], 48, seed=2)
q, offs, cache, table, lens = c.cuda()
out, lse = torch.zeros(43, 48, 512, dtype=torch.bfloat16, device="cuda"), torch.zeros(43, 48, device="cuda")
cws = binding.alloc_chunk_workspace(43, 2, 48, num_splits=8)
e = Case([500, 20000], [200, 9000], seed=11)
w, p, ln, kp, tb, ca = (t.cuda() for t in (e.weight, e.pos, e.lens, e.keep, e.table, e.cache))
nw, np_, nl = torch.zeros_like(w), torch.zeros_like(p), torch.zeros_like(ln)
ews = binding.alloc_evict_workspace(2, tb.shape[1])
freqs = binding.mla_rope_freqs()
y, pos = torch.zeros(43, 48, 64, dtype=torch.bfloat16, device="cuda"), torch.arange(43, dtype=torch.int32, device="cuda")
rows, app = torch.randn(43, 576, device="cuda").bfloat16(), torch.zeros_like(cache)
seq = torch.ones(43, dtype=torch.int32, device="cuda")
torch.cuda.synchronize()
"""
CALLS = {
    "rope": ("binding.mla_rope(q[..., 512:], pos, freqs, y)", "y"),
    "append": ("binding.mla_cache_append_rope(rows[:, :512], rows[:, 512:], seq, pos, pos, freqs, table, app)", "app"),
    "chunk": ("binding.mla_chunk_attend(q, offs, cache, table, lens, SCALE, out, lse, cws, num_splits=8)", "out"),
    "evict": ("binding.mla_cache_evict(w, p, ln, kp, 4, 32, tb, ca, nw, np_, nl, ews)", "nw"),
}
RUN = """
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    {call}
torch.cuda.synchronize()
assert not {result}.any(), "ran while it was captured"
g.replay()
torch.cuda.synchronize()
first = {result}.clone()
assert first.any()
{again}
assert torch.equal(first, {result})
print("ok")
"""


@pytest.mark.parametrize("name", CALLS)
def test_first_call_is_captured(name):
    call, result = CALLS[name]
    # an eviction moves rows: its second run starts from the first one's cache, but the same weights
    code = SET_UP + RUN.format(call=call, result=result, again=f"{result}.zero_()\n{call}\ntorch.cuda.synchronize()")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and r.stdout.strip().endswith("ok"), r.stdout + r.stderr
