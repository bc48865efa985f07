"""Numbers beyond 32 bits that the binding hands to int arguments: refused, not cut."""
import pytest
import torch

from mla_latent_kv_25_b200 import binding
from tests.test_evict_gpu import Case


@pytest.mark.parametrize("call", [
    lambda: binding.mla_chunk_workspace_bytes(2 ** 32 + 4, 2, 128, 4),
    lambda: binding.mla_chunk_workspace_bytes(4, 2 ** 32 + 2, 128, 4),
    lambda: binding.mla_chunk_workspace_bytes(4, 2, 128, 2 ** 32),
    lambda: binding.mla_chunk_fp8_workspace_bytes(4, 2, 128, 2 ** 32 + 4, 4),
    lambda: binding.mla_evict_workspace_bytes(2 ** 32 + 1, 4),
    lambda: binding.mla_evict_workspace_bytes(1, -2 ** 32 + 4),
    lambda: binding.alloc_evict_workspace(1, 2 ** 31, device="cpu")])
def test_sizes(call):
    with pytest.raises(ValueError, match="does not fit 32 bits"):
        call()


@pytest.mark.gpu
@pytest.mark.parametrize("first,recent", [(0, 2 ** 32 + 5), (2 ** 31, 0), (2 ** 32, 3), (0, -2 ** 32)])
def test_eviction_windows(first, recent):
    c = Case([100], [50], seed=1)
    with pytest.raises(ValueError, match="does not fit 32 bits"):
        c.run(first, recent, False)


@pytest.mark.gpu
def test_rows_four_gigabytes_apart():
    """Two rows whose stride has the low 32 bits of a plausible one."""
    far = torch.empty(2 ** 32 + 1024, dtype=torch.bfloat16, device="cuda")
    near = torch.zeros(2, 576, dtype=torch.bfloat16, device="cuda")
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    cache = torch.ones(1, 64, 576, dtype=torch.bfloat16, device="cuda")
    args = (i32(0, 0), i32(0, 1), i32(0, 1), binding.mla_rope_freqs(), i32(0).view(1, 1), cache)
    with pytest.raises(ValueError, match="does not fit 32 bits"):
        binding.mla_cache_append_rope(far.as_strided((2, 512), (2 ** 32 + 512, 1)), near[:, 512:], *args)
    with pytest.raises(ValueError, match="does not fit 32 bits"):
        binding.mla_cache_append_rope(near[:, :512], far.as_strided((2, 64), (2 ** 32 + 64, 1)), *args)
    assert bool((cache == 1).all())
