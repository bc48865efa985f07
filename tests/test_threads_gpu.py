"""Calls from host threads other than the one that loaded the library."""
import threading

import pytest
import torch

import oracle
from mla_latent_kv_25_b200 import binding, inputs
from oracle import serving
from tests._serving import SCALE, Chunk, check_attention, f64
from tests._util import assert_close, to_np
from tests.test_chunk_gpu import check_weights
from tests.test_evict_gpu import Case

pytestmark = pytest.mark.gpu


def in_thread(fn):
    got = []

    def body():
        try:
            got.append(fn())
        except Exception as x:  # noqa: BLE001
            got.append(x)

    t = threading.Thread(target=body)
    t.start()
    t.join()
    if isinstance(got[0], Exception):
        raise got[0]
    return got[0]


def test_first_call_of_a_thread():
    """A thread's first CUDA call may be any of the library's that build tensor maps."""
    c = Chunk([4], [100], 32, seed=1)
    t = c.cuda()
    out, lse = torch.empty(4, 32, 512, dtype=torch.bfloat16, device="cuda"), torch.empty(4, 32, device="cuda")
    w = torch.zeros(1, c.table.shape[1] * 64, device="cuda")
    ws = binding.alloc_chunk_workspace(4, 1, 32)
    st = torch.cuda.current_stream()
    in_thread(lambda: binding.mla_chunk_attend(*t, SCALE, out, lse, ws, stream=st))
    in_thread(lambda: binding.mla_cache_weigh(t[0], t[1], lse, t[2], t[3], t[4], SCALE, None, w, stream=st))
    assert binding.mla_get_device_error(ws) == 0
    check_attention(f64(out), f64(lse), *serving.chunk_attend(*c.np(), SCALE), 100, "a thread's first call")
    check_weights(w, c, lse.cpu(), None, untouched=0.0)
    v = inputs.make("v3", B=2, H=32, L=[70, 130], seed=5)
    d = binding.to_device(v)
    o, l = torch.empty(2, 32, 512, dtype=torch.bfloat16, device="cuda"), torch.empty(2, 32, device="cuda")
    dw = binding.alloc_workspace(2, 32)
    in_thread(lambda: binding.mla_decode(d["q"], d["cache"], d["block_table"], d["seq_lens"], v.softmax_scale, o, l, dw, stream=st))
    assert binding.mla_get_device_error(dw) == 0
    ro, rl = oracle.decode_workload(v)
    assert_close(to_np(o).reshape(-1, 512), ro, "a thread's first decode")
    assert_close(to_np(l).reshape(-1), rl, "a thread's first decode, lse")
    x = torch.randn(2, 32, 128, device="cuda").bfloat16()
    uk = torch.randn(32, 128, 512, device="cuda").bfloat16()
    qa = [torch.zeros(2, 32, 576, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    oa = [torch.zeros(2, 32, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    binding.mla_absorb_q(x, uk, None, qa[0])
    in_thread(lambda: binding.mla_absorb_q(x, uk, None, qa[1], stream=st))
    binding.mla_absorb_o(o, uk, oa[0])
    in_thread(lambda: binding.mla_absorb_o(o, uk, oa[1], stream=st))
    assert binding.mla_absorb_get_error() == 0
    assert torch.equal(qa[0], qa[1]) and torch.equal(oa[0], oa[1]) and bool(oa[1].any())


def test_calls_from_several_threads():
    """Four threads with streams and workspaces of their own, the same call twenty times each."""
    runs, failed = [], []
    for k in range(4):
        c = Chunk([30, 5 + k], [700, 64], (16, 48, 64, 128)[k], seed=k)
        e = Case([900, 70], [300, 64], seed=k)
        t = c.cuda()
        d = [x.cuda() for x in (e.weight, e.pos, e.lens, e.keep, e.table, e.cache)]
        outs = (torch.empty(c.T, c.H, 512, dtype=torch.bfloat16, device="cuda"), torch.empty(c.T, c.H, device="cuda"),
                torch.zeros(2, c.table.shape[1] * 64, device="cuda"), torch.zeros_like(d[0]), torch.zeros_like(d[1]),
                torch.zeros_like(d[2]))
        runs.append((c, e, t, d, outs, binding.alloc_chunk_workspace(c.T, 2, c.H),
                     binding.alloc_evict_workspace(2, e.table.shape[1]), torch.cuda.Stream()))
    torch.cuda.synchronize()

    def work(c, e, t, d, outs, ws, ew, st):
        try:
            for i in range(20):
                binding.mla_chunk_attend(*t, SCALE, outs[0], outs[1], ws, stream=st)
                binding.mla_cache_weigh(t[0], t[1], outs[1], t[2], t[3], t[4], SCALE, None, outs[2], stream=st)
                if i == 0:      # the cache is cut once
                    binding.mla_cache_evict(*d[:4], 4, 32, d[4], d[5], outs[3], outs[4], outs[5], ew, stream=st)
        except Exception as x:  # noqa: BLE001
            failed.append(x)

    threads = [threading.Thread(target=work, args=r) for r in runs]
    for x in threads:
        x.start()
    for x in threads:
        x.join()
    torch.cuda.synchronize()
    assert not failed
    for c, e, t, d, outs, ws, ew, st in runs:
        assert binding.mla_get_device_error(ws) == 0 and binding.mla_get_device_error(ew) == 0
        check_attention(f64(outs[0]), f64(outs[1]), *serving.chunk_attend(*c.np(), SCALE), 700, "thread")
        check_weights(outs[2], c, outs[1].cpu(), None, untouched=0.0)
        kept = serving.evict(e.weight.numpy(), e.pos.numpy(), e.lens.numpy(), e.keep.numpy(), 4, 32)
        for b, s in enumerate(kept):
            assert int(outs[5][b]) == len(s) and torch.equal(outs[4][b, :len(s)].cpu(), e.pos[b][torch.from_numpy(s)])
