"""Cases and plain forms of the chunked-prefill and cache-eviction operators.

Four operators of one serving path over the paged latent cache:

  rope / append  rotary positions of the queries, and of the keys on their way into the cache, with
                 frequencies scaled for long contexts
  chunk          attention of ragged chunks of new tokens over the paged cache (absorbed form)
  weigh          the attention weight every cached token received, accumulated over heads and queries
  evict          keep the heaviest, the first and the latest tokens of a sequence, compact the cache

With ``own`` false, ``run`` computes an operator from elementary torch operations in fp32 (angles in
fp64), rounded once at the end.  With ``own`` true it makes the library's calls.
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

D_C, D_R, D_ROW, D_NOPE, BLOCK = 512, 64, 576, 128, 64
SCALE = 1.0 / math.sqrt(D_NOPE + D_R)


# ------------------------------------------------------------------------------------------ cases

def listed():
    return [
        # the queries of one decode step (B = 64, H = 128) rotated into the packed rows decode reads
        dict(name="rope_step", op="rope", T=64, H=128, half=False, wide=True, span=4096, factor=1.0),
        # the queries of a long prompt: the last 64 of each head's 192 values, half layout, stretched 40x
        dict(name="rope_prompt", op="rope", T=8192, H=128, half=True, wide=False, span=131072, factor=40.0),
        # a prompt's latent rows and keys written into the cache, rotated at positions other than slots
        dict(name="append_prompt", op="append", T=8191, B=7, half=False, span=131072, factor=40.0),
        # the smallest call: five tokens of a 16-head shard over a short cache
        dict(name="chunk_tiny", op="chunk", B=1, H=16, n=5, L=261, ragged=False),
        # a mixed serving batch: chunks of 1 to 64 tokens over contexts of up to 4096
        dict(name="chunk_ragged", op="chunk", B=8, H=128, n=64, L=4096, ragged=True),
        # a few tokens over a very long context: the cache has to be split over the whole chip
        dict(name="chunk_long", op="chunk", B=1, H=128, n=16, L=131072, ragged=False),
        # a prefill chunk of a long prompt: tensor-core bound
        dict(name="chunk_prefill", op="chunk", B=1, H=128, n=512, L=16384, ragged=False),
        # the weights of one decode step at B = 64, H = 128, L = 4096
        dict(name="weigh_step", op="weigh", B=64, H=128, n=1, L=4096, ragged=False),
        # an observation window: the last 32 queries of prompts weigh the whole prompt
        dict(name="weigh_window", op="weigh", B=4, H=128, n=32, L=16384, ragged=False),
        # one short sequence cut to a budget
        dict(name="evict_small", op="evict", B=1, L=300, keep=128, ragged=False),
        # the decode batch cut to half its cache
        dict(name="evict_batch", op="evict", B=64, L=4096, keep=2048, ragged=False),
        # long contexts cut to half
        dict(name="evict_long", op="evict", B=4, L=131072, keep=65536, ragged=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "append", "chunk", "chunk", "weigh", "evict"])
    if op == "rope":
        return dict(op=op, T=_log(rng, 1, 8192), H=16 * rng.randint(1, 8), half=rng.random() < 0.5,
                    wide=rng.random() < 0.5, span=_log(rng, 64, 131072), factor=rng.choice([1.0, 4.0, 40.0]))
    if op == "append":
        return dict(op=op, T=_log(rng, 1, 8192), B=rng.randint(1, 16), half=rng.random() < 0.5,
                    span=_log(rng, 64, 131072), factor=rng.choice([1.0, 4.0, 40.0]))
    if op == "evict":
        B = _log(rng, 1, 64)
        L = _log(rng, 2, min(131072, 524288 // B))
        return dict(op=op, B=B, L=L, keep=max(1, int(L * rng.uniform(0.1, 1.0))), ragged=rng.random() < 0.5)
    # no dearer than the largest listed case: 512 queries of 128 heads over 16384 tokens (chunk),
    # 32 over 4 x 16384 (weigh)
    most = 512 * 128 * 16384 if op == "chunk" else 128 * 128 * 16384
    while True:
        B, H = _log(rng, 1, 64), 16 * rng.randint(1, 8)
        L = _log(rng, 1, 131072)
        n = _log(rng, 1, 512 if op == "chunk" else 32)
        n = min(n, L)
        if B * n * H * L <= most and B * L <= 524288:
            return dict(op=op, B=B, H=H, n=n, L=L, ragged=rng.random() < 0.5)


# ----------------------------------------------------------------------------------------- inputs

def _freqs(factor, rot=D_R, base=10000.0, orig=4096.0, fast=32.0, slow=1.0):
    """Angle per position of each pair: base^(-2i/rot); with factor > 1, pairs that turn fewer than
    `slow` times over the original context are slowed by `factor`, those that turn more than `fast`
    times stay, with a linear ramp between (over the pair index, whole bounds)."""
    i = torch.arange(rot // 2, dtype=torch.float64)
    theta = base ** (-2.0 * i / rot)
    if factor <= 1.0:
        return theta
    pair = lambda turns: rot * math.log(orig / (turns * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
    lo = max(0, math.floor(pair(fast)))
    hi = min(rot - 1, math.ceil(pair(slow)))
    ramp = ((i - lo) / max(hi - lo, 1e-3)).clamp(0, 1)
    return theta * (1 - ramp) + theta / factor * ramp


def _mscale(factor):
    return 0.1 * math.log(factor) + 1.0 if factor > 1.0 else 1.0


def _lens(case, gs):
    B, L = case["B"], case["L"]
    if not case["ragged"]:
        return torch.full((B,), L, dtype=torch.int64)
    return torch.randint(1, L + 1, (B,), generator=gs)


def _paged(lens, g, dev):
    """Shuffled block table (-1 past each sequence) for these lengths, and the number of blocks."""
    nblk = (lens + BLOCK - 1) // BLOCK
    NB = int(nblk.sum())
    mb = int(nblk.max())
    perm = torch.randperm(NB, generator=g)
    table = torch.full((len(lens), mb), -1, dtype=torch.int64)
    live = torch.arange(mb)[None, :] < nblk[:, None]
    table[live] = perm
    return table.to(torch.int32).to(dev), NB


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator().manual_seed(seed)
    gs = torch.Generator().manual_seed(11)  # lengths belong to the case, values and placement to the seed
    gd = torch.Generator(device=dev).manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, generator=gd, device=dev, dtype=torch.float32)

    op = case["op"]
    s = dict(case=case, op=op)
    if op in ("rope", "append"):
        s["freqs"] = _freqs(case["factor"]).to(dev)
        s["mscale"] = _mscale(case["factor"])
    if op == "rope":
        T, H = case["T"], case["H"]
        s["x"] = randn(T, H, D_NOPE + D_R).bfloat16()
        s["pos"] = torch.randint(0, case["span"], (T,), generator=gd, device=dev, dtype=torch.int32)
        # the rotated values go into columns 512.. of the packed query rows, or into a tensor of their own
        s["y"] = torch.zeros(T, H, D_ROW if case["wide"] else D_R, device=dev, dtype=torch.bfloat16)
    elif op == "append":
        T, B = case["T"], case["B"]
        s["x"] = randn(T, D_ROW).bfloat16()
        cut = sorted(torch.randint(0, T + 1, (B - 1,), generator=gs).tolist())
        n = torch.tensor([b - a for a, b in zip([0] + cut, cut + [T])])
        had = torch.randint(0, 200, (B,), generator=gs)
        s["table"], NB = _paged(had + n + 1, g, dev)
        seq = torch.repeat_interleave(torch.arange(B), n)
        slot = torch.cat([torch.arange(int(h), int(h + k)) for h, k in zip(had, n)])
        first = torch.randint(0, case["span"], (B,), generator=g)
        s["seq"] = seq.to(torch.int32).to(dev)
        s["slot"] = slot.to(torch.int32).to(dev)
        s["pos"] = (first[seq] + slot).to(torch.int32).to(dev)
        s["cache"] = (randn(NB, BLOCK, D_ROW) / math.sqrt(D_C)).bfloat16()
        s["slot_pos"] = torch.full((B, s["table"].shape[1] * BLOCK), -1, device=dev, dtype=torch.int32)
    elif op in ("chunk", "weigh"):
        B, H = case["B"], case["H"]
        lens = _lens(case, gs)
        if case["ragged"]:
            n = torch.minimum(torch.randint(1, case["n"] + 1, (B,), generator=gs), lens)
        else:
            n = torch.minimum(torch.full((B,), case["n"]), lens)
        s["table"], NB = _paged(lens, g, dev)
        s["lens"] = lens.to(torch.int32).to(dev)
        s["offs"] = torch.cat([torch.zeros(1, dtype=torch.int64), n.cumsum(0)]).to(torch.int32).to(dev)
        T = int(n.sum())
        s["nmax"], s["T"] = int(n.max()), T
        s["q"] = randn(T, H, D_ROW).bfloat16()
        s["cache"] = (randn(NB, BLOCK, D_ROW) / math.sqrt(D_C)).bfloat16()
        if own and op == "chunk":
            from mla_latent_kv_25_b200 import binding
            s["out"] = torch.empty(T, H, D_C, device=dev, dtype=torch.bfloat16)
            s["lse"] = torch.empty(T, H, device=dev, dtype=torch.float32)
            s["ws"] = binding.alloc_chunk_workspace(T, B, H)
        if op == "weigh":
            S = s["table"].shape[1] * BLOCK
            s["lse"] = _attention(s, None)[1]
            s["weight"] = torch.rand(B, S, generator=gd, device=dev)
            s["weight_out"] = torch.zeros(B, S, device=dev)
    else:
        B = case["B"]
        lens = _lens(case, gs)
        s["table"], NB = _paged(lens, g, dev)
        S = s["table"].shape[1] * BLOCK
        s["lens"] = lens.to(torch.int32).to(dev)
        s["keep"] = torch.full((B,), case["keep"], device=dev, dtype=torch.int32)
        # accumulated weights are heavy-tailed: a few tokens take most of the mass
        s["weight"] = randn(B, S).mul_(2.0).exp_()
        s["pos"] = torch.arange(S, device=dev, dtype=torch.int32).repeat(B, 1)
        s["sink"], s["recent"] = 4, 32
        s["cache"] = (randn(NB, BLOCK, D_ROW) / math.sqrt(D_C)).bfloat16()
        s["new_weight"] = torch.zeros(B, S, device=dev)
        s["new_pos"] = torch.full((B, S), -1, device=dev, dtype=torch.int32)
        s["new_lens"] = torch.zeros(B, device=dev, dtype=torch.int32)
        if own:
            from mla_latent_kv_25_b200 import binding
            s["ws"] = binding.alloc_evict_workspace(B, s["table"].shape[1])
    return s


# ------------------------------------------------------------------------------------ plain forms

def _rotate(x, pos, freqs, mscale, half):
    """x [..., rot] in fp32, rotated by pos * freqs (angles in fp64), broadcast over the middle axes."""
    ang = pos.double()[:, None] * freqs
    c, sn = (ang.cos() * mscale).float(), (ang.sin() * mscale).float()
    while c.dim() < x.dim():
        c, sn = c.unsqueeze(1), sn.unsqueeze(1)
    r = x.shape[-1] // 2
    a, b = (x[..., :r], x[..., r:]) if half else (x[..., 0::2], x[..., 1::2])
    u, v = a * c - b * sn, a * sn + b * c
    return torch.cat([u, v], -1) if half else torch.stack([u, v], -1).flatten(-2)


def _padded(s):
    """Queries [B, n*H, 576] and cached rows [B, L, 576] in fp32, zero past each sequence, and the
    number of cached tokens every query row sees."""
    H = s["q"].shape[1]
    offs, lens = s["offs"].long(), s["lens"].long()
    n = offs[1:] - offs[:-1]
    j = torch.arange(s["nmax"], device=offs.device)
    at = (offs[:-1, None] + j).clamp(max=s["T"] - 1)
    has = j < n[:, None]
    q = s["q"][at].float() * has[..., None, None]
    sees = torch.where(has, lens[:, None] - (n[:, None] - 1 - j), 0).clamp(min=0)
    k = s["cache"][s["table"].long().clamp(min=0)].flatten(1, 2)
    k = k.float() * (torch.arange(k.shape[1], device=k.device) < lens[:, None])[..., None]
    return q.flatten(1, 2), k, sees.repeat_interleave(H, 1), has.flatten(), H


def _attention(s, value):
    """Softmax over the visible tokens: (weighted sum of the latent if value, lse)."""
    q, k, sees, has, H = _padded(s)
    p = torch.bmm(q, k.transpose(1, 2)).mul_(SCALE)
    p.masked_fill_(torch.arange(k.shape[1], device=k.device) >= sees[..., None], -math.inf)
    m = p.amax(-1, keepdim=True)
    p = p.sub_(torch.where(m == -math.inf, 0.0, m)).exp_()
    z = p.sum(-1, keepdim=True)
    lse = (z.log() + m).view(-1, H)[has]
    if value is None:
        return None, lse
    o = torch.bmm(p, k[..., :D_C]) / torch.where(z == 0, 1.0, z)
    return o.view(-1, H, D_C)[has].bfloat16(), lse


def _weights(s):
    q, k, sees, has, H = _padded(s)
    lse = torch.full((has.shape[0], H), math.inf, device=q.device)
    lse[has] = s["lse"]
    p = torch.bmm(q, k.transpose(1, 2)).mul_(SCALE)
    p = p.sub_(lse.view(q.shape[0], -1, 1)).exp_()
    p.masked_fill_(torch.arange(k.shape[1], device=k.device) >= sees[..., None], 0.0)
    w = s["weight"] + p.sum(1)
    live = torch.arange(w.shape[1], device=w.device) < s["lens"][:, None]
    return torch.where(live, w, s["weight_out"])


def _evict(s):
    w, pos, lens, keep = s["weight"], s["pos"], s["lens"].long(), s["keep"].long()
    B, S = w.shape
    slot = torch.arange(S, device=w.device).expand(B, S)
    live = slot < lens[:, None]
    new = torch.minimum(keep, lens)
    last = torch.where(live, pos, -1).amax(1, keepdim=True)
    kept_first = (pos < s["sink"]) | (pos > last - s["recent"])
    # by class (protected, others, past the end), then weight from the largest, then slot
    order = w.sort(dim=1, descending=True, stable=True).indices
    group = torch.where(live, torch.where(kept_first, 0, 1), 2)
    order = order.gather(1, group.gather(1, order).sort(dim=1, stable=True).indices)
    rank = torch.empty_like(order).scatter_(1, order, slot)
    kept = live & (rank < new[:, None])
    hole = (slot < new[:, None]) & ~kept
    mover = (slot >= new[:, None]) & kept
    src = torch.zeros_like(order).scatter_(1, torch.where(mover, mover.cumsum(1) - 1, S - 1), torch.where(mover, slot, 0))
    src = src.gather(1, (hole.cumsum(1) - 1).clamp(min=0))
    src = torch.where(hole, src, slot)
    stays = slot < new[:, None]
    s["new_weight"] = torch.where(stays, w.gather(1, src), torch.where(live, 0.0, s["new_weight"]))
    s["new_pos"] = torch.where(stays, pos.gather(1, src), torch.where(live, -1, s["new_pos"]))
    s["new_lens"] = new.to(torch.int32)
    rows = s["cache"].view(-1, D_ROW)
    at = (s["table"].long().clamp(min=0)[:, :, None] * BLOCK + torch.arange(BLOCK, device=w.device)).view(B, S)
    rows[at[hole]] = rows[at.gather(1, src)[hole]]
    return s["new_lens"], s["new_weight"], s["new_pos"], s["cache"]


def run(s):
    op = s["op"]
    if own:
        from mla_latent_kv_25_b200 import binding
        layout = "half" if s["case"].get("half") else "interleaved"
        if op == "rope":
            y = s["y"][..., D_C:] if s["case"]["wide"] else s["y"]
            binding.mla_rope(s["x"][..., D_NOPE:], s["pos"], s["freqs"], y, mscale=s["mscale"], layout=layout)
            return s["y"]
        if op == "append":
            binding.mla_cache_append_rope(s["x"][:, :D_C], s["x"][:, D_C:], s["seq"], s["slot"], s["pos"], s["freqs"],
                                          s["table"], s["cache"], slot_pos=s["slot_pos"], mscale=s["mscale"],
                                          layout=layout)
            return s["cache"], s["slot_pos"]
        if op == "chunk":
            binding.mla_chunk_attend(s["q"], s["offs"], s["cache"], s["table"], s["lens"], SCALE, s["out"], s["lse"],
                                     s["ws"])
            return s["out"], s["lse"]
        if op == "weigh":
            binding.mla_cache_weigh(s["q"], s["offs"], s["lse"], s["cache"], s["table"], s["lens"], SCALE,
                                    s["weight"], s["weight_out"])
            return s["weight_out"]
        binding.mla_cache_evict(s["weight"], s["pos"], s["lens"], s["keep"], s["sink"], s["recent"], s["table"],
                                s["cache"], s["new_weight"], s["new_pos"], s["new_lens"], s["ws"])
        return s["new_lens"], s["new_weight"], s["new_pos"], s["cache"]
    if op == "rope":
        y = _rotate(s["x"][..., D_NOPE:].float(), s["pos"], s["freqs"], s["mscale"], s["case"]["half"]).bfloat16()
        s["y"][..., -D_R:] = y
        return s["y"]
    if op == "append":
        key = _rotate(s["x"][:, D_C:].float(), s["pos"], s["freqs"], s["mscale"], s["case"]["half"]).bfloat16()
        blk = s["table"][s["seq"].long(), s["slot"].long() // BLOCK].long()
        s["cache"][blk, s["slot"].long() % BLOCK] = torch.cat([s["x"][:, :D_C], key], 1)
        s["slot_pos"][s["seq"].long(), s["slot"].long()] = s["pos"]
        return s["cache"], s["slot_pos"]
    if op == "chunk":
        return _attention(s, True)
    if op == "weigh":
        return _weights(s)
    return _evict(s)


# ------------------------------------------------------------------------------------------ floors

def work(case):
    op = case["op"]
    if op == "rope":
        n = case["T"] * case["H"] * D_R
        return {"bytes": n * 4 + case["T"] * 4, "flops": n * 3}
    if op == "append":
        return {"bytes": case["T"] * (D_ROW * 4 + 16), "flops": case["T"] * D_R * 3}
    share = 0.5 if case["ragged"] else 1.0  # ragged lengths are uniform: half the largest on average
    tokens = case["B"] * case["L"] * share
    if op in ("chunk", "weigh"):
        rows = max(1.0, case["B"] * case["n"] * share) * case["H"]
        pairs = rows * case["L"] * share
        if op == "chunk":
            return {"bytes": tokens * D_ROW * 2 + rows * (D_ROW * 2 + D_C * 2 + 4), "flops": 2 * pairs * (D_ROW + D_C)}
        return {"bytes": tokens * (D_ROW * 2 + 8) + rows * (D_ROW * 2 + 4), "flops": 2 * pairs * (D_ROW + 1)}
    keep = min(1.0, case["keep"] / case["L"])
    # kept rows behind the budget move into the holes before it: keep * (1 - keep) of the tokens
    return {"bytes": tokens * (8 + 8 + keep * (1 - keep) * D_ROW * 4), "flops": tokens * 4}


# ---------------------------------------------------------------------------------- 64-bit results

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "rope":
        x, y = s["x"][..., D_NOPE:].double(), s["y"].double()
        y[..., -D_R:] = _turn64(x, s["pos"].double()[:, None, None] * s["freqs"], s["mscale"], case["half"])
        return y
    if op == "append":
        cache, where = s["cache"].double(), s["slot_pos"].clone()
        rows = s["x"].double()
        rows[:, D_C:] = _turn64(rows[:, D_C:], s["pos"].double()[:, None] * s["freqs"], s["mscale"], case["half"])
        for b in range(case["B"]):
            mine = s["seq"] == b
            slot = s["slot"][mine].long()
            cache[s["table"][b].long()[slot // BLOCK], slot % BLOCK] = rows[mine]
            where[b, slot] = s["pos"][mine]
        return cache, None
    if op == "evict":
        cache, weight = s["cache"].double(), s["new_weight"].double()
        w, pos, table = s["weight"].cpu().numpy(), s["pos"].cpu().numpy(), s["table"].cpu().numpy()
        for b, L in enumerate(s["lens"].tolist()):
            other = (pos[b, :L] >= s["sink"]) & (pos[b, :L] <= pos[b, :L].max() - s["recent"])
            kept = np.lexsort((np.arange(L), -w[b, :L].astype(np.float64), other))[: case["keep"]]
            new = len(kept)
            src = np.sort(kept[kept >= new])
            dst = np.setdiff1d(np.arange(new), kept)
            weight[b, :L] = 0.0
            now = w[b, :new].astype(np.float64)
            now[dst] = w[b, src]
            weight[b, :new] = torch.from_numpy(now).to(weight.device)
            at = [torch.from_numpy(table[b, i // BLOCK].astype(np.int64) * BLOCK + i % BLOCK) for i in (src, dst)]
            cache.view(-1, D_ROW)[at[1].to(cache.device)] = s["cache"].view(-1, D_ROW)[at[0].to(cache.device)].double()
        return None, weight, None, cache
    if op == "weigh":
        total = s["weight_out"].double()
    outs, lses = [], []
    offs, lens = s["offs"].tolist(), s["lens"].tolist()
    for b in range(case["B"]):
        n, L = offs[b + 1] - offs[b], lens[b]
        blocks = s["table"][b, : (L + BLOCK - 1) // BLOCK].long()
        rows = s["cache"][blocks].reshape(-1, D_ROW)[:L].double()
        if op == "weigh":
            total[b, :L] = s["weight"][b, :L].double()
        for j0 in range(0, n, 32):
            q = s["q"][offs[b] + j0 : min(offs[b] + j0 + 32, offs[b + 1])].double()
            sees = L - (n - 1 - torch.arange(j0, j0 + q.shape[0], device=q.device))
            sc = torch.einsum("jhd,td->jht", q, rows) * SCALE
            hidden = torch.arange(L, device=q.device)[None, None, :] >= sees[:, None, None]
            if op == "weigh":
                lse = s["lse"][offs[b] + j0 : offs[b] + j0 + q.shape[0]].double()
                total[b, :L] += torch.exp(sc - lse[..., None]).masked_fill(hidden, 0.0).sum((0, 1))
            else:
                sc = sc.masked_fill(hidden, -math.inf)
                lse = torch.logsumexp(sc, -1)
                lses.append(lse)
                outs.append(torch.exp(sc - lse[..., None]) @ rows[:, :D_C])
    return total if op == "weigh" else (torch.cat(outs), torch.cat(lses))


def _turn64(x, ang, mscale, half):
    """Rotation as a complex product in 64 bits."""
    r = x.shape[-1] // 2
    z = torch.complex(x[..., :r], x[..., r:]) if half else torch.view_as_complex(x.unflatten(-1, (r, 2)).contiguous())
    z = z * torch.polar(torch.full_like(ang, mscale), ang)
    return torch.cat([z.real, z.imag], -1) if half else torch.view_as_real(z).flatten(-2)
