"""Host model of the chunk plan's cuts (csrc/chunk_sm100.cu: engines_of, chunk_plan_kernel, Walker and the
merge's choice of tiles): every tile with rows to read is written exactly once, whole by one engine or as
pieces that exactly one boundary merges, each from the slot it was left in.  A transcription: a change to the
kernels' cuts must be made here too."""
import random

import pytest

TILE, MIN_UNITS, WHOLE, MAX_ENGINES = 8, 10, 16, 64


def tile_of(pre, nt, x):
    return max(t for t in range(nt) if pre[t] <= x)


def plan(blocks, asked, slack_share=2):
    """(s, e, first tile) of every engine; blocks: cache blocks of every tile."""
    nt = len(blocks)
    pre = [0]
    for b in blocks:
        pre.append(pre[-1] + (b + TILE if b else 0))
    total = pre[-1]
    P = min(asked, -(-total // MIN_UNITS))
    start = lambda e: e * total // P  # noqa: E731
    move = 1 < P <= MAX_ENGINES and nt > 1 and 2 * nt >= P
    cut = [start(e) for e in range(P + 1)] if P else []
    if move:
        share = total // P
        near, slack = min(TILE, share // 16), min(WHOLE, share // slack_share)
        even, whole = list(cut), list(cut)
        for e in range(1, P):
            x = cut[e]
            t = tile_of(pre, nt, x)
            a, z = pre[t], pre[t + 1]
            whole[e] = a if x - a <= z - x else z
            if abs(whole[e] - x) <= near:
                even[e] = whole[e]
        cut = even if any(whole[e + 1] - whole[e] > share + slack for e in range(P)) else whole
    engines = [(cut[e], cut[e + 1], tile_of(pre, nt, cut[e])) for e in range(P)]
    return pre, engines + [(0, 0, nt)] * (asked - P)


def run(blocks, asked, **kw):
    nt = len(blocks)
    pre, engines = plan(blocks, asked, **kw)
    written, slots = {}, {}          # tile -> writes of its rows; slot -> (tile, blocks)
    for p, (s, e, t0) in enumerate(engines):
        count = 0
        for t in range(t0, nt):
            a, z = pre[t] + TILE, pre[t + 1]
            if a - TILE >= e:
                break
            lo, hi = max(s, a), min(e, z)
            if lo >= hi:
                continue
            if (lo, hi) == (a, z):
                written[t] = written.get(t, 0) + 1
            else:
                slot = 2 * p + (1 if count else 0)
                assert slot not in slots
                slots[slot] = (t, lo - a, hi - a)
            count += 1
    for p in range(asked - 1):       # boundary between engines p and p + 1
        x, _, t = engines[p + 1]
        s0 = engines[p][0]
        if t >= nt:
            continue
        a, z = pre[t], pre[t + 1]
        if x <= a + TILE or s0 > a + TILE:
            continue
        n = 1
        while p + n < asked and engines[p + n][2] < nt and engines[p + n][0] < z:
            n += 1
        at = 0
        for i in range(n):
            slot = 2 * (p + i) + (1 if i == 0 and s0 < a else 0)
            assert slot in slots, f"tile {t}: slot {slot} was not written"
            tile, lo, hi = slots.pop(slot)
            assert (tile, lo) == (t, at)
            at = hi
        assert at == blocks[t]
        written[t] = written.get(t, 0) + 1
    assert not slots, "pieces that nobody merges"
    assert written == {t: 1 for t in range(nt) if blocks[t]}


@pytest.mark.parametrize("seed", range(8))
def test_every_tile_is_written_once(seed):
    rng = random.Random(seed)
    for _ in range(1500):
        nt = rng.choice([1, 1, 2, 3, rng.randint(1, 12), rng.randint(1, 90)])
        most = rng.choice([1, 3, 8, 40, 300])
        shape = rng.random()
        blocks = [rng.randint(0, most) for _ in range(nt)]
        if shape < 0.3:
            blocks = [most] * nt
        elif shape < 0.5:            # a long tile somewhere, often the last
            blocks[rng.choice([0, nt - 1, nt - 1])] = rng.randint(1, 20 * most)
        if rng.random() < 0.3:
            blocks += [0] * rng.randint(0, 3)
        run(blocks, rng.choice([1, 2, 3, 5, 13, 33, 33, 33, 64, 65, 200]))


def test_more_slack_would_let_the_merge_take_a_whole_tile():
    """The invariant beside `slack`: with more than half a range, a cut reaches the end of the last tile."""
    with pytest.raises(AssertionError):
        for last in range(1, 60):
            for n in range(1, 12):
                run([1] * n + [last], 2, slack_share=1)
                run([1] * n + [last], 3, slack_share=0.25)
