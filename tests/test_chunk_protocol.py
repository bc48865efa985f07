"""Host model of the chunk kernel's barrier protocol (csrc/chunk_sm100.cu): the
roles of the four CTAs of an engine as generators over mbarrier phases, run in
random interleavings over many segment patterns and rescale flags.  As for the
decode kernel's model, a test fails on a deadlock, on more arrivals than a
barrier's count and on a waiter lapped by two phases; commits and TMA loads
complete at once.  A change to the kernel's waits, arrivals, ring sizes or
counts must be made here too."""
import random

import pytest

from tests.test_pipeline_protocol import Bar, _patterns

K_SLOTS, V_SLOTS, N_REC, CHUNKS, PASS = 13, 4, 4, 9, 2
Q_SLOTS = CHUNKS - 1                                 # chunks of Q that go through the ring to TMEM


def _passes(lo, hi):
    for j in range(lo, hi, PASS):
        yield j, min(PASS, hi - j)


def _k_slots(lo, hi):
    """Slots of a segment's K: two chunks each, over the ends of passes."""
    return (CHUNKS * len(list(_passes(lo, hi))) + 1) // 2


class Exact(Bar):
    """Also fails on a wait that passes before its phase is complete (a waiter two phases early)."""

    def passes(self, parity, phase):
        ok = super().passes(parity, phase)
        assert not ok or self.done > phase, f"{self.name}: waiter for phase {phase} early ({self.done} done)"
        return ok


def roles(segs, flags, counts):
    B = {}

    def bar(name, count):
        B[name] = Exact(name, counts.get(name.rstrip("0123456789_"), count))

    def at(name, rank):
        return f"{name}_{rank}"

    for s in range(K_SLOTS):
        bar(f"k_full{s}", 2)                         # rank 0's arrival with its bytes, rank 1's bytes
        for r in (0, 1):
            bar(at(f"k_empty{s}", r), 1)
    bar("q_full", 2)                                 # the last chunk of Q
    for r in (0, 1):
        bar(at("q_empty", r), 1)
    for s in range(2):
        bar(f"s_empty{s}", 8)
        for r in (0, 1):
            bar(at(f"s_full{s}", r), 1)
        for r in (0, 1):                             # one quadrant's warp of each half
            bar(at(f"m_set{s}", r), 1)
            bar(at(f"l_set{s}", r), 1)
    for i in range(N_REC):
        for r in (0, 1):
            bar(at(f"p_empty{i}", r), 1)
        for r in (2, 3):
            bar(at(f"p_full{i}", r), 4)
        bar(f"p_ready{i}", 2)
    for s in range(V_SLOTS):
        for r in (2, 3):
            bar(at(f"v_full{s}", r), 1)
            bar(at(f"v_empty{s}", r), 1)
        bar(f"v_ready{s}", 2)
    for r in (2, 3):
        bar(at("epi_req", r), 2)
        bar(at("meta_done", r), 8)
    bar("corr_done", 16)
    bar("o_free", 16)

    def score_tma(rank):
        fit = 0
        for lo, hi in segs:
            for _ in range(Q_SLOTS + _k_slots(lo, hi)):
                s = fit % K_SLOTS
                yield at(f"k_empty{s}", rank), ((fit // K_SLOTS) & 1) ^ 1, fit // K_SLOTS - 1
                B[f"k_full{s}"].arrive()
                fit += 1

    def score_q(rank):
        for seg, _ in enumerate(segs):
            yield at("q_empty", rank), (seg & 1) ^ 1, seg - 1
            B["q_full"].arrive()

    def score_mma():
        fit = pit = 0

        def full():
            return f"k_full{fit % K_SLOTS}", (fit // K_SLOTS) & 1, fit // K_SLOTS

        def done(name):
            for r in (0, 1):
                B[at(name, r)].arrive()

        for seg, (lo, hi) in enumerate(segs):
            if pit > 0:                              # the MMAs that read the last segment's Q
                yield at(f"s_full{(pit - 1) & 1}", 0), ((pit - 1) >> 1) & 1, (pit - 1) >> 1
            for _ in range(Q_SLOTS):
                yield full()
                done(f"k_empty{fit % K_SLOTS}")
                fit += 1
            half = 0
            for j, nb in _passes(lo, hi):
                last = j + nb >= hi
                yield f"s_empty{pit & 1}", ((pit >> 1) & 1) ^ 1, (pit >> 1) - 1
                for ch in range(CHUNKS):
                    if half == 0:
                        yield full()
                    if ch == CHUNKS - 1:
                        if j == lo:
                            yield "q_full", seg & 1, seg
                        if last:
                            done("q_empty")
                    if half or (last and ch == CHUNKS - 1):
                        done(f"k_empty{fit % K_SLOTS}")
                        fit += 1
                        half = 0
                    else:
                        half = 1
                done(f"s_full{pit & 1}")
                pit += 1

    def softmax(rank, half):
        it = pit = joined = 0
        for lo, hi in segs:
            for j0, nb in _passes(lo, hi):
                if pit & 1 != half:
                    it += nb
                    pit += 1
                    continue
                first, last = j0 == lo, j0 + nb >= hi
                yield at(f"s_full{half}", rank), (pit >> 1) & 1, pit >> 1
                B[f"s_empty{half}"].arrive(4)
                if pit > 0:
                    yield at(f"m_set{half ^ 1}", rank), ((pit - 1) >> 1) & 1, (pit - 1) >> 1
                if not last:
                    B[at(f"m_set{half}", rank)].arrive()
                for kb in range(nb):
                    ib = it + kb
                    r = ib % N_REC
                    yield at(f"p_empty{r}", rank), ((ib // N_REC) & 1) ^ 1, ib // N_REC - 1
                    if not (last and kb == nb - 1):
                        B[at(f"p_full{r}", rank + 2)].arrive(4)
                it += nb
                if not last:
                    if j0 + 2 * PASS >= hi:
                        B[at(f"l_set{half}", rank)].arrive()
                else:
                    if not first:
                        yield at(f"l_set{half ^ 1}", rank), joined & 1, joined
                        joined += 1
                    B[at(f"m_set{half}", rank)].arrive()
                    B[at(f"p_full{(it - 1) % N_REC}", rank + 2)].arrive(4)
                pit += 1

    def blocks():
        i = 0
        for lo, hi in segs:
            for j in range(lo, hi):
                yield i, j == lo, j == hi - 1
                i += 1

    def value_tma(rank):
        for i, _, _ in blocks():
            s = i % V_SLOTS
            yield at(f"v_empty{s}", rank), ((i // V_SLOTS) & 1) ^ 1, i // V_SLOTS - 1
            B[at(f"v_full{s}", rank)].arrive()

    def fixup(rank):
        for i, _, _ in blocks():
            s = i % V_SLOTS
            yield at(f"v_full{s}", rank), (i // V_SLOTS) & 1, i // V_SLOTS
            B[f"v_ready{s}"].arrive()

    def relay(rank):
        for i, _, _ in blocks():
            r = i % N_REC
            yield at(f"p_full{r}", rank), (i // N_REC) & 1, i // N_REC
            B[f"p_ready{r}"].arrive()

    def value_mma():
        ncorr = seg = 0
        for i, first, last in blocks():
            r, s = i % N_REC, i % V_SLOTS
            if first and seg > 0:
                yield "o_free", (seg - 1) & 1, seg - 1
            yield f"p_ready{r}", (i // N_REC) & 1, i // N_REC
            if flags[i] and not first:
                for c in (2, 3):
                    B[at("epi_req", c)].arrive(2)
                yield "corr_done", ncorr & 1, ncorr
                ncorr += 1
            yield f"v_ready{s}", (i // V_SLOTS) & 1, i // V_SLOTS
            for c in (2, 3):
                B[at(f"v_empty{s}", c)].arrive()
                if last:
                    B[at("epi_req", c)].arrive(2)
                else:
                    B[at(f"p_empty{r}", c - 2)].arrive()
            if last:
                seg += 1

    def epilogue(rank):
        nreq = nfinal = 0
        for i, first, last in blocks():
            r = i % N_REC
            if flags[i] and not first:
                yield at("epi_req", rank), nreq & 1, nreq
                nreq += 1
                B["corr_done"].arrive(8)
            if last:
                yield at("epi_req", rank), nreq & 1, nreq
                nreq += 1
                B[at("meta_done", rank)].arrive(8)
                yield at("meta_done", rank), nfinal & 1, nfinal
                nfinal += 1
                B[at(f"p_empty{r}", rank - 2)].arrive()
                B["o_free"].arrive(8)

    procs = {"score_mma": score_mma(), "value_mma": value_mma()}
    for r in (0, 1):
        procs |= {f"k{r}": score_tma(r), f"q{r}": score_q(r), f"soft{r}a": softmax(r, 0), f"soft{r}b": softmax(r, 1),
                  f"v{r + 2}": value_tma(r + 2), f"relay{r + 2}": relay(r + 2), f"fix{r + 2}": fixup(r + 2), f"epi{r + 2}": epilogue(r + 2)}
    return B, procs


def simulate(segs, seed, counts=()):
    rng = random.Random(seed)
    flags = [rng.random() < 0.3 for _ in range(sum(hi - lo for lo, hi in segs))]
    B, procs = roles(segs, flags, dict(counts))
    waiting = {}
    for name in list(procs):
        waiting[name] = next(procs[name], None)
    alive = {n for n in procs if waiting[n] is not None}
    while alive:
        moved = False
        for name in rng.sample(sorted(alive), len(alive)):
            while name in alive and B[waiting[name][0]].passes(*waiting[name][1:]):
                moved = True
                waiting[name] = next(procs[name], None)
                if waiting[name] is None:
                    alive.discard(name)
                if rng.random() < 0.3:
                    break
        if not moved:
            return {n: waiting[n] for n in alive}
    return True


def test_protocol_finishes_in_every_interleaving():
    for i, segs in enumerate(_patterns()):
        for seed in range(8):
            res = simulate(segs, 1000 * seed + i)
            assert res is True, f"segments {segs}, seed {seed}: blocked {res}"


@pytest.mark.parametrize("name,count", [("p_empty", 2), ("v_ready", 3), ("q_full", 3), ("s_empty", 9), ("m_set", 2), ("corr_done", 17)])
def test_model_finds_planted_counts(name, count):
    assert all(simulate([(0, 40), (0, 9), (0, 30)], seed, {name: count}) is not True for seed in range(3))
