"""A host model of the barrier protocol of the wide and narrow block-scaled kernels
(gemm_bs_wide.cuh, gemm_bs_narrow.cuh) under random interleavings: the TMA producer, the MMA
issuers and the accumulating warps as coroutines over modelled mbarriers, the loads of different
stages landing late and in any order, each issuer's commits completing late and in its order.

k-block q of a CTA is issued by issuer q % issuers into partial q % partials (wide: 2 and 2;
narrow: 1 and 8).  An issuer first waits PEMPTY of the partial, then FULL of the stage.  That
order matters: PEMPTY of k-block q shows that k-blocks up to q - partials were added, hence that
their loads have landed, so FULL's parity cannot be that of an earlier use of the stage.  With
the waits exchanged two issuers read a stale stage of a three-stage ring, which the model catches."""
import random

import pytest


class Bar:
    def __init__(self, count):
        self.count, self.pending, self.phase = count, count, 0

    def arrive(self):
        self.pending -= 1
        assert self.pending >= 0
        if self.pending == 0:
            self.phase += 1
            self.pending = self.count

    def done(self, parity):
        return (self.phase & 1) != parity


class Stale(AssertionError):
    pass


def run(kblocks, stages, issuers, partials, warps, seed, full_first=False):
    rng = random.Random(seed)
    full, empty = [Bar(1) for _ in range(stages)], [Bar(1) for _ in range(stages)]
    pfull, pempty = [Bar(1) for _ in range(partials)], [Bar(warps) for _ in range(partials)]
    stage_tag, partial_tag = [None] * stages, [None] * partials
    loads, commits = [], []   # in flight: (stage, k-block) in any order; (issuer, action) in an issuer's order

    def producer():
        for q in range(kblocks):
            s = q % stages
            while not empty[s].done((q // stages & 1) ^ 1):
                yield
            loads.append((s, q))
            yield

    def issuer(r):
        for q in range(r, kblocks, issuers):
            s, b = q % stages, q % partials
            waits = [(pempty[b], (q // partials & 1) ^ 1), (full[s], q // stages & 1)]
            for bar, parity in reversed(waits) if full_first else waits:
                while not bar.done(parity):
                    yield
            if stage_tag[s] != q:
                raise Stale(f"k-block {q} read stage {s} holding {stage_tag[s]}")
            partial_tag[b] = None   # being written

            def finish(q=q, s=s, b=b):
                if stage_tag[s] != q:
                    raise Stale(f"stage {s} was refilled under k-block {q}")
                partial_tag[b] = q
                empty[s].arrive()
            commits.append((r, finish))
            commits.append((r, pfull[b].arrive))
            yield

    def accumulator():
        for q in range(kblocks):
            b = q % partials
            while not pfull[b].done(q // partials & 1):
                yield
            if partial_tag[b] != q:
                raise Stale(f"k-block {q} added from partial {b} holding {partial_tag[b]}")
            yield
            if partial_tag[b] != q:
                raise Stale(f"partial {b} was overwritten under k-block {q}")
            pempty[b].arrive()

    def land():
        if loads:
            s, q = loads.pop(rng.randrange(len(loads)))
            stage_tag[s] = q
            full[s].arrive()

    def commit():
        if commits:
            r = rng.choice([c[0] for c in commits])
            commits.pop(next(i for i, c in enumerate(commits) if c[0] == r))[1]()

    land_rate = rng.choice([0.2, 0.02])   # loads as fast as the rest, or far behind it
    agents = [producer()] + [issuer(r) for r in range(issuers)] + [accumulator() for _ in range(warps)]
    alive, idle = list(range(len(agents))), 0
    while alive:
        if rng.random() < land_rate:
            land()
        if rng.random() < 0.3:
            commit()
        a = rng.choice(alive)
        try:
            next(agents[a])
            idle += 1
        except StopIteration:
            alive.remove(a)
            idle = 0
        assert idle < 50000, f"deadlock: agents {alive} still waiting"


FORMS = {"wide": (2, 2, 8), "narrow": (1, 8, 4)}


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("stages", [2, 3, 4, 5])
def test_protocol_completes_without_stale_reads(form, stages):
    rng = random.Random(stages)
    for trial in range(20):
        run(rng.randint(1, 40), stages, *FORMS[form], trial)


def test_model_catches_the_exchanged_waits():
    with pytest.raises(Stale):
        for seed in range(50):
            run(40, 3, *FORMS["wide"], seed, full_first=True)
