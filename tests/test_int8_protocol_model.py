"""Host model of the int8 GEMM kernel's barrier protocol (gemm_int8.cuh): the two TMA producers, the weights'
warpgroups in turn, the two MMA issuers and the summing warps over modelled mbarriers under random
interleavings.  Loads land in any order and MMAs complete late.  A wait returns on the parity of the phase
alone, as the hardware's does, so an actor that falls two phases behind is let through too early: the model
then meets a stage with another k-block than it expects, or a barrier with more arrivals than it counts.

The kernel's forms come through; forms that break one of its rules (a stage always the same warpgroup's, the
same issuer's; converted k-blocks for every warpgroup) are caught, which shows that the model can."""
import random

import pytest

FOLD = 8


class Wrong(Exception):
    pass


class Barrier:
    def __init__(self, count):
        self.count, self.pending, self.phase = count, count, 0

    def arrive(self):
        if self.pending == 0:
            raise Wrong("an arrival too many")
        self.pending -= 1
        if self.pending == 0:
            self.phase += 1
            self.pending = self.count

    def done(self, parity):   # what mbarrier.try_wait.parity answers
        return (self.phase & 1) != parity


class Ring:
    def __init__(self, n):
        self.n, self.at, self.phase = n, 0, 0

    def next(self):
        self.at += 1
        if self.at == self.n:
            self.at, self.phase = 0, self.phase ^ 1


def simulate(seed, blocks, stages, cv, xs, wsets, bufs, global_parity=True):
    """blocks: k-blocks of each tile.  Runs to the end or raises."""
    rng = random.Random(seed)
    bars = lambda n, c: [Barrier(c) for _ in range(n)]  # noqa: E731
    full, empty, cv_full, cv_empty = bars(stages, 1), bars(stages, 1), bars(cv, 1), bars(cv, 1)
    x_full, x_empty = bars(xs, 1), bars(xs, 1)
    acc_full, acc_empty = [bars(bufs, 1) for _ in range(2)], [bars(bufs, 1) for _ in range(2)]
    w_smem, w_tmem, x_smem = [None] * stages, [None] * cv, [None] * xs
    acc = [[None] * bufs for _ in range(2)]          # k-blocks summed in each accumulator
    total = sum(blocks)
    flying = []                                      # loads under way: (function)
    mma = [[], []]                                   # each issuer's queue of MMAs and commits, in order
    summed = []

    def producer(n, ring, fulls, empties, where):
        for i in range(n):
            while not empties[ring.at].done(ring.phase ^ 1):
                yield
            at = ring.at

            def land(at=at, i=i):
                where[at] = i
                fulls[at].arrive()
            flying.append(land)
            ring.next()
            yield

    def weights(which):
        r, t = Ring(stages), Ring(cv)
        for _ in range(which):
            r.next(), t.next()
        for i in range(which, total, wsets):
            while not full[r.at].done(r.phase):
                yield
            if w_smem[r.at] != i:
                raise Wrong(f"weights of {w_smem[r.at]}, not of {i}")
            while not cv_empty[t.at].done(t.phase ^ 1):
                yield
            yield
            w_tmem[t.at] = i
            yield
            cv_full[t.at].arrive()
            empty[r.at].arrive()
            for _ in range(wsets):
                r.next(), t.next()

    def issuer(which):
        r, x, a = Ring(cv), Ring(xs), Ring(bufs)
        count = 0
        for n in blocks:
            for i in range(n):
                if ((count if global_parity else i) & 1) == which:
                    in_fold = (i >> 1) % FOLD
                    while in_fold == 0 and not acc_empty[which][a.at].done(a.phase ^ 1):
                        yield
                    while not x_full[x.at].done(x.phase):
                        yield
                    while not cv_full[r.at].done(r.phase):
                        yield

                    def run(kb=count, r=r.at, x=x.at, a=a.at, fresh=in_fold == 0):
                        if w_tmem[r] != kb or x_smem[x] != kb:
                            raise Wrong(f"operands of {w_tmem[r]} and {x_smem[x]}, not of {kb}")
                        acc[which][a] = [kb] if fresh else acc[which][a] + [kb]
                        if len(acc[which][a]) > FOLD:
                            raise Wrong("more than an accumulator holds exactly")
                    mma[which].append(run)
                    mma[which].append(cv_empty[r.at].arrive)
                    mma[which].append(x_empty[x.at].arrive)
                    if in_fold == FOLD - 1 or i + 2 >= n:
                        mma[which].append(acc_full[which][a.at].arrive)
                        a.next()
                    yield
                r.next(), x.next()
                count += 1

    def sums():
        ring = [Ring(bufs), Ring(bufs)]
        count = 0
        for n in blocks:
            got, i = [], 0
            while i < n:
                w = ((count + i) if global_parity else i) & 1
                a = ring[w]
                while not acc_full[w][a.at].done(a.phase):
                    yield
                got += acc[w][a.at]
                yield
                acc_empty[w][a.at].arrive()
                a.next()
                i += 2 * FOLD - 1 if i & 1 else 1
            if sorted(got) != list(range(count, count + n)):
                raise Wrong(f"a tile of {n} from {count} summed {got}")
            summed.append(n)
            count += n

    actors = [producer(total, Ring(stages), full, empty, w_smem), producer(total, Ring(xs), x_full, x_empty, x_smem), issuer(0), issuer(1), sums()]
    actors += [weights(s) for s in range(wsets)]
    # some actors far slower than others, differently from run to run
    speed = [rng.choice([1, 1, 4, 20]) for _ in actors]
    land, execute = rng.choice([1, 3, 12]), rng.choice([1, 3, 12])
    idle = 0
    while len(summed) < len(blocks):
        before = (len(summed), len(flying), sum(map(len, mma)), [b.phase for b in full + cv_full + cv_empty + x_full])
        for _ in range(64):
            pick = rng.choices(range(len(actors) + 3), weights=speed + [land, execute, execute])[0]
            if pick < len(actors):
                try:
                    next(actors[pick])
                except StopIteration:
                    pass
            elif pick == len(actors):
                if flying:
                    flying.pop(rng.randrange(len(flying)))()
            else:
                q = mma[pick - len(actors) - 1]
                if q:
                    q.pop(0)()
        after = (len(summed), len(flying), sum(map(len, mma)), [b.phase for b in full + cv_full + cv_empty + x_full])
        idle = idle + 1 if after == before else 0
        if idle > 400:
            raise Wrong("nothing moves")
    assert summed == list(blocks)


#      rows: stages, cv, xs, wsets, bufs
FORMS = {16: (12, 6, 6, 3, 2), 32: (9, 6, 8, 3, 2), 64: (6, 6, 6, 3, 1), 128: (4, 4, 4, 2, 1)}
TILES = [[1] * 9, [2, 1, 3, 1, 1, 2], [17] * 4, [33, 32, 31], [4, 5, 16, 17, 18, 1], [64, 3]]


@pytest.mark.parametrize("rows", sorted(FORMS))
@pytest.mark.parametrize("tiles", TILES, ids=str)
def test_the_kernels_forms_come_through(rows, tiles):
    for seed in range(12):
        simulate(seed, tiles, *FORMS[rows])


@pytest.mark.parametrize("broken", [dict(stages=7, cv=6, xs=6, wsets=4, bufs=2),                        # a stage of several warpgroups
                                    dict(stages=8, cv=6, xs=6, wsets=4, bufs=2, global_parity=False),   # a stage of both issuers, after an odd tile
                                    dict(stages=8, cv=7, xs=6, wsets=4, bufs=2), dict(stages=8, cv=6, xs=3, wsets=4, bufs=2),
                                    dict(stages=8, cv=2, xs=6, wsets=4, bufs=2)], ids=str)
def test_broken_forms_are_caught(broken):
    with pytest.raises(Wrong):
        for seed in range(400):
            simulate(seed, [17] * 6, **broken)


def test_the_forms_are_the_kernels():
    """FORMS against the constants of Int8Cfg, recomputed from its definition."""
    for nt, (stages, cv, xs, wsets, bufs) in FORMS.items():
        assert wsets == (2 if nt == 128 else 3) and bufs == (1 if nt >= 64 else 2) and xs == {32: 8, 128: 4}.get(nt, 6)
        assert cv == (512 - 2 * bufs * nt) // 128 * 2
        fixed = 1024 + xs * nt * 256 + (3 * 512 + 4) * 4 + 512
        assert stages == (232448 - fixed) // 16384 // wsets * wsets
        assert stages % wsets == 0 and cv >= wsets and cv % 2 == 0 and xs % 2 == 0
