"""A model of the barriers of the 8-bit products (fp8_many.cu: a pair of CTAs;
fp8_matmul.cu: one), checked on the CPU under random interleavings: when a CTA leaves,
nothing may still be on its way to its shared memory, which the next kernel's CTA gets.

On their own way travel the copies (bytes that land, then count on the leader's `full`
barrier) and the signals of the MMAs' commits (arrivals on `empty`, `tfull` and `drain` of
every CTA of the pair). No order between two of them is assumed. The agents follow the
kernels: per CTA a copying thread and summing warps, the leader's MMA thread. The negative
control is the exit as first written, which saw the last `tfull` and the leader's `drain`
only."""
import random

import pytest


class Late(Exception):
    """Something landed, or was still to land, in a CTA that had left."""


class Bar:
    def __init__(self, count):
        self.count, self.pend, self.tx, self.done = count, count, 0, 0

    def arrive(self):
        self.pend -= 1
        self._complete()

    def expect(self, n):
        self.tx += n
        self.arrive()

    def land(self, n):
        self.tx -= n
        self._complete()

    def _complete(self):
        if self.pend == 0 and self.tx == 0:
            self.done += 1
            self.pend = self.count
        assert self.pend >= 0

    def passes(self, parity):
        return (self.done & 1) != parity


def simulate(ctas, stages, blocks, seed, waits):
    """One launch of `blocks` blocks of the reduction; raises Late, or AssertionError on a
    deadlock."""
    rnd = random.Random(seed)
    R = range(ctas)
    full = [Bar(1) for _ in range(stages)]           # the leader's: every CTA's copies
    empty = [[Bar(1) for _ in range(stages)] for _ in R]
    tfull = [[Bar(1) for _ in range(2)] for _ in R]
    tempty = [Bar(ctas) for _ in range(2)]           # the leader's
    drain = [Bar(1) for _ in R]
    flying = []                                      # (CTA that it writes to, what it does)

    def commit(bars):
        for r in R:
            flying.append((r, bars[r].arrive))

    def copier(r):
        st, ph = 0, 0
        for _ in range(blocks):
            while not empty[r][st].passes(ph ^ 1):
                yield
            if r == 0:
                full[st].expect(ctas)
            flying.append((r, lambda st=st: full[st].land(1)))
            st, ph = (st + 1, ph) if st + 1 < stages else (0, ph ^ 1)
        last = range(max(0, blocks - stages), blocks)
        if r == 0:
            for i in last:
                while not full[i % stages].passes((i // stages) & 1):
                    yield
        if waits:
            for i in last:
                while not empty[r][i % stages].passes((i // stages) & 1):
                    yield
            if r != 0:
                while not drain[r].passes(0):
                    yield

    def mma():
        st, ph, ac, aph = 0, 0, 0, 0
        for _ in range(blocks):
            while not (full[st].passes(ph) and tempty[ac].passes(aph ^ 1)):
                yield
            commit([e[st] for e in empty])
            commit([t[ac] for t in tfull])
            st, ph = (st + 1, ph) if st + 1 < stages else (0, ph ^ 1)
            ac, aph = ac ^ 1, aph ^ ac
            yield
        commit(drain)
        while not drain[0].passes(0):
            yield

    def sums(r):
        ac, aph = 0, 0
        for _ in range(blocks):
            while not tfull[r][ac].passes(aph):
                yield
            tempty[ac].arrive()
            ac, aph = ac ^ 1, aph ^ ac
            yield

    agents = [copier(r) for r in R] + [sums(r) for r in R] + [mma()]
    idle = 0
    while agents:
        if flying and (idle > 4 * len(agents) or rnd.random() < 0.3):
            _, land = flying.pop(rnd.randrange(len(flying)))
            land()
            idle = 0
            continue
        a = rnd.choice(agents)
        try:
            next(a)
            idle += 1
            assert flying or idle < 10000, "deadlock"
        except StopIteration:
            agents.remove(a)
            idle = 0
    if flying:  # (the closing cluster barrier has been passed)
        raise Late(sorted(r for r, _ in flying))


SIZES = [(stages, blocks) for stages in (2, 4, 5) for blocks in (1, 2, 3, 4, 5, 7, 16, 41)]


@pytest.mark.parametrize("ctas", [1, 2])
@pytest.mark.parametrize("stages,blocks", SIZES)
def test_nothing_is_on_its_way_to_a_cta_that_has_left(ctas, stages, blocks):
    for seed in range(150):
        simulate(ctas, stages, blocks, seed, waits=True)


def test_model_catches_an_exit_without_the_waits():
    late = set()
    for seed in range(300):
        try:
            simulate(2, 5, 7, seed, waits=False)
        except Late as e:
            late.update(e.args[0])
    assert late == {0, 1}  # the second CTA's drain and both CTAs' last `empty` signals
