"""CPU model of the barrier protocol of the kernel of many query rows over the
4-bit history (history_chunk.cu): the record warp, the K and V producers, the MMA
warp and the two softmax warpgroups as processes over mbarriers with phases and
parities, run under random interleavings.

Checked: every run ends (no deadlock); a wait on a parity that passes passes for
the phase that it means, never for one two away; and no buffer is overwritten
while somebody may still read it."""
import random

import pytest


class Bar:
    """An mbarrier: phase counter and the arrivals that the phase still expects."""

    def __init__(self, count):
        self.count, self.left, self.phase = count, count, 0

    def arrive(self):
        assert self.left > 0, "more arrivals than the phase expects"
        self.left -= 1
        if self.left == 0:
            self.phase += 1
            self.left = self.count

    def passed(self, parity):
        return (self.phase & 1) != parity


class Model:
    def __init__(self, segments, seed):
        """segments: [(tiles T, has1, part)] of one block."""
        self.rng = random.Random(seed)
        self.segs = segments
        two = lambda c: [Bar(c), Bar(c)]  # noqa: E731
        self.q_full, self.k_full, self.k_empty = two(4), two(3), two(1)
        self.s_full, self.p_full, self.o_full = two(1), two(4), two(1)
        self.v_full, self.v_empty = two(3), two(1)
        self.tile_full = [Bar(1) for _ in range(4)]
        self.tile_empty = [Bar(1) for _ in range(4)]
        self.part, self.join = two(4), two(1)
        self.mma = []            # issued products and commits, in order
        self.record, self.K, self.V, self.S, self.P, self.O, self.Q = {}, {}, {}, {}, {}, {}, {}

    # a wait for phase `index` of the barrier: by parity, and checked
    def wait(self, bar, index):
        while not bar.passed(index & 1):
            yield
        assert bar.phase >= index + 1, "a wait passed before its phase"
        assert bar.phase <= index + 2

    def recorder(self):
        for n in range(sum(T for T, _, _ in self.segs)):
            yield from self.wait_free(self.tile_empty[n % 4], n >> 2)
            yield
            self.record[n % 4] = n
            self.tile_full[n % 4].arrive()

    def producer(self, is_v):
        buf = self.V if is_v else self.K
        full, empty = (self.v_full, self.v_empty) if is_v else (self.k_full, self.k_empty)
        for n in range(sum(T for T, _, _ in self.segs)):
            yield from self.wait(self.tile_full[n % 4], n >> 2)
            yield from self.wait_free(empty[n & 1], n >> 1)
            assert self.record[n % 4] == n
            yield
            assert self.record[n % 4] == n
            buf[n & 1] = n
            full[n & 1].arrive()

    def wait_free(self, bar, use):
        """A place's `use`-th use: free once its (use - 1)-th was released."""
        if use > 0:
            yield from self.wait(bar, use - 1)
        else:
            assert bar.passed(1)

    def issuer(self):
        n0, segs, segs1, pc1 = 0, 0, 0, 0
        for T, has1, part in self.segs:
            yield from self.wait(self.q_full[0], segs)
            segs += 1
            if has1:
                yield from self.wait(self.q_full[1], segs1)
                segs1 += 1
            yield from self.wait(self.k_full[n0 & 1], n0 >> 1)
            qk = lambda k, n: self.mma.extend([("qk", k, n), ("commit", self.s_full[k])])  # noqa: E731
            qk(0, n0)
            if has1:
                qk(1, n0)
            self.mma.append(("commit", self.k_empty[n0 & 1]))
            for t in range(T):
                n, more = n0 + t, t + 1 < T
                yield from self.wait(self.v_full[n & 1], n >> 1)
                yield from self.wait(self.p_full[0], n)
                self.mma.append(("pv", 0, n))
                if not more:
                    self.mma.append(("commit", self.o_full[0]))
                if more:
                    yield from self.wait(self.k_full[(n + 1) & 1], (n + 1) >> 1)
                    qk(0, n + 1)
                if has1:
                    yield from self.wait(self.p_full[1], pc1)
                    pc1 += 1
                    self.mma.append(("pv", 1, n))
                    if not more:
                        self.mma.append(("commit", self.o_full[1]))
                    if more:
                        qk(1, n + 1)
                if more:
                    self.mma.append(("commit", self.k_empty[(n + 1) & 1]))
                self.mma.append(("commit", self.v_empty[n & 1]))
                self.mma.append(("commit", self.tile_empty[n % 4]))
            n0 += T

    def softmax(self, kt, w):
        n = sc = segs = parts = 0
        for seg, (T, has1, part) in enumerate(self.segs):
            if kt and not has1:
                n += T
                continue
            self.Q[kt, w] = seg
            self.q_full[kt].arrive()
            for u in range(T):
                yield from self.wait(self.s_full[kt], sc)
                yield from self.wait(self.tile_full[n % 4], n >> 2)
                assert self.record[n % 4] == n and self.S[kt] == n
                yield
                assert self.S[kt] == n and self.record[n % 4] == n
                self.P[kt, w] = n
                self.p_full[kt].arrive()
                n += 1
                sc += 1
            yield from self.wait(self.o_full[kt], segs)
            segs += 1
            assert self.O[kt] == (seg, T)
            yield
            if part:
                self.part[kt].arrive()
                if w == 0:
                    yield from self.wait(self.part[kt], parts)
                    self.join[kt].arrive()
                yield from self.wait(self.join[kt], parts)
                parts += 1

    def seg_of(self, n):
        for s, (T, _, _) in enumerate(self.segs):
            if n < T:
                return s, n
            n -= T

    def hardware(self):
        """Products run in order, at any time."""
        if self.mma:
            op = self.mma.pop(0)
            if op[0] == "commit":
                op[1].arrive()
            elif op[0] == "qk":
                _, k, n = op
                assert self.K[n & 1] == n
                assert all(self.Q[k, w] == self.seg_of(n)[0] for w in range(4))
                self.S[k] = n
            else:
                _, k, n = op
                assert self.V[n & 1] == n and all(self.P[k, w] == n for w in range(4))
                s, t = self.seg_of(n)
                assert t == 0 or self.O[k] == (s, t)
                self.O[k] = (s, t + 1)

    def run(self):
        procs = [self.producer(v) for v in (False, True) for _ in range(3)]
        procs += [self.recorder(), self.issuer()]
        procs += [self.softmax(kt, w) for kt in range(2) for w in range(4)]
        idle = 0
        while procs or self.mma:
            if self.rng.random() < 0.3:
                self.hardware()
                continue
            if not procs:
                self.hardware()
                continue
            p = self.rng.choice(procs)
            before = self.state()
            try:
                next(p)
            except StopIteration:
                procs.remove(p)
                idle = 0
                continue
            idle = 0 if self.state() != before or self.mma else idle + 1
            assert idle < 3000, "deadlock"

    def state(self):
        return tuple((b.phase, b.left) for v in vars(self).values()
                     for b in (v if isinstance(v, list) else [v]) if isinstance(b, Bar))


@pytest.mark.parametrize("segs", [
    [(1, False, False)], [(1, True, False)], [(3, True, False), (1, True, True)],
    [(2, True, True), (1, True, False), (1, True, False)],
    [(5, False, True), (1, True, False), (2, False, False), (7, True, True)],
    [(1, True, False)] * 6, [(6, False, False), (6, True, True)], [(4, True, True), (9, False, True)],
])
def test_every_interleaving_ends_and_no_buffer_is_reused_early(segs):
    for seed in range(12):
        Model(segs, seed).run()
