"""Host model of the barriers between the roles of a prompt-attention CTA: the warp that
hands out segments, loading warps of keys and of values, an issuer of products and four
softmax warps for each half of the rows. The roles run as generators in random order, the
commits of an issuer's products land late but in its order. Every parity wait
names the phase that it means: the model checks that the barrier is in that phase or just past
it (a parity cannot be mistaken), that nobody waits for ever, and that buffers are written
only when their readers are done. No GPU involved."""

import random

import pytest

LOADERS = 4
SIDES = 8
RING = 16


class Barrier:
    def __init__(self, count):
        self.count, self.left, self.done = count, count, 0

    def arrive(self):
        assert self.left > 0
        self.left -= 1
        if self.left == 0:
            self.left, self.done = self.count, self.done + 1


class Model:
    """Segments are (rows, tiles)."""

    def __init__(self, segments, stages, halves, seed):
        self.segments, self.stages, self.halves = segments, stages, halves
        self.slots = 2 // halves        # tiles of scores of a half
        self.rng = random.Random(seed)
        ring = range(stages)
        self.k_full, self.v_full = ([Barrier(LOADERS) for _ in ring] for _ in range(2))
        self.k_empty, self.v_empty = ([Barrier(halves) for _ in ring] for _ in range(2))
        self.q_full = [Barrier(4) for _ in range(2)]
        self.s_full, self.p_full = ([Barrier(n) for _ in range(2)] for n in (1, 4))
        self.o_full, self.o_empty = ([Barrier(n) for _ in range(2)] for n in (1, 4))
        self.maxed = [Barrier(LOADERS) for _ in range(2)]
        readers = 5 * halves + 2 * LOADERS
        self.seg_full = [Barrier(1) for _ in range(RING)]
        self.seg_empty = [Barrier(readers) for _ in range(RING)]
        self.ring = [None] * RING
        self.queues = [[], []]          # an issuer's products and commits under way, in order
        self.holds = [[[None] * LOADERS for _ in range(stages)] for _ in range(2)]
        self.q_holds = [[None] * 4 for _ in range(2)]
        self.side = [[None] * LOADERS for _ in range(SIDES)]
        self.s_holds, self.o_holds = [None] * 2, [[], []]
        self.out = []

    def streams(self, rows):
        return 2 if rows > 128 and self.halves == 2 else 1

    @staticmethod
    def wait(barrier, phase):
        """Wait for the barrier's phase number `phase` through its parity."""
        if phase < 0:                   # a buffer that is empty at first
            return
        while True:
            assert barrier.done in (phase, phase + 1), (barrier.done, phase)
            if barrier.done == phase + 1:
                return
            yield

    def planner(self):
        for n in range(len(self.segments) + 1):   # (rows that see nothing get no segment)
            yield from self.wait(self.seg_empty[n % RING], n // RING - 1)
            self.ring[n % RING] = n if n < len(self.segments) else -1
            self.seg_full[n % RING].arrive()
            yield

    def take(self, n):
        yield from self.wait(self.seg_full[n % RING], n // RING)
        return self.ring[n % RING] >= 0

    def release(self, n):
        assert self.ring[n % RING] == n
        self.seg_empty[n % RING].arrive()

    def loader(self, which, w):
        full, empty = ((self.k_full, self.k_empty), (self.v_full, self.v_empty))[which]
        tiles, number = [], 0            # tiles asked for and not yet laid out
        more = True

        def ask():
            nonlocal number, more
            while more and len(tiles) < 4:
                more = yield from self.take(number)
                if more:
                    tiles.extend((number, i) for i in range(self.segments[number][1]))
                    self.release(number)
                    number += 1

        stage = use = tile = 0
        yield from ask()
        while tiles:
            n, i = tiles.pop(0)
            if which == 0:
                self.side[tile % SIDES][w] = (n, i)
            self.maxed[which].arrive()
            yield from self.wait(self.maxed[which], tile)
            yield from ask()
            yield from self.wait(empty[stage], use - 1)
            self.holds[which][stage][w] = (n, i)
            full[stage].arrive()
            tile += 1
            stage += 1
            if stage == self.stages:
                stage, use = 0, use + 1
            yield

    def issuer(self, me):
        queue = self.queues[me]
        k = v = number = q = oe = 0
        p = [0, 0]
        while (yield from self.take(number)):
            n = number
            rows, tiles = self.segments[n]
            self.release(number)
            number += 1
            mine = me < self.streams(rows)

            def scores(i):
                nonlocal k
                stage, slot = k % self.stages, me + i % self.slots
                yield from self.wait(self.k_full[stage], k // self.stages)
                if mine:
                    queue.append(("s", slot, (n, i, me), stage))
                    queue.append(self.s_full[slot])
                    queue.append(self.k_empty[stage])
                else:
                    self.k_empty[stage].arrive()
                k += 1

            if mine:
                yield from self.wait(self.q_full[me], q)
                q += 1
            for i in range(min(tiles, self.slots)):
                yield from scores(i)
            for i in range(tiles):
                stage, slot = v % self.stages, me + i % self.slots
                if mine and i == 0:
                    yield from self.wait(self.o_empty[me], oe - 1)
                    oe += 1
                yield from self.wait(self.v_full[stage], v // self.stages)
                if mine:
                    yield from self.wait(self.p_full[slot], p[i % self.slots])
                    p[i % self.slots] += 1
                    queue.append(("o", slot, (n, i, me), stage))
                    queue.append(self.o_full[me])
                    queue.append(self.v_empty[stage])
                else:
                    self.v_empty[stage].arrive()
                v += 1
                if i + self.slots < tiles:
                    yield from scores(i + self.slots)
                yield

    def softmax(self, me, w):
        s, o, tile = [0, 0], 0, 0

        def load_q(n):
            if self.segments[n][1] and me < self.streams(self.segments[n][0]):
                self.q_holds[me][w] = n
                self.q_full[me].arrive()

        number = 0
        running = yield from self.take(0)
        if running:
            load_q(0)
        while running:
            n = number
            rows, tiles = self.segments[n]
            mine = me < self.streams(rows)
            if mine:
                for i in range(tiles):
                    turn = i % self.slots
                    slot, waited = me + turn, self.slots == 1
                    yield from self.wait(self.s_full[slot], s[turn])
                    s[turn] += 1
                    assert self.s_holds[slot] == (n, i, me)
                    yield
                    if i > 0 and self.rng.random() < 0.5:     # rescales O
                        if not waited:
                            yield from self.wait(self.o_full[me], o - 1)
                            waited = True
                        assert self.o_holds[me][-1] == (n, i - 1, me)
                        yield
                    assert self.s_holds[slot] == (n, i, me)
                    assert self.side[(tile + i) % SIDES] == [(n, i)] * LOADERS
                    if i > 0 and not waited:
                        yield from self.wait(self.o_full[me], o - 1)
                    self.p_full[slot].arrive()
                    o += 1
                    yield
            running = yield from self.take(number + 1)
            if running:
                load_q(number + 1)
            if mine and tiles:
                yield from self.wait(self.o_full[me], o - 1)
                assert self.o_holds[me] == [(n, i, me) for i in range(tiles)]
            tile += tiles
            if mine:
                yield
                if tiles:
                    assert self.o_holds[me] == [(n, i, me) for i in range(tiles)]
                    self.o_empty[me].arrive()
                self.out.append((n, me, w))
            self.release(number)
            number += 1

    def tensor_core(self, queue):
        """One queued product or commit."""
        x = queue.pop(0)
        if isinstance(x, Barrier):
            x.arrive()
            return
        kind, slot, task, stage = x
        n, i, stream = task
        if kind == "s":
            assert self.holds[0][stage] == [(n, i)] * LOADERS
            assert self.q_holds[stream] == [n] * 4
            self.s_holds[slot] = task
        else:
            assert self.holds[1][stage] == [(n, i)] * LOADERS
            assert self.s_holds[slot] == task
            if i == 0:
                self.o_holds[stream] = []
            self.o_holds[stream].append(task)

    def run(self):
        roles = [self.loader(x, w) for x in range(2) for w in range(LOADERS)]
        roles += [self.issuer(me) for me in range(self.halves)] + [self.planner()]
        roles += [self.softmax(me, w) for me in range(self.halves) for w in range(4)]
        idle = 0
        speed = [self.rng.choice((1, 1, 3, 10, 40)) for _ in roles]
        while roles:
            before = [len(x) for x in self.queues]
            queue = self.rng.choice(self.queues)
            if queue and self.rng.random() < 0.3:
                self.tensor_core(queue)
                idle = 0
            i = self.rng.randrange(len(roles))
            if self.rng.randrange(speed[i]) == 0:
                try:
                    next(roles[i])
                except StopIteration:
                    roles.pop(i)
                    speed.pop(i)
                    idle = 0
            idle = 0 if [len(x) for x in self.queues] != before else idle + 1
            assert idle < 20000, "a role waits for ever"
        for queue in self.queues:
            while queue:
                self.tensor_core(queue)


@pytest.mark.parametrize("halves,stages", [(2, 2), (2, 3), (1, 2)])
def test_roles_of_a_cta(halves, stages):
    rng = random.Random(halves * 10 + stages)
    for trial in range(50):
        segments = [(rng.choice((5, 128, 129, 256)), rng.choice((1, 1, 1, 2, 3, 4, 7)))
                    for _ in range(rng.randint(0, 40))]
        m = Model(segments, stages, halves, trial)
        m.run()
        want = [(n, me, w) for n, (rows, _) in enumerate(segments)
                for me in range(m.streams(rows)) for w in range(4)]
        assert sorted(m.out) == sorted(want)
