"""Host model of the barriers between the roles of a prompt-attention CTA: the warp that
hands out segments, loading warps of keys and of values, the issuer of the products, and
two halves of softmax warps. The roles run as generators in random order, the products'
commits land late but in order. Every parity wait
names the phase that it means: the model checks that the barrier is in that phase or just past
it (a parity cannot be mistaken), that nobody waits for ever, and that buffers are written
only when their readers are done. No GPU involved."""

import random

import pytest

LOADERS = 4
SIDES = 8
RING = 16
AHEAD = 6      # tiles that a loading warp has looked up, the one it lays out included


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
        self.k_empty, self.v_empty = ([Barrier(1) for _ in ring] for _ in range(2))
        self.q_full = [Barrier(4) for _ in range(2)]
        self.s_full, self.p_full = ([Barrier(n) for _ in range(2)] for n in (1, 4))
        self.o_full, self.o_empty = ([Barrier(n) for _ in range(2)] for n in (1, 4))
        self.maxed = [Barrier(LOADERS) for _ in range(2)]
        readers = 4 * halves + 2 * LOADERS + 1
        self.seg_full = [Barrier(1) for _ in range(RING)]
        self.seg_empty = [Barrier(readers) for _ in range(RING)]
        self.ring = [None] * RING
        self.queue = []                 # products and commits under way, in order
        self.holds = [[[None] * LOADERS for _ in range(stages)] for _ in range(2)]
        self.q_holds = [[None] * 4 for _ in range(2)]
        self.side = [[None] * LOADERS for _ in range(SIDES)]
        self.s_holds, self.o_holds = [None] * 2, [[], []]
        self.out = []

    def mode(self, n):
        """0: the first half alone; 1: the same rows, every other tile; 2: rows of their own."""
        rows, tiles = self.segments[n]
        if self.halves == 1:
            return 0
        return 2 if rows > 128 else 1 if rows == 128 and tiles >= 4 else 0

    def tiles_of(self, n, me):
        mode, tiles = self.mode(n), self.segments[n][1]
        if mode == 0:
            return list(range(tiles)) if me == 0 else []
        return list(range(me, tiles, 2)) if mode == 1 else list(range(tiles))

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
            while more and len(tiles) < AHEAD:
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

    def issuer(self):
        queue = self.queue
        k = v = number = 0              # tiles used
        p, q, oe = [0, 0], [0, 0], [0, 0]
        while (yield from self.take(number)):
            n = number
            mode, tiles = self.mode(n), self.segments[n][1]
            self.release(number)
            number += 1
            tasks = 2 * tiles if mode == 2 else tiles
            each = 1 if mode == 0 else 2        # streams
            ahead = self.slots if mode == 0 else 2

            def of(t):
                stream = t % each
                return stream, (t % 2 if self.slots == 2 else stream), t // 2 if mode == 2 else t

            def closes(t):
                return mode != 2 or t % 2 == 1

            def opens(t):
                return mode != 2 or t % 2 == 0

            def scores(t):
                nonlocal k
                stream, slot, tile = of(t)
                stage = k % self.stages
                if t < each:
                    yield from self.wait(self.q_full[stream], q[stream])
                    q[stream] += 1
                if opens(t):
                    yield from self.wait(self.k_full[stage], k // self.stages)
                queue.append(("s", slot, (n, tile, stream), stage))
                queue.append(self.s_full[slot])
                if closes(t):
                    queue.append(self.k_empty[stage])
                    k += 1

            for t in range(min(tasks, ahead)):
                yield from scores(t)
            for t in range(tasks):
                stream, slot, tile = of(t)
                stage = v % self.stages
                if t < each:
                    yield from self.wait(self.o_empty[stream], oe[stream] - 1)
                    oe[stream] += 1
                if opens(t):
                    yield from self.wait(self.v_full[stage], v // self.stages)
                yield from self.wait(self.p_full[slot], p[slot])
                p[slot] += 1
                queue.append(("o", slot, (n, tile, stream), stage))
                if self.slots == 2 or t >= tasks - each:
                    queue.append(self.o_full[stream])
                if closes(t):
                    queue.append(self.v_empty[stage])
                    v += 1
                if t + ahead < tasks:
                    yield from scores(t + ahead)
                yield

    def softmax(self, me, w):
        s, o, tile = [0, 0], 0, 0

        def load_q(n):
            if self.tiles_of(n, me):
                self.q_holds[me][w] = n
                self.q_full[me].arrive()

        number = 0
        running = yield from self.take(0)
        if running:
            load_q(0)
        while running:
            n = number
            mine = self.tiles_of(n, me)
            for at, i in enumerate(mine):
                turn = i % 2 if self.slots == 2 else 0
                slot, waited = me + turn, self.slots == 1
                yield from self.wait(self.s_full[slot], s[turn])
                s[turn] += 1
                assert self.s_holds[slot] == (n, i, me)
                yield
                if at > 0 and self.rng.random() < 0.5:     # rescales O
                    if not waited:
                        yield from self.wait(self.o_full[me], o - 1)
                        waited = True
                    assert self.o_holds[me][-1] == (n, mine[at - 1], me)
                    yield
                assert self.s_holds[slot] == (n, i, me)
                assert self.side[(tile + i) % SIDES] == [(n, i)] * LOADERS
                if at > 0 and not waited:
                    yield from self.wait(self.o_full[me], o - 1)
                self.p_full[slot].arrive()
                if self.slots == 2 or at == len(mine) - 1:
                    o += 1
                yield
            running = yield from self.take(number + 1)
            if running:
                load_q(number + 1)
            if mine:
                yield from self.wait(self.o_full[me], o - 1)
                assert self.o_holds[me] == [(n, i, me) for i in mine]
            tile += self.segments[n][1]
            if mine:
                yield
                assert self.o_holds[me] == [(n, i, me) for i in mine]
                self.o_empty[me].arrive()
                self.out.append((n, me, w))
            self.release(number)
            number += 1

    def tensor_core(self):
        """One queued product or commit."""
        x = self.queue.pop(0)
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
            if i == self.tiles_of(n, stream)[0]:
                self.o_holds[stream] = []
            self.o_holds[stream].append(task)

    def run(self):
        roles = [self.loader(x, w) for x in range(2) for w in range(LOADERS)]
        roles += [self.issuer(), self.planner()]
        roles += [self.softmax(me, w) for me in range(self.halves) for w in range(4)]
        idle = 0
        speed = [self.rng.choice((1, 1, 3, 10, 40)) for _ in roles]
        while roles:
            before = len(self.queue)
            if self.queue and self.rng.random() < 0.3:
                self.tensor_core()
                idle = 0
            i = self.rng.randrange(len(roles))
            if self.rng.randrange(speed[i]) == 0:
                try:
                    next(roles[i])
                except StopIteration:
                    roles.pop(i)
                    speed.pop(i)
                    idle = 0
            idle = 0 if len(self.queue) != before else idle + 1
            assert idle < 20000, "a role waits for ever"
        while self.queue:
            self.tensor_core()


@pytest.mark.parametrize("halves,stages", [(2, 2), (2, 3), (1, 2)])
def test_roles_of_a_cta(halves, stages):
    rng = random.Random(halves * 10 + stages)
    for trial in range(50):
        segments = [(rng.choice((5, 128, 129, 256)), rng.choice((1, 1, 1, 2, 3, 4, 7)))
                    for _ in range(rng.randint(0, 40))]
        m = Model(segments, stages, halves, trial)
        m.run()
        want = [(n, me, w) for n in range(len(segments))
                for me in range(halves) if m.tiles_of(n, me) for w in range(4)]
        assert sorted(m.out) == sorted(want)
