"""Host model of the barriers between the roles of a prompt-attention CTA: loading warps,
the issuer of the products, and two halves of softmax warps. The roles run as
generators in random order, the products' commits land late but in order. Every parity wait
names the phase that it means: the model checks that the barrier is in that phase or just past
it (a parity cannot be mistaken), that nobody waits for ever, and that buffers are written
only when their readers are done. No GPU involved."""

import random

import pytest

LOADERS = 4
SIDES = 8


class Barrier:
    def __init__(self, count):
        self.count, self.left, self.done = count, count, 0

    def arrive(self):
        assert self.left > 0
        self.left -= 1
        if self.left == 0:
            self.left, self.done = self.count, self.done + 1


class Model:
    def __init__(self, segments, stages, halves, seed):
        self.segments, self.stages, self.halves = segments, stages, halves
        self.rng = random.Random(seed)
        ring = range(stages)
        self.k_full, self.v_full = ([Barrier(LOADERS) for _ in ring] for _ in range(2))
        self.k_empty, self.v_empty = ([Barrier(1) for _ in ring] for _ in range(2))
        self.q_full = [Barrier(4) for _ in range(2)]
        self.s_full, self.o_full = ([Barrier(1) for _ in range(2)] for _ in range(2))
        self.p_full, self.o_empty = ([Barrier(4) for _ in range(2)] for _ in range(2))
        self.both, self.maxed = Barrier(8), Barrier(LOADERS)
        self.queue = []                 # products and commits under way, in order
        self.k_holds, self.v_holds = [None] * stages, [None] * stages
        self.q_holds = [[None] * 4 for _ in range(2)]
        self.side = [[None] * LOADERS for _ in range(SIDES)]
        self.s_holds, self.o_holds = [None, None], [[], []]
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

    def loader(self, w):
        stage = use = tile = 0
        for n, (rows, tiles) in enumerate(self.segments):
            if tiles == 0:
                continue
            for i in range(tiles):
                self.side[tile % SIDES][w] = (n, i)
                self.maxed.arrive()
                yield from self.wait(self.maxed, tile)
                yield from self.wait(self.k_empty[stage], use - 1)
                self.k_holds[stage] = (n, i)
                self.k_full[stage].arrive()
                yield
                yield from self.wait(self.v_empty[stage], use - 1)
                self.v_holds[stage] = (n, i)
                self.v_full[stage].arrive()
                tile += 1
                stage += 1
                if stage == self.stages:
                    stage, use = 0, use + 1
                yield

    def issuer(self):
        k = v = 0                       # tiles used
        p, oe, q = [0, 0], [0, 0], [0, 0]
        for n, (rows, tiles) in enumerate(self.segments):
            if tiles == 0:
                continue
            streams = self.streams(rows)
            tasks = tiles * streams

            def scores(t):
                nonlocal k
                stream = t % streams
                stage = k % self.stages
                if t < streams:
                    yield from self.wait(self.q_full[stream], q[stream])
                    q[stream] += 1
                if stream == 0:
                    yield from self.wait(self.k_full[stage], k // self.stages)
                self.queue.append(("s", t & 1, (n, t // streams, stream), stage))
                self.queue.append(self.s_full[t & 1])
                if stream == streams - 1:
                    self.queue.append(self.k_empty[stage])
                    k += 1

            yield from scores(0)
            if tasks > 1:
                yield from scores(1)
            for t in range(tasks):
                stream, slot, stage = t % streams, t & 1, v % self.stages
                if t < streams:
                    yield from self.wait(self.o_empty[stream], oe[stream] - 1)
                    oe[stream] += 1
                if stream == 0:
                    yield from self.wait(self.v_full[stage], v // self.stages)
                yield from self.wait(self.p_full[slot], p[slot])
                p[slot] += 1
                self.queue.append(("o", slot, (n, t // streams, stream), stage))
                self.queue.append(self.o_full[stream])
                if stream == streams - 1:
                    self.queue.append(self.v_empty[stage])
                    v += 1
                if t + 2 < tasks:
                    yield from scores(t + 2)
                yield

    def softmax(self, me, w):
        s, o, both, tile = [0, 0], 0, 0, 0

        def load_q(n):
            if n < len(self.segments) and self.segments[n][1] and \
                    me < self.streams(self.segments[n][0]):
                self.q_holds[me][w] = n
                self.q_full[me].arrive()

        load_q(0)
        for n, (rows, tiles) in enumerate(self.segments):
            streams = self.streams(rows)
            mine = me < streams
            if mine and tiles:
                for i in range(tiles):
                    slot = me if streams == 2 else i & 1
                    yield from self.wait(self.s_full[slot], s[slot])
                    s[slot] += 1
                    assert self.s_holds[slot] == (n, i, me)
                    yield
                    if i > 0 and streams == 1:
                        yield from self.wait(self.o_full[me], o - 1)
                    if i > 0 and self.rng.random() < 0.5:     # rescales O
                        assert self.o_holds[me][-1] == (n, i - 1, me)
                        yield
                    assert self.s_holds[slot] == (n, i, me)
                    assert self.side[(tile + i) % SIDES] == [(n, i)] * LOADERS
                    self.p_full[slot].arrive()
                    o += 1
                    yield
            load_q(n + 1)
            if mine and tiles:
                yield from self.wait(self.o_full[me], o - 1)
                assert self.o_holds[me] == [(n, i, me) for i in range(tiles)]
            if tiles:
                if streams == 2:
                    s[me ^ 1] += tiles
                elif not mine:
                    s[0] += (tiles + 1) // 2
                    s[1] += tiles // 2
                tile += tiles
                if streams == 1 and self.halves == 2:
                    self.both.arrive()
                    yield from self.wait(self.both, both)
                    both += 1
            if mine:
                yield
                if tiles:
                    assert self.o_holds[me] == [(n, i, me) for i in range(tiles)]
                    self.o_empty[me].arrive()
                self.out.append((n, me, w))

    def tensor_core(self):
        """One queued product or commit."""
        x = self.queue.pop(0)
        if isinstance(x, Barrier):
            x.arrive()
            return
        kind, slot, task, stage = x
        n, i, stream = task
        if kind == "s":
            assert self.k_holds[stage] == (n, i) and self.q_holds[stream] == [n] * 4
            self.s_holds[slot] = task
        else:
            assert self.v_holds[stage] == (n, i) and self.s_holds[slot] == task
            if i == 0:
                self.o_holds[stream] = []
            self.o_holds[stream].append(task)

    def run(self):
        roles = [self.loader(w) for w in range(LOADERS)] + [self.issuer()]
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
    for trial in range(300):
        segments = [(rng.choice((5, 128, 129, 256)), rng.choice((0, 1, 1, 2, 3, 4, 7)))
                    for _ in range(rng.randint(1, 7))]
        m = Model(segments, stages, halves, trial)
        m.run()
        want = [(n, me, w) for n, (rows, _) in enumerate(segments)
                for me in range(m.streams(rows)) for w in range(4)]
        assert sorted(m.out) == sorted(want)
