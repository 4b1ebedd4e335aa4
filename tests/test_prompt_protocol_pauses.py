"""The host model of a prompt-attention CTA's barriers where the warp that hands out the work
pauses between segments, as it does for rows that see nothing. No GPU involved."""

import random

import pytest

from tests.test_prompt_protocol import RING, Model


class Pausing(Model):
    """(A pause of 8 of the slowest role's steps is some 8 x 40 x 18 steps of the model, which
    gives up after 20000 without progress.)"""

    def planner(self):
        for n in range(len(self.segments) + 1):
            for _ in range(self.rng.choice((0, 0, 0, 3, 8))):
                yield
            yield from self.wait(self.seg_empty[n % RING], n // RING - 1)
            self.ring[n % RING] = n if n < len(self.segments) else -1
            self.seg_full[n % RING].arrive()
            yield


@pytest.mark.parametrize("halves,stages", [(2, 2), (2, 3), (1, 2)])
def test_pauses_between_segments(halves, stages):
    rng = random.Random(halves * 100 + stages)
    for trial in range(40):
        segments = [(rng.choice((5, 128, 129, 256)), rng.choice((1, 1, 1, 2, 3, 4, 7)))
                    for _ in range(rng.randint(0, 40))]
        m = Pausing(segments, stages, halves, trial)
        m.run()
        want = [(n, me, w) for n in range(len(segments))
                for me in range(halves) if m.tiles_of(n, me) for w in range(4)]
        assert sorted(m.out) == sorted(want)
