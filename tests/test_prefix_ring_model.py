"""The shared prefix's ring of K and V tiles as a model: one loader, a warp that issues scores, one that
issues outputs, and the softmax of two row tiles, each a sequence of steps whose barriers know a phase
only by its parity.  Loads land after any delay.  Over random interleavings every wait that passes must
have waited for the right use of its slot, and nobody is stuck.  With the ring's wait before the others
(the slot's use before may then still be under way) the model fails."""
import random

import pytest


class Barrier:
    def __init__(self, count):
        self.count, self.left, self.phase = count, count, 0

    def arrive(self):
        self.left -= 1
        assert self.left >= 0
        if self.left == 0:
            self.left, self.phase = self.count, self.phase + 1

    def passed(self, k):           # what a wait for phase k sees: a parity
        return (self.phase & 1) != (k & 1)


def run(segments, ring, seed, ring_wait_first=False):
    rng = random.Random(seed)
    full, empty = [Barrier(1) for _ in range(ring)], [Barrier(1) for _ in range(ring)]
    s_full, s_free, p_full, o_done = ([Barrier(1), Barrier(1)] for _ in range(4))
    q_full = Barrier(2)
    landed, flying = set(), []

    def k_at(j):
        return 0 if j == 0 else 2 * j - 1

    def v_at(j, n):
        return 2 * j + 2 if j + 1 < n else 2 * j + 1

    def loader():
        for c in range(sum(2 * n for n in segments)):
            if c >= ring:
                yield empty[c % ring], c // ring - 1
                assert empty[c % ring].phase == c // ring
            flying.append(c)

    def use(c):
        assert c in landed, ("tile used before it landed", c)

    def scores():
        i = c = 0
        for g, n in enumerate(segments):
            yield q_full, g
            for j in range(n):
                ck = c + k_at(j)
                ready = (full[ck % ring], ck // ring)
                if ring_wait_first:
                    yield ready
                for t in range(2):
                    if i + j > 0:
                        yield s_free[t], i + j - 1
                    if t == 0 and not ring_wait_first:
                        yield ready
                    use(ck)
                    s_full[t].arrive()
                empty[ck % ring].arrive()
            i, c = i + n, c + 2 * n

    def outputs():
        i = c = 0
        for n in segments:
            for j in range(n):
                cv = c + v_at(j, n)
                ready = (full[cv % ring], cv // ring)
                if ring_wait_first:
                    yield ready
                for t in range(2):
                    yield p_full[t], i + j
                    if t == 0 and not ring_wait_first:
                        yield ready
                    use(cv)
                    o_done[t].arrive()
                empty[cv % ring].arrive()
            i, c = i + n, c + 2 * n

    def softmax(t):
        i = 0
        for n in segments:
            q_full.arrive()
            for _ in range(n):
                yield s_full[t], i
                assert s_full[t].phase == i + 1
                s_free[t].arrive()
                if i > 0:
                    yield o_done[t], i - 1
                    assert o_done[t].phase == i
                p_full[t].arrive()
                i += 1
            yield o_done[t], i - 1
            assert o_done[t].phase == i

    actors = [loader(), scores(), outputs(), softmax(0), softmax(1)]
    waits = [None] * len(actors)
    weight = [rng.random() ** 3 + 0.01 for _ in range(len(actors) + 1)]     # some are slow for a whole run
    while any(a is not None for a in actors):
        ready = [x for x, a in enumerate(actors) if a is not None and (waits[x] is None or waits[x][0].passed(waits[x][1]))]
        if flying:
            ready.append(len(actors))
        assert ready, "stuck"
        x = rng.choices(ready, [weight[r] for r in ready])[0]
        if x == len(actors):
            c = flying.pop(rng.randrange(len(flying)))
            landed.add(c)
            full[c % ring].arrive()
            continue
        try:
            waits[x] = next(actors[x])
        except StopIteration:
            actors[x] = None


CASES = [[1], [2], [7], [1, 1, 1], [3, 1, 5], [12, 4]]


@pytest.mark.parametrize("ring", [3, 6])
@pytest.mark.parametrize("segments", CASES)
def test_every_wait_is_for_its_own_use(ring, segments):
    for seed in range(300):
        run(segments, ring, seed)


def test_the_model_sees_a_wait_for_the_wrong_use():
    seen = 0
    for seed in range(300):
        try:
            run([12, 4], 3, seed, ring_wait_first=True)
        except AssertionError:
            seen += 1
    assert seen > 0
