"""A model of the FP4 GEMMs' mbarrier protocols under randomized schedules, on
the CPU: the pair of CTAs with its one accumulator, and one CTA of the split
kernel. Barriers pass by parity as in the kernels (a barrier that runs two
phases ahead of a waiter is a lost wake-up), commits complete in issue order."""
import random

import pytest

from tests.test_pipeline_protocol import Barrier


def run(roles, pipe, rng, limit=200_000):
    """Advances the roles (generators that yield what they wait for) and the
    pipe of issued MMAs in random order; returns whether all of them ended."""
    state = {}
    for name, g in roles.items():
        state[name] = (g, next(g, None))
    for _ in range(limit):
        ready = [n for n, (g, w) in state.items() if w is not None and w[0].passed(w[1])]
        if pipe:
            ready.append(None)
        if not ready:
            break
        pick = rng.choice(ready)
        if pick is None:
            pipe.pop(0)()
        else:
            g, _w = state[pick]
            state[pick] = (g, next(g, None))
    return all(w is None for _, w in state.values()) and not pipe


def simulate_pair(tiles, kblocks, rng, stages=5, warps=8, arrivals=None):
    full = [Barrier(f"full{s}", 2) for s in range(stages)]
    empty = [[Barrier(f"empty{r}{s}") for s in range(stages)] for r in range(2)]
    tfull = [Barrier(f"tfull{r}") for r in range(2)]
    tempty = Barrier("tempty", 2 * warps if arrivals is None else arrivals)
    pipe, reading = [], [0] * stages  # MMAs in flight per stage
    held = {"tile": -1, "left": 0}    # the tile in the accumulator, warps that have to read it

    def producer(r):
        n = 0
        for _ in range(tiles * kblocks):
            s, ph = n % stages, n // stages & 1
            yield empty[r][s], ph ^ 1
            assert reading[s] == 0, "a stage is overwritten under its MMAs"
            full[s].arrive()
            n += 1

    def issuer():
        n = 0
        for t in range(tiles):
            yield tempty, 1 ^ (t & 1)
            assert held["left"] == 0, "an accumulator is overwritten before it was read"
            for kb in range(kblocks):
                s, ph = n % stages, n // stages & 1
                yield full[s], ph
                reading[s] += 1

                def done(s=s):
                    reading[s] -= 1
                    for r in range(2):
                        empty[r][s].arrive()

                pipe.append(done)
                n += 1

            def whole(t=t):
                held.update(tile=t, left=2 * warps)
                for b in tfull:
                    b.arrive()

            pipe.append(whole)

    def epilogue(r):
        for t in range(tiles):
            yield tfull[r], t & 1
            assert held["tile"] == t, "a wait passed for another tile"
            held["left"] -= 1
            tempty.arrive()

    roles = {f"p{r}": producer(r) for r in range(2)}
    roles["mma"] = issuer()
    roles.update({f"e{r}{w}": epilogue(r) for r in range(2) for w in range(warps)})
    return run(roles, pipe, rng)


def simulate_split(kblocks, rng, stages):
    full = [Barrier(f"full{s}") for s in range(stages)]
    empty = [Barrier(f"empty{s}") for s in range(stages)]
    tfull = Barrier("tfull")
    pipe, reading = [], [0] * stages

    def producer():
        for n in range(kblocks):
            yield empty[n % stages], (n // stages & 1) ^ 1
            assert reading[n % stages] == 0
            full[n % stages].arrive()
        for n in range(max(0, kblocks - stages), kblocks):  # the loads have landed
            yield full[n % stages], n // stages & 1

    def issuer():
        for n in range(kblocks):
            s = n % stages
            yield full[s], n // stages & 1
            reading[s] += 1

            def done(s=s):
                reading[s] -= 1
                empty[s].arrive()

            pipe.append(done)
        pipe.append(tfull.arrive)
        yield tfull, 0

    def epilogue():
        yield tfull, 0
        assert not any(reading)

    return run({"p": producer(), "m": issuer(), "e0": epilogue(), "e1": epilogue()}, pipe, rng)


@pytest.mark.parametrize("tiles,kblocks", [(1, 1), (2, 1), (7, 1), (1, 9), (3, 4), (4, 5), (5, 6), (3, 21)])
@pytest.mark.parametrize("stages,warps", [(5, 8), (4, 16)], ids=["long", "short"])
def test_pair_runs_to_the_end(tiles, kblocks, stages, warps):
    for seed in range(30):
        assert simulate_pair(tiles, kblocks, random.Random(seed), stages, warps)


@pytest.mark.parametrize("kblocks", [1, 2, 3, 4, 5, 9, 16])
@pytest.mark.parametrize("stages", [3, 4])
def test_split_runs_to_the_end(kblocks, stages):
    for seed in range(40):
        assert simulate_split(kblocks, random.Random(seed), stages)


def test_the_model_sees_mistakes():
    """A drain barrier that counts too few warps lets the next tile's MMAs in, one
    that counts too many stops them."""
    with pytest.raises(AssertionError):
        for seed in range(40):
            simulate_pair(4, 2, random.Random(seed), arrivals=8)
    assert not any(simulate_pair(4, 2, random.Random(seed), arrivals=17) for seed in range(5))
