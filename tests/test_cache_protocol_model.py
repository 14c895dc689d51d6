"""A CPU model of the loading warp of the 4-bit cache's attention for few rows (`cache_attn_small_kernel` in
csrc/cache_attn_small.cu).

Lane w of that warp fills warp w's ring.  The lanes go round one loop together, held by full-mask votes (is anything
left to load, was any stage ready), and leave it when everything is loaded, when another warp has raised the abort
flag, or when no stage was emptied for the longest wait.  The flag and the clock are read by each lane at its own
moment, so the lanes may see different things; a vote completes only when every lane of the warp is at that vote.

The model runs the lanes' steps in random order beside a warp that empties stages for a while and then stops, and one
that may raise the flag.  It checks that the lanes always leave together, that every copy issued was drained first, and
that a way out by time leaves the flag and the status set.  The rule that each lane decides for itself (planted) must be
caught.
"""
import random

import pytest

LANES, STAGES, WAIT = 8, 2, 40


class Deadlock(AssertionError):
    pass


class Warp:
    def __init__(self, seed, rule, flag_at, empties):
        self.rng = random.Random(seed)
        self.rule, self.flag_at, self.empties = rule, flag_at, empties
        self.now, self.abort, self.status = 0, False, None
        self.issued, self.emptied = [0] * LANES, [0] * LANES
        self.units = [self.rng.randint(0, 12) for _ in range(LANES)]
        self.drained = [False] * LANES

    def lane(self, w):
        """The loop's steps in program order; ("vote", site, value) gets whether any lane's value is true."""
        idle, since = False, 0
        while True:
            want = self.issued[w] < self.units[w]
            if not (yield ("vote", "want", want)):
                break
            ready = want and self.issued[w] < self.emptied[w] + STAGES
            yield ("step",)
            if ready:
                self.issued[w] += 1
            if (yield ("vote", "ready", ready)):
                idle = False
                continue
            yield ("step",)
            now = self.now
            if not idle:
                since = now
            idle = True
            yield ("step",)
            give_up = self.abort or now - since > WAIT
            if self.rule == "vote":
                give_up = yield ("vote", "give up", give_up)
            if give_up:
                if w == 0:
                    self.abort, self.status = True, "timeout"
                yield ("step",)
                self.drained[w] = True
                break
        yield ("vote", "end", False)

    def run(self):
        lanes = [self.lane(w) for w in range(LANES)]
        at = [next(x) for x in lanes]  # what each lane waits at; None: it has left
        while any(a is not None for a in at):
            self.now += 1
            if self.flag_at is not None and self.now >= self.flag_at:
                self.abort = True
                self.status = self.status or "timeout"  # by the warp that raised it
            w = self.rng.randrange(LANES)
            if self.now < self.empties and self.emptied[w] < self.issued[w] and self.rng.random() < 0.3:
                self.emptied[w] += 1
            steps = [i for i, a in enumerate(at) if a is not None and a[0] == "step"]
            if steps:
                i = self.rng.choice(steps)
                at[i] = next(lanes[i], None)
                continue
            sites = {a[1] if a is not None else "gone" for a in at}
            if len(sites) > 1:
                raise Deadlock(f"lanes at {sites}")
            value = any(a[2] for a in at)
            for i in range(LANES):
                try:
                    at[i] = lanes[i].send(value)
                except StopIteration:
                    at[i] = None
        if any(i < u for i, u in zip(self.issued, self.units)):
            assert self.status == "timeout" and self.abort and all(self.drained)


CASES = [(None, 30), (None, 10**9), (25, 30), (90, 10**9), (60, 40)]


@pytest.mark.parametrize("flag_at,empties", CASES)
def test_the_lanes_leave_together(flag_at, empties):
    for seed in range(300):
        Warp(seed, "vote", flag_at, empties).run()


def test_lanes_that_decide_alone_are_caught():
    caught = 0
    for flag_at, empties in CASES:
        for seed in range(300):
            try:
                Warp(seed, "alone", flag_at, empties).run()
            except AssertionError:
                caught += 1
    assert caught > 50, caught
