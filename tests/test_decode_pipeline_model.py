"""A model of the decode kernel's ring (paged_decode.cu) on the CPU: the
producer, the teams of consumer warps that take stages in turn, and copies that
land at any time, in random interleavings.  A stage is read as it was copied, no
barrier is armed while its copies are on the way, the CTA always comes to its
end, and when waits run out it leaves only after its copies have landed.  Mutants
have to fail; the rules that the model rests on are looked up in the source."""
import os
import random
import re

import pytest

from test_chunk_pipeline_model import Barrier, CopyBarrier, Wrong

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "full_gqa_decode_gb300", "csrc",
                      "paged_decode.cu")
RING, WARPS = 6, 8


def test_the_model_follows_the_source():
    text = " ".join(re.sub(r"//.*", "", open(SOURCE).read()).split())
    for rule in (
        f"constexpr int kRing = {RING};", "constexpr int kFulls = 2 * kRing;", f"constexpr int kWarps = {WARPS};",
        "mbar_init(&full[i], 1);", "mbar_init(&empty[i], team_warps(KV));",
        "if (!dead) dead = !__all_sync(0xffffffffu, mbar_wait(&empty[st], ph ^ 1));",
        "if (!dead && issued >= kFulls) dead = !__all_sync(0xffffffffu, mbar_try_wait(&full[st + odd], (uint32_t)(issued / kFulls - 1) & 1));",
        "if (!dead && !__all_sync(0xffffffffu, mbar_wait(&full[fb], ph))) {", "int fb = team;", "fb += kTeams;",
        "mbar_wait(&full[lane], (uint32_t)((copied - 1 - lane) / kFulls) & 1)",
    ):
        assert " ".join(rule.split()) in text, rule


def run(stages, team_warps, seed, lost=None, impatient=False, mutant=None):
    rnd = random.Random(seed)
    fulls = RING if mutant == "one round" else 2 * RING
    full = [CopyBarrier(f"full {i}") for i in range(fulls)]
    empty = [Barrier(f"empty {i}", team_warps) for i in range(RING)]
    slot, copies, readers = [None] * RING, [], [0] * RING
    teams, state = WARPS // team_warps, dict(late=False)

    class Role:
        dead = late = False

    def wait(role, barrier, parity):
        if not (role.dead or barrier.over(parity)):
            yield lambda: barrier.over(parity) or role.late
            role.dead = not barrier.over(parity)

    def producer(role):
        copied = 0
        for i in range(stages):
            st, fb = i % RING, i % fulls
            yield from wait(role, empty[st], (i // RING & 1) ^ 1)
            if not role.dead and i >= fulls and mutant != "arm unseen" and not full[fb].over((i // fulls - 1) & 1):
                role.dead = True
            if not (role.dead or (lost is not None and i >= lost)):
                copied += 1
                full[fb].arm()
                yield None
                copies.append((fb, st, i))
            yield None
        if mutant != "leave at once":
            for fb in range(min(fulls, copied)):
                last = (copied - 1 - fb) // fulls
                yield lambda: full[fb].over(last & 1)

    def consumer(role, team):
        for i in range(team, stages, teams):
            st, fb = i % RING, i % fulls
            yield from wait(role, full[fb], i // fulls & 1)
            if not role.dead:
                readers[st] += 1
                yield None
                if slot[st] != i and not state["late"]:
                    raise Wrong(f"stage {i} reads {slot[st]}")
                readers[st] -= 1
            empty[st].arrive()
            yield None

    live = []
    for gen in [producer] + [consumer] * WARPS:
        role = Role()
        live.append([role, gen(role) if gen is producer else gen(role, (len(live) - 1) // team_warps), None])
    pace = {id(x): rnd.choice((0.02, 0.3, 1, 3)) for x in live}
    hasty = rnd.choice((0.01, 0.1, 0.5))
    while live:
        ready = [x for x in live if x[2] is None or x[2]()]
        if not (ready or copies) or (impatient and rnd.random() < 0.02):
            if lost is None and not impatient:
                raise Wrong("stuck")
            waiting = [x for x in live if x[2] is not None and not x[2]()]
            if waiting:
                rnd.choice(waiting)[0].late = state["late"] = True
            elif not (ready or copies):
                raise Wrong("stuck after a wait ran out")
            continue
        if copies and (not ready or rnd.random() < hasty):
            fb, st, i = copies.pop(rnd.randrange(len(copies)))
            if readers[st] and not state["late"]:
                raise Wrong(f"stage {i} lands in a slot that is read")
            slot[st] = i
            full[fb].land()
            continue
        x = rnd.choices(ready, [pace[id(y)] for y in ready])[0]
        try:
            x[2] = next(x[1])
        except StopIteration:
            live.remove(x)
    if copies:
        raise Wrong("the CTA leaves while copies into it are under way")


LENGTHS = (1, 2, 3, 5, 6, 7, 11, 12, 13, 18, 24, 25, 40, 61)


@pytest.mark.parametrize("team_warps", [2, 4])
def test_every_interleaving_tried_holds(team_warps):
    for n in LENGTHS:
        for seed in range(30):
            run(n, team_warps, seed)


@pytest.mark.parametrize("team_warps", [2, 4])
def test_a_cta_whose_waits_run_out_leaves_nothing_under_way(team_warps):
    for n in LENGTHS:
        for seed in range(20):
            run(n, team_warps, seed, lost=seed % n)
            run(n, team_warps, seed, impatient=True)


@pytest.mark.parametrize("mutant,impatient,team_warps", [("one round", False, 2), ("leave at once", True, 2),
                                                         ("leave at once", True, 4), ("arm unseen", True, 2),
                                                         ("arm unseen", True, 4)])   # two teams: one round would do
def test_mutants_fail(mutant, impatient, team_warps):
    with pytest.raises(Wrong):
        for seed in range(300):
            run(61, team_warps, seed, impatient=impatient, mutant=mutant)
