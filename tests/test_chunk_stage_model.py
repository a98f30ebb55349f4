"""The chunk kernel's two stage warps for bf16 pages, in the model of its pipeline
(test_chunk_pipeline_model.py): the first waits for every copy and hands K on,
the second meets it for each V operand and hands that on, some time later.
Mutants: a second warp that waits for copies itself, for its own alone or for
all, can find a slot's barrier two phases on, which its parity does not tell."""
import os
import re

import pytest

from test_chunk_pipeline_model import SLOTS, SOURCE, Barrier, Pair, Wrong, sequences


class StagePair(Pair):
    def __init__(self, tiles, seed, **kw):
        super().__init__(tiles, False, seed, **kw)
        self.ready = [Barrier(f"ready {i}", 2) for i in range(SLOTS)]
        self.q_ready = Barrier("q ready", 2)
        self.stage = 2                       # roles of a CTA that hand operands on
        self.met = [[0, 0], [0, 0]]          # [CTA][warp]: V operands that each has come to

    def meet(self, cta, w):
        """A named barrier of the two warps (it has no limit: both come as often)."""
        self.met[cta][w] += 1
        n = self.met[cta][w]
        yield lambda: self.met[cta][1 - w] >= n

    def stage_bf16(self, role, cta, w):
        number = 0
        for s, L in enumerate(self.tiles):
            if w == 0:
                yield from self.wait(role, self.q_full[cta], s & 1)
                self.q_ready.arrive()
            kinds = [kind for i in range(L + 1) for kind in ("K", "V") if (i < L if kind == "K" else i > 0)]
            for kind in kinds:
                st = number % SLOTS
                mine = (kind == "V") == (w == 1)
                if self.mutant == "wait for own" and mine or self.mutant == "wait for all":
                    yield from self.wait(role, self.full[cta][st], number // SLOTS & 1)
                elif self.mutant not in ("wait for own", "wait for all"):
                    if w == 0:
                        yield from self.wait(role, self.full[cta][st], number // SLOTS & 1)
                    if kind == "V":
                        yield from self.meet(cta, w)
                yield None
                if mine:
                    yield None
                    if not self.gave_up and (self.slot[cta][st][0] is None or self.number[self.slot[cta][st][0]] != number):
                        raise Wrong(f"operand {number} handed on before it has landed")
                    self.ready[st].arrive()
                number += 1


def test_the_model_follows_the_source():
    text = " ".join(re.sub(r"//.*", "", open(SOURCE).read()).split())
    for rule in ("} else if (!kFp8 && warp == kStageWarp) {", "if (SCORED && kind == 1) { v_landed(); } else {",
                 "} else if (SCORED && !kFp8 && warp == kStageWarp + 1) {", "pos.step(w.L > 1 ? 2 : 1);", "pos.step(k + 2 < w.L ? 2 : 1);",
                 'asm volatile("bar.sync 6, 64;" ::: "memory");'):
        assert rule in text, rule


def test_every_interleaving_tried_holds():
    for i, tiles in enumerate(sequences(11, 250)):
        for seed in range(4):
            StagePair(tiles, 1000 * i + seed).run()


def test_pairs_whose_waits_run_out_leave_nothing_under_way():
    for i, tiles in enumerate(sequences(12, 200)):
        StagePair(tiles, i, lost=i % (2 * sum(tiles))).run()
        for seed in range(3):
            StagePair(tiles, 1000 * i + seed, impatient=True).run()


@pytest.mark.parametrize("mutant", ["wait for own", "wait for all"])
def test_a_second_warp_that_waits_for_copies_fails(mutant):
    with pytest.raises(Wrong):
        for i, tiles in enumerate(sequences(13, 400)):
            for seed in range(6):
                StagePair(tiles, 1000 * i + seed, mutant=mutant).run()
