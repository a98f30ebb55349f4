"""A model of the chunk kernel's pipeline (paged_chunk.cu) on the CPU: two CTAs,
all roles, their mbarriers with the one bit of parity that a wait sees, copies
that land and matrix products that complete at any time, in random
interleavings.  It checks that

  * a product reads the operands it is meant to, in both CTAs, and nobody
    overwrites a slot, the query rows, a score buffer or the output in use;
  * no barrier is armed while its copy is still on the way (a fault on a GPU);
  * the pair always comes to its end;
  * when waits run out, a CTA leaves only after its copies have landed and the
    pair's products are complete.

The rules in the model are the kernel's, statement for statement; the test of
the source names those that the model rests on, so that a change there asks for
one here.  Mutants -- the rule of an earlier kernel, whose waits named phases
that their barrier could have left behind, and others -- have to fail."""
import os
import random
import re

import pytest

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "full_gqa_decode_gb300", "csrc",
                      "paged_chunk.cu")
SLOTS, BLOCK_PHASES = 5, 4


def test_the_model_follows_the_source():
    text = " ".join(re.sub(r"//.*", "", open(SOURCE).read()).split())
    for rule in (
        f"constexpr int kSlots = {SLOTS};",
        # barriers and their counts
        "mbar_init(&bar[BAR_FULL + i], 1);", "mbar_init(&bar[BAR_READY + i], 2 * kStage);",
        "mbar_init(&bar[BAR_EMPTY + i], 1);", "mbar_init(&bar[BAR_Q_READY], 2 * kStage);", "mbar_init(&bar[BAR_Q_EMPTY], 1);",
        f"for (int i = 0; i < {BLOCK_PHASES}; ++i) mbar_init(&bar[BAR_BLOCK + i], 1);",
        "mbar_init(&bar[BAR_P + i], 2 * kSoftWarps);", "mbar_init(&bar[BAR_O_FREE], 2 * kSoftWarps);",
        # waits
        f"wait_warp(&bar[BAR_BLOCK + (i & {BLOCK_PHASES - 1})], (uint32_t)(i >> 2) & 1,",
        "const int r = blocks + (kind == 0 ? i : i + 1);",
        "const int before = max(__shfl_sync(0xffffffffu, last_read, pos.st), r - 4);", "if (before >= 0) wait_block(before);",
        "if (i == 2 && seg) wait_thread(&bar[BAR_O_FREE], (seg - 1) & 1,",
        "if (i == 0) wait_thread(&bar[BAR_Q_READY], seg & 1,",
        "if (!pos.first) wait_warp(&bar[BAR_EMPTY + pos.st], pos.ph ^ 1,",
        "wait_block(blocks + k);", "wait_block(blocks + k + 1);", "wait_warp(&bar[BAR_O_FULL], seg & 1,",
        # commits
        "pair_commit(&bar[BAR_BLOCK + ((blocks + i) & 3)]);", "if (i == w.L - 1) pair_commit(&bar[BAR_Q_EMPTY]);",
        "if (i == w.L + 1) pair_commit(&bar[BAR_O_FULL]);", "blocks += w.L + 2;",
        # the E4M3 stage warps' way through the ring
        "(k + 1 < L ? (k ? 2 : 1) : (k ? 3 : 2));", "(L > 1 ? 2 : 1);", "(k + 2 < L ? 2 : 1);",
        # once a wait has run out: no barrier armed unseen, no way out before copies and products are through
        "dead = __any_sync(0xffffffffu, dead || !mbar_try_wait(&bar[BAR_Q_FULL], (seg - 1) & 1));",
        "if (!pos.first) dead = __any_sync(0xffffffffu, dead || !mbar_try_wait(full, pos.ph ^ 1));",
        "mbar_wait(&bar[BAR_FULL + lane], (uint32_t)((copied - 1 - lane) / kSlots) & 1);",
        "mbar_wait(&bar[BAR_Q_FULL], (q_copied - 1) & 1);", "pair_commit(&bar[BAR_DRAIN]);", "mbar_wait(&bar[BAR_DRAIN], 0)",
    ):
        assert " ".join(rule.split()) in text, rule


class Wrong(Exception):
    pass


class Barrier:
    """A phase ends after `count` arrivals; a wait sees the parity of the current phase alone."""

    def __init__(self, name, count):
        self.name, self.count, self.left, self.phase = name, count, count, 0

    def arrive(self):
        self.left -= 1
        if self.left == 0:
            self.phase, self.left = self.phase + 1, self.count

    def over(self, parity):
        return self.phase & 1 != parity


class CopyBarrier:
    """Armed once per phase; the phase ends when the copy lands."""

    def __init__(self, name):
        self.name, self.phase, self.armed = name, 0, False

    def arm(self):
        if self.armed:
            raise Wrong(f"{self.name} armed while its copy is on the way")
        self.armed = True

    def land(self):
        self.armed, self.phase = False, self.phase + 1

    def over(self, parity):
        return self.phase & 1 != parity


class Pair:
    """One run over segments of the given numbers of key tiles.  soft, stage: softmax warps and stage warps of a CTA (the
    kernel has 8 and 1 or 4; two show the same).  lost: the operand from which no copy is issued.  impatient: waits
    may run out although what they wait for is on its way.  mutant: a rule to break."""

    def __init__(self, tiles, e4m3, seed, soft=2, lost=None, impatient=False, mutant=None):
        self.rnd = random.Random(seed)
        self.tiles, self.e4m3, self.lost, self.impatient, self.mutant = tiles, e4m3, lost, impatient, mutant
        self.stage = 2 if e4m3 else 1
        self.soft = soft
        two = range(2)
        self.full = [[CopyBarrier(f"full {i} of {c}") for i in range(SLOTS)] for c in two]
        self.q_full = [CopyBarrier(f"q full of {c}") for c in two]
        self.ready = [Barrier(f"ready {i}", 2 * self.stage) for i in range(SLOTS)]
        self.q_ready = Barrier("q ready", 2 * self.stage)
        self.p = [Barrier(f"p {i}", 2 * soft) for i in range(2)]
        self.o_free = Barrier("o free", 2 * soft)
        own = lambda name: [Barrier(f"{name} of {c}", 1) for c in two]
        self.empty = [own(f"empty {i}") for i in range(SLOTS)]
        self.block = [own(f"block {i}") for i in range(BLOCK_PHASES)]
        self.q_empty, self.o_full, self.drain = own("q empty"), own("o full"), own("drain")
        pieces = self.stage if e4m3 else 1
        self.slot = [[[None] * pieces for _ in range(SLOTS)] for _ in two]   # operand whose piece each holds
        self.read = set()                                                   # operands that their product has read
        self.rows = [None, None]                                            # segment of the query rows
        self.softmaxed = {}                                                 # tile -> softmax warps done with its scores
        self.drained = {}                                                   # segment -> softmax warps done with its output
        self.in_output = []                                                 # tiles of the segment that O holds
        self.copies, self.products = [], []                                 # under way
        self.gave_up = False
        self.number = {}
        for s, L in enumerate(tiles):
            for i in range(L + 1):
                for op in ([("K", s, i)] if i < L else []) + ([("V", s, i - 1)] if i else []):
                    self.number[op] = len(self.number)

    # ---- asynchronous work ----
    def land(self):
        barrier, cta, st, op = self.copies.pop(self.rnd.randrange(len(self.copies)))
        if st is None:
            self.rows[cta] = op
        else:
            held = self.slot[cta][st][0]
            if not self.gave_up and held is not None and held not in self.read:
                raise Wrong(f"a copy of {op} overwrites {held}, not yet read")
            self.slot[cta][st][0] = op
        barrier.land()

    def complete(self):
        """The oldest product or commit; a commit arrives in each CTA at its own time."""
        what, *x = self.products[0]
        if what == "commit":
            x[0].pop(self.rnd.randrange(len(x[0]))).arrive()
            if x[0]:
                return
        elif what == "S" and not self.gave_up:
            st, op, tile = x
            for c in range(2):
                if any(h != op for h in self.slot[c][st]) or self.rows[c] != op[1]:
                    raise Wrong(f"S of {op} reads {self.slot[c][st]} and rows of segment {self.rows[c]}")
            if tile >= 2 and self.softmaxed.get(tile - 2, 0) != 2 * self.soft:
                raise Wrong(f"S of tile {tile} overwrites the weights of {tile - 2}")
            self.read.add(op)
        elif what == "O" and not self.gave_up:
            st, op, tile = x
            for c in range(2):
                if any(h != op for h in self.slot[c][st]):
                    raise Wrong(f"O of {op} reads {self.slot[c][st]}")
            if self.softmaxed.get(tile, 0) != 2 * self.soft:
                raise Wrong(f"O of tile {tile} without its weights")
            if op[2] == 0:
                if op[1] and self.drained.get(op[1] - 1, 0) != 2 * self.soft:
                    raise Wrong(f"O of segment {op[1]} over the one before")
                self.in_output = []
            self.in_output.append(op[2])
            self.read.add(op)
        self.products.pop(0)

    # ---- waits ----
    def wait(self, role, barrier, parity):
        """A wait with a limit, which `role` does not make any more once one ran out."""
        if role.dead or barrier.over(parity):
            return
        yield lambda: barrier.over(parity) or role.timed_out
        if not barrier.over(parity):
            role.dead = True

    def wait_block(self, role, cta, i):
        yield from self.wait(role, self.block[i % BLOCK_PHASES][cta], (i // BLOCK_PHASES) & 1)

    # ---- roles ----
    def copy(self, role, cta):
        number = blocks = copied = rows_copied = 0
        last_read = [-1] * SLOTS
        for s, L in enumerate(self.tiles):
            if s:
                if self.mutant != "rows early":
                    yield from self.wait(role, self.q_empty[cta], (s - 1) & 1)
                if self.mutant != "arm unseen" and not self.q_full[cta].over((s - 1) & 1):
                    role.dead = True
            if not role.dead:
                rows_copied += 1
                self.q_full[cta].arm()
                self.copies.append((self.q_full[cta], cta, None, s))
            for i in range(0 if self.e4m3 else L + 1):
                for kind in ("K", "V"):
                    if (i >= L) if kind == "K" else (i == 0):
                        continue
                    op, st = (kind, s, i if kind == "K" else i - 1), number % SLOTS
                    r = blocks + (i if kind == "K" else i + 1)
                    before = max(last_read[st], r - 4)
                    if self.mutant == "last block only":
                        before = last_read[st]
                    if before >= 0:
                        yield from self.wait_block(role, cta, before)
                    last_read[st] = r
                    if self.mutant != "arm unseen" and number >= SLOTS and not self.full[cta][st].over((number // SLOTS & 1) ^ 1):
                        role.dead = True
                    if not (role.dead or (self.lost is not None and number >= self.lost)):
                        copied += 1
                        self.full[cta][st].arm()
                        yield None
                        self.copies.append((self.full[cta][st], cta, st, op))
                    number += 1
                    yield None
            blocks += L + 2
        if self.mutant != "leave at once":
            for st in range(min(SLOTS, copied)):
                last = (copied - 1 - st) // SLOTS
                yield lambda: self.full[cta][st].over(last & 1)
            if rows_copied:
                yield lambda: self.q_full[cta].over((rows_copied - 1) & 1)

    def stage_bf16(self, role, cta, _):
        number = 0
        for s, L in enumerate(self.tiles):
            yield from self.wait(role, self.q_full[cta], s & 1)
            self.q_ready.arrive()
            for _ in range(2 * L):
                st = number % SLOTS
                yield from self.wait(role, self.full[cta][st], number // SLOTS & 1)
                yield None
                self.ready[st].arrive()
                number += 1

    def put(self, cta, w, st, op):
        held = self.slot[cta][st][w]
        if not self.gave_up and held is not None and held not in self.read:
            raise Wrong(f"{op} overwrites {held}, not yet read")
        self.slot[cta][st][w] = op

    def stage_e4m3(self, role, cta, w, kind):
        number = 0
        for s, L in enumerate(self.tiles):
            if kind == "K":
                yield from self.wait(role, self.q_full[cta], s & 1)
                self.q_ready.arrive()
            else:
                number += 2 if L > 1 else 1
            for k in range(L):
                op, st = (kind, s, k), number % SLOTS
                if number != self.number[op]:
                    raise Wrong(f"{op} is operand {self.number[op]}, stored as {number}")
                if number >= SLOTS and self.mutant != "slot early":
                    yield from self.wait(role, self.empty[st][cta], (number // SLOTS & 1) ^ 1)
                self.put(cta, w, st, op)
                yield None
                if self.lost is None or number < self.lost:
                    self.ready[st].arrive()
                if kind == "K":
                    number += (2 if k else 1) if k + 1 < L else (3 if k else 2)
                else:
                    number += 2 if k + 2 < L else 1
                if self.mutant == "ring step" and kind == "V" and L == 2 and k == 0:
                    number += 1

    def commit(self, barriers):
        self.products.append(("commit", list(barriers)))

    def mma(self, role):
        number = blocks = tiles = 0
        for s, L in enumerate(self.tiles):
            for i in range(L + 2):
                if i >= 2:
                    g, st = tiles + i - 2, number % SLOTS
                    if i == 2 and s:
                        yield from self.wait(role, self.o_free, (s - 1) & 1)
                    yield from self.wait(role, self.ready[st], number // SLOTS & 1)
                    if self.mutant != "weights early":
                        yield from self.wait(role, self.p[g & 1], g >> 1 & 1)
                    if not role.dead:
                        self.products.append(("O", st, ("V", s, i - 2), g))
                    if self.e4m3:
                        self.commit(self.empty[st])
                    number += 1
                    yield None
                if i < L:
                    if i == 0:
                        yield from self.wait(role, self.q_ready, s & 1)
                    st = number % SLOTS
                    yield from self.wait(role, self.ready[st], number // SLOTS & 1)
                    if not role.dead:
                        self.products.append(("S", st, ("K", s, i), tiles + i))
                    if self.e4m3:
                        self.commit(self.empty[st])
                    number += 1
                    yield None
                self.commit(self.block[(blocks + i) % BLOCK_PHASES])
                if i == L - 1:
                    self.commit(self.q_empty)
                if i == L + 1:
                    self.commit(self.o_full)
            blocks += L + 2
            tiles += L
        self.commit(self.drain)

    def softmax(self, role, cta, _):
        blocks = tiles = 0
        for s, L in enumerate(self.tiles):
            for k in range(L):
                yield from self.wait_block(role, cta, blocks + k)
                if k and self.rnd.random() < 0.3:
                    yield from self.wait_block(role, cta, blocks + k + 1)
                    if not self.gave_up and self.in_output != list(range(k)):
                        raise Wrong(f"O is rescaled for tile {k} while it holds {self.in_output}")
                yield None
                self.softmaxed[tiles + k] = self.softmaxed.get(tiles + k, 0) + 1
                self.p[(tiles + k) & 1].arrive()
            yield from self.wait(role, self.o_full[cta], s & 1)
            if not self.gave_up and self.in_output != list(range(L)):
                raise Wrong(f"segment {s} of {L} tiles drained while O holds {self.in_output}")
            yield None
            self.drained[s] = self.drained.get(s, 0) + 1
            self.o_free.arrive()
            blocks += L + 2
            tiles += L

    def run(self):
        class Role:
            def __init__(self, name):
                self.name, self.dead, self.timed_out = name, False, False

        live = []

        def add(name, f, *args):
            role = Role(name)
            live.append([role, f(role, *args), None])

        add("mma", self.mma)
        for c in range(2):
            add(f"copy {c}", self.copy, c)
            for w in range(self.stage):
                if self.e4m3:
                    add(f"K {c}.{w}", self.stage_e4m3, c, w, "K")
                    add(f"V {c}.{w}", self.stage_e4m3, c, w, "V")
                else:
                    add(f"stage {c}", self.stage_bf16, c, w)
            for w in range(self.soft):
                add(f"softmax {c}.{w}", self.softmax, c, w)
        pace = {id(x): self.rnd.choice((0.02, 0.1, 1, 1, 3)) for x in live}
        hasty = self.rnd.choice((0.05, 0.3, 0.6))
        while live:
            ready = [x for x in live if x[2] is None or x[2]()]
            work = [f for f, n in ((self.land, self.copies), (self.complete, self.products)) if n]
            slow = not ready and not work
            if slow or (self.impatient and self.rnd.random() < 0.01):   # some wait runs out
                if self.lost is None and not self.impatient:
                    raise Wrong("stuck: " + ", ".join(x[0].name for x in live))
                waiting = [x for x in live if x[2] is not None and not x[2]()]
                if waiting:
                    self.rnd.choice(waiting)[0].timed_out = self.gave_up = True
                elif slow:
                    raise Wrong("stuck after a wait ran out")
                continue
            if work and (not ready or self.rnd.random() < hasty):
                self.rnd.choice(work)()
                continue
            x = self.rnd.choices(ready, [pace[id(x)] for x in ready])[0]
            try:
                x[2] = next(x[1])
            except StopIteration:
                live.remove(x)
        # Every thread of the pair is through; the CTAs leave once the last commit has reached them.
        if self.mutant != "leave at once":
            while self.products and not all(d.over(0) for d in self.drain):
                self.complete()
        if self.copies:
            raise Wrong("a CTA leaves while copies into it are under way")
        if any(x[0] != "commit" for x in self.products):
            raise Wrong("a CTA leaves while products read from it")
        if not self.gave_up and len(self.read) != len(self.number):
            raise Wrong("operands that no product read")


def sequences(seed, n):
    rnd = random.Random(seed)
    yield from ([1], [2], [3], [1, 1, 1], [2, 1, 2, 1], [3, 3], [20], [1, 17, 1], [2, 2, 2, 2], [9, 1, 1, 8])
    for _ in range(n):
        yield [rnd.choice((1, 1, 1, 2, 2, 3, 4, 5, 11)) for _ in range(rnd.choice((1, 2, 3, 4, 6)))]


@pytest.mark.parametrize("e4m3", [False, True])
def test_every_interleaving_tried_holds(e4m3):
    for i, tiles in enumerate(sequences(1, 250)):
        for seed in range(4):
            Pair(tiles, e4m3, 1000 * i + seed).run()


@pytest.mark.parametrize("e4m3", [False, True])
def test_pairs_whose_waits_run_out_leave_nothing_under_way(e4m3):
    for i, tiles in enumerate(sequences(2, 200)):
        Pair(tiles, e4m3, i, lost=i % (2 * sum(tiles))).run()
        for seed in range(3):
            Pair(tiles, e4m3, 1000 * i + seed, impatient=True).run()


@pytest.mark.parametrize("mutant,e4m3", [("last block only", False), ("rows early", False), ("rows early", True),
                                         ("weights early", False), ("weights early", True), ("slot early", True),
                                         ("ring step", True)])
def test_mutants_fail(mutant, e4m3):
    with pytest.raises(Wrong):
        for i, tiles in enumerate(sequences(3, 300)):
            for seed in range(4):
                Pair(tiles, e4m3, 1000 * i + seed, mutant=mutant).run()


@pytest.mark.parametrize("mutant,e4m3", [("leave at once", False), ("leave at once", True), ("arm unseen", False)])
def test_mutants_fail_once_waits_run_out(mutant, e4m3):
    with pytest.raises(Wrong):
        for i, tiles in enumerate(sequences(3, 300)):
            for seed in range(4):
                Pair(tiles, e4m3, 1000 * i + seed, impatient=True, mutant=mutant).run()
