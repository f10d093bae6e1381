"""The hand-overs of the linear-attention prefill kernel, as a model on the CPU.

A wait names a barrier's phase by its parity, so it must not begin before the
phase ahead of its own is over (it would take that one's end for its own), and
must be looked at before the barrier has passed one phase more (it would never
see its phase and run into its time limit).  The model has the kernel's groups of
warps, its tiled copies and its products as actors that wait for and complete
the same barriers, and lets them run in random orders, each actor in turn held
back for as long as the others can go on.  In no order may a wait be early or overrun,
and every order has to come to its end.  How many barriers the partial chunks
and the staged outputs have is read from the kernel's source."""
import os
import random
import re

import pytest

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "selective_state_update_gb300", "csrc",
                      "ssu_linattn_prefill.cu")
CHUNK, QUARTER = 128, 32


def barriers(name):
    """How many barriers of this name the kernel has: one, or one for each of its two stages."""
    with open(SOURCE) as f:
        enum = re.search(r"enum : int \{(.*?)kBars", f.read(), re.S).group(1)
    found = set(re.findall(rf"\b(k{name}\d?)\b", re.sub(r"//.*", "", enum)))
    assert found in ({f"k{name}"}, {f"k{name}0", f"k{name}1"})
    return len(found)


class Overrun(Exception):
    pass


class Model:
    """One CTA that works on `units` (their lengths in tokens).  An actor yields (barrier, phase) to wait, None otherwise."""

    def __init__(self, units, grow, tails=2, staged=2):
        self.units, self.grow, self.tails, self.staged = [*units, -1], grow, tails, staged
        self.need, self.left, self.done = {}, {}, {}
        self.ring, self.products, self.copies = [None, None], [], []
        helpers = 2 if grow else 1
        for s in (0, 1):
            for name, count in (("QFull", 1), ("QFree", 1), ("Full", 1), ("Free", 1 + helpers), ("UnitFull", 1),
                                ("UnitFree", 4 if grow else 5), ("VFull", 1), ("VFree", 1), ("Tail", 1), ("Staged", 1),
                                ("Growth", 1), ("GrowthFree", 1)):
                self.barrier(f"{name}{s}", count)
        for name in ("Score", "State", "Enter", "P", "Inside", "OutFree"):
            self.barrier(name, 1)
        self.actors = {"loads": self.loads(), "products": self.issue(), "state": self.state(), "values": self.values(0)}
        if grow:
            self.actors["values 1"] = self.values(1)
        else:
            self.actors["rows"] = self.rows()
            self.actors["stores"] = self.stores()

    def barrier(self, name, count):
        self.need[name], self.left[name], self.done[name] = count, count, 0

    def arrive(self, name):
        self.left[name] -= 1
        assert self.left[name] >= 0, name
        if self.left[name] == 0:
            self.left[name], self.done[name] = self.need[name], self.done[name] + 1

    def loads(self):
        n = ch = 0

        def publish(length):
            nonlocal n
            if n >= 2:
                yield f"UnitFree{n & 1}", (n >> 1) - 1
            self.ring[n & 1] = length
            self.arrive(f"UnitFull{n & 1}")
            n += 1

        coming = iter(self.units)
        unit = next(coming)
        yield from publish(unit)
        while unit >= 0:
            after = next(coming)
            yield from publish(after)
            for _ in range(0, unit, CHUNK):
                s = ch & 1
                if ch >= 2:
                    yield f"Free{s}", (ch >> 1) - 1
                self.copies.append(f"Full{s}")
                yield
                if not self.grow:
                    if ch >= 2:
                        yield f"QFree{s}", (ch >> 1) - 1
                    self.copies.append(f"QFull{s}")
                    yield
                ch += 1
            unit = after

    def each_chunk(self, chunk, ends=None):
        n = ch = 0
        while True:
            yield f"UnitFull{n & 1}", n >> 1
            unit = self.ring[n & 1]
            self.arrive(f"UnitFree{n & 1}")
            n += 1
            yield
            if unit < 0:
                return
            if ends:
                yield from ends(ch)
            for c in range(0, unit, CHUNK):
                yield from chunk(ch, min(CHUNK, unit - c))
                ch += 1
            if ends:
                yield from ends(ch)

    def values(self, helper):
        quarters = 0

        def chunk(ch, n):
            nonlocal quarters
            s = ch & 1
            yield f"Full{s}", ch >> 1
            if n < CHUNK:
                self.arrive(f"Tail{s if self.tails == 2 else 0}")
                yield
            for quarter in range(0, n, QUARTER):
                if not self.grow or (quarter // QUARTER & 1) == helper:
                    if quarters >= 2:
                        yield f"VFree{quarters & 1}", (quarters >> 1) - 1
                    self.arrive(f"VFull{quarters & 1}")
                    yield
                quarters += 1
            self.arrive(f"Free{s}")
            yield

        yield from self.each_chunk(chunk)

    def issue(self):
        quarters, tails = 0, [0, 0]

        def growth(ch, n, quarter):
            nonlocal quarters
            if quarter * QUARTER >= n:
                return
            s, own = ch & 1, ch & 1 if self.grow else 0
            if quarter == 0:
                yield f"Full{s}", ch >> 1
                if n < CHUNK:
                    t = s if self.tails == 2 else 0
                    yield f"Tail{t}", tails[t]
                    tails[t] += 1
                if ch > (1 if self.grow else 0):
                    yield f"GrowthFree{own}", (ch >> 1 if self.grow else ch) - 1
            yield f"VFull{quarters & 1}", quarters >> 1
            self.products.append(f"VFree{quarters & 1}")
            quarters += 1
            if (quarter + 1) * QUARTER >= n:
                self.products.append(f"Growth{own}")
                if self.grow:
                    self.products.append(f"Free{s}")
            yield

        def chunk(ch, n):
            s = ch & 1
            yield from growth(ch, n, 0)
            if not self.grow:
                yield f"QFull{s}", ch >> 1
                if ch:
                    yield "Inside", ch - 1
                self.products.append("Score")
                yield
                yield from growth(ch, n, 1)
                yield "State", ch
                if ch:
                    yield "OutFree", ch - 1
                self.products.append("Enter")
                yield
            else:
                yield from growth(ch, n, 1)
            yield from growth(ch, n, 2)
            yield from growth(ch, n, 3)
            if not self.grow:
                yield "P", ch
                self.products += ["Inside", f"Free{s}"]
                yield

        yield from self.each_chunk(chunk)

    def rows(self):
        def chunk(ch, n):
            yield "Score", ch
            yield "Enter", ch
            self.arrive("P")
            yield
            yield "Inside", ch
            self.arrive("OutFree")
            yield
            self.arrive(f"Staged{ch & 1 if self.staged == 2 else 0}")
            yield

        yield from self.each_chunk(chunk)

    def stores(self):
        def chunk(ch, n):
            yield (f"Staged{ch & 1}", ch >> 1) if self.staged == 2 else ("Staged0", ch)
            self.arrive(f"QFree{ch & 1}")
            yield

        yield from self.each_chunk(chunk)

    def state(self):
        def place_free(ch):  # a state on its way in or out takes the place of the last entering product's operand
            if ch and not self.grow:
                yield "Enter", ch - 1

        def chunk(ch, n):
            own, phase = (ch & 1, ch >> 1) if self.grow else (0, ch)
            if not self.grow:
                yield from place_free(ch)
                self.arrive("State")
                yield
            yield f"Growth{own}", phase
            self.arrive(f"GrowthFree{own}")
            yield

        yield from self.each_chunk(chunk, place_free)

    def run(self, seed, late, watched):
        """`late` goes on only where nothing else can.  Raises where a wait on a barrier of `watched` is early or overrun; other
        waits are taken as they are meant."""
        rng = random.Random(seed)
        at = {name: next(actor) for name, actor in self.actors.items()}
        engines = {"tensor cores": self.products, "copy engine": self.copies}
        while True:
            for name, where in at.items():
                if where and where[0].rstrip("01") in watched and self.done[where[0]] not in (where[1], where[1] + 1):
                    raise Overrun(f"{name} waits for phase {where[1]} of {where[0]}, which is in phase {self.done[where[0]]}")
            able = [n for n, w in at.items() if w is None or self.done[w[0]] > w[1]] + [n for n, q in engines.items() if q]
            if not able:
                assert not at, f"stuck: {at}"
                return
            name = rng.choice([n for n in able if n != late] or able)
            if name in engines:
                self.arrive(engines[name].pop(0))
                continue
            try:
                at[name] = next(self.actors[name])
            except StopIteration:
                del at[name]


ACTORS = [None, "loads", "products", "state", "values", "rows", "stores", "tensor cores", "copy engine"]
LENGTHS = [[5] * 12, [40] * 8, [128] * 6, [130, 3, 1, 256, 31, 0, 0, 7, 128, 129, 33], [1, 128, 1, 128, 1],
           [64, 5, 70, 20, 300, 9, 9, 9], [0, 1, 0, 1, 0, 1, 2, 3]]
WATCHED = ["Tail", "Staged", "Score", "State", "Enter", "P", "Inside", "OutFree", "QFull", "QFree", "Full", "Free", "UnitFull", "UnitFree",
           "VFull", "VFree", "Growth", "GrowthFree"]


@pytest.mark.parametrize("late", ACTORS)
def test_no_wait_is_overrun(late):
    for lengths in LENGTHS:
        for seed in range(30):
            Model(lengths, False, barriers("Tail"), barriers("Staged")).run(seed, late, WATCHED)


@pytest.mark.parametrize("late", [None, "loads", "products", "state", "values", "values 1", "tensor cores", "copy engine"])
def test_no_wait_is_overrun_in_the_growth_pass(late):
    """Its pieces are whole chunks."""
    for lengths in ([128] * 5, [256, 512, 128], [640]):
        for seed in range(30):
            Model(lengths, True).run(seed, late, WATCHED)


@pytest.mark.parametrize("name,late", [("Tail", "products"), ("Staged", "stores")])
def test_one_barrier_for_both_stages_is_overrun(name, late):
    """The model tells the difference."""
    with pytest.raises(Overrun, match=name):
        Model([5] * 12, False, 1 if name == "Tail" else 2, 1 if name == "Staged" else 2).run(0, late, WATCHED)
