"""A model of the barriers of the two block-sparse gradient kernels, run in random orders (no GPU).

Each warp role is a generator that yields the barrier phase it waits for; the products and their
commits finish in the order issued, the copies in any.  A run shows that no order leaves every role
waiting, that no stage is loaded while a step that reads it is unfinished, and that every step is taken once.
The roles follow the waits and arrivals of csrc/blocksparse_backward.cu; a change there is made here too.
"""

import random

import pytest

WARPS = 3  # softmax warps; the kernels have sixteen, all alike


class Bar:
    """An mbarrier: `count` arrivals end a phase; a wait names a parity and is over if the phase before the
    current one has it (so a barrier that was never used passes a wait for the odd one)."""

    def __init__(self, count=1):
        self.count, self.have, self.phase = count, 0, 0

    def arrive(self):
        self.have += 1
        if self.have == self.count:
            self.have, self.phase = 0, self.phase + 1

    def over(self, parity):
        return (self.phase & 1) != parity


class Ring:
    def __init__(self, n, count=1):
        self.bars = [Bar(count) for _ in range(n)]

    def nth(self, k):
        """The barrier and the parity of its use number k, counted over the ring."""
        return self.bars[k % len(self.bars)], (k // len(self.bars)) & 1


class Machine:
    def __init__(self, rng):
        self.rng, self.queue, self.copies, self.done = rng, [], [], set()

    def load(self, bar, *free):
        """A copy that arrives at `bar`; `free` are the (what, step) whose stage it goes to."""
        self.need(*free)
        self.copies.append(bar)

    def need(self, *ops):
        for op in ops:
            assert op[1] < 0 or op in self.done, f"stage still read by {op}"

    def run(self, roles):
        rng, live, wait = self.rng, dict(roles), dict.fromkeys(roles)
        speed = {k: rng.random() ** 3 + 1e-3 for k in [*roles, "tensor", "copies"]}
        while live:
            can = [k for k in live if wait[k] is None or wait[k][0].over(wait[k][1])]
            can += ["tensor"] * bool(self.queue) + ["copies"] * bool(self.copies)
            if not can:
                return sorted(live)
            k = rng.choices(can, [speed[c] for c in can])[0]
            if rng.random() < 0.01:
                speed[k] = rng.random() ** 3 + 1e-3
            if k == "tensor":
                op = self.queue.pop(0)
                self.done.add(op) if isinstance(op, tuple) else op.arrive()
            elif k == "copies":
                self.copies.pop(rng.randrange(len(self.copies))).arrive()
            else:
                try:
                    wait[k] = next(live[k])
                except StopIteration:
                    del live[k]
        return []


def steps_of(items):
    """(first, last) of each step, all items' in a row."""
    return [(i == 0, i == n - 1) for n in items for i in range(n)]


def dkdv(rng, items, do_stages, row_slots, through_ring=False):
    """`items`: steps of each; 0: no query sees the tile.  `through_ring`: such tiles handed to the softmax
    warps in the ring of rows."""
    m, steps = Machine(rng), steps_of(items)
    n, q_stages, warps = len(steps), 3, range(WARPS)
    k_full, k_empty, v_full, v_empty, s_full, acc_full = (Bar() for _ in range(6))
    p_full, ds_full, acc_empty = (Bar(WARPS) for _ in range(3))
    q_full, do_full, dp_full = Ring(q_stages), Ring(do_stages), Ring(2)
    row_full, row_empty = Ring(row_slots), Ring(row_slots, WARPS)
    rows = {}  # what the ring of rows holds, by use

    def row(r, what):
        bar, parity = row_empty.nth(r)
        yield bar, parity ^ 1
        m.need(*[("row", r - row_slots, w) for w in warps])
        rows[r] = what

    def loader():
        at = r = item = 0
        for size in items:
            if size == 0:
                if through_ring:
                    yield from row(r, "unseen")
                    row_full.nth(r)[0].arrive()
                    r += 1
                continue
            for i in range(size):
                yield from row(r, at)
                m.load(row_full.nth(r)[0])
                r += 1
                if i == 0:
                    yield k_empty, (item & 1) ^ 1
                    m.load(k_full, ("S", at - 1))
                if do_stages == q_stages and at + 1 - do_stages >= 0:
                    yield dp_full.nth(at + 1 - do_stages)
                m.load(q_full.nth(at)[0], ("S", at - q_stages), ("dK", at - q_stages))
                if i == 0:
                    yield v_empty, (item & 1) ^ 1
                    m.load(v_full, ("dP", at - 1))
                if do_stages < q_stages and at >= 2:
                    yield dp_full.nth(at - 1)
                m.load(do_full.nth(at)[0], ("dP", at - do_stages), ("dV", at - do_stages))
                at += 1
            item += 1
        yield from row(r, "end")
        row_full.nth(r)[0].arrive()
        m.need(("S", at - q_stages))
        q_full.nth(at)[0].arrive()

    def issuer():
        items_s = items_dp = 0

        def s(at):
            nonlocal items_s
            yield q_full.nth(at)
            if at == n:
                return
            if steps[at][0]:
                yield k_full, items_s & 1
                items_s += 1
            m.queue += [("S", at), s_full] + [k_empty] * steps[at][1]

        def dp(at):
            nonlocal items_dp
            if steps[at][0]:
                yield v_full, items_dp & 1
                items_dp += 1
            yield do_full.nth(at)
            m.queue += [("dP", at), dp_full.nth(at)[0]] + [v_empty] * steps[at][1]

        yield from s(0)
        if n:
            yield from dp(0)
        item = 0
        for at in range(n):
            yield p_full, at & 1
            if steps[at][0]:
                yield acc_empty, (item & 1) ^ 1
                item += 1
            m.queue.append(("dV", at))
            yield from s(at + 1)
            yield ds_full, at & 1
            m.queue += [("dK", at)] + [acc_full] * steps[at][1]
            if at + 1 < n:
                yield from dp(at + 1)

    def softmax(w):
        at, r, items_done, stores, expect = None, 0, 0, False, 0
        freed = 0
        while True:
            if at is not None:
                yield s_full, at & 1
                m.need(("S", at))
                p_full.arrive()
            if stores:
                yield acc_full, items_done & 1
                items_done += 1
                acc_empty.arrive()
                stores = False
            if at is None and r and rows[r - 1] == "end":
                return
            before = at
            yield row_full.nth(r)
            what = rows[r]
            r += 1
            if before is not None:
                yield dp_full.nth(before)
                m.need(("dP", before))
                ds_full.arrive()
                m.done.add(("row", freed, w))
                row_empty.nth(freed)[0].arrive()
                freed += 1
                stores = steps[before][1]
            if what == "unseen":
                m.done.add(("row", freed, w))
                row_empty.nth(freed)[0].arrive()
                freed += 1
            at = what if isinstance(what, int) else None
            if at is not None:
                assert at == expect
                expect += 1

    return m.run({"loader": loader(), "issuer": issuer(), **{f"softmax {w}": softmax(w) for w in warps}})


def dq(rng, items):
    """`items`: steps of each; 0: a query block without keys."""
    m, steps = Machine(rng), steps_of(items)
    n, slots, k_stages, v_stages = len(steps), 3, 3, 2
    item_full, item_empty = Ring(slots), Ring(slots, 1 + WARPS)
    q_full, q_empty, do_full, do_empty, s_full, dq_full = (Bar() for _ in range(6))
    s_empty, ds_full, dq_empty = (Bar(WARPS) for _ in range(3))
    k_full, v_full, dp_full = Ring(k_stages), Ring(v_stages), Ring(2)
    held = {}

    def loader():
        at = real = 0
        for i, size in enumerate([*items, None]):
            bar, parity = item_empty.nth(i)
            yield bar, parity ^ 1
            held[i] = size
            item_full.nth(i)[0].arrive()
            for t in range(size or 0):
                if t == 0:
                    yield q_empty, (real & 1) ^ 1
                    m.load(q_full)
                if at >= 2:
                    yield dp_full.nth(at - 2)
                m.load(k_full.nth(at)[0], ("S", at - k_stages), ("dQ", at - k_stages))
                if t == 0:
                    yield do_empty, (real & 1) ^ 1
                    m.load(do_full)
                    real += 1
                m.load(v_full.nth(at)[0], ("dP", at - v_stages))
                at += 1

    def issuer():
        slot = left = at_s = at_dp = qs = dos = 0

        def following():
            nonlocal slot, left
            while left == 0:
                yield item_full.nth(slot)
                left = held[slot]
                if left is None:
                    return
                item_empty.nth(slot)[0].arrive()
                slot += 1
            left -= 1

        def s(at):
            nonlocal qs
            if steps[at][0]:
                yield q_full, qs & 1
                qs += 1
            yield k_full.nth(at)
            yield s_empty, (at & 1) ^ 1
            m.queue += [q_empty] * steps[at][0] + [("S", at), s_full]

        def dp(at):
            nonlocal dos
            if steps[at][0]:
                yield do_full, dos & 1
                dos += 1
            yield v_full.nth(at)
            m.queue += [do_empty] * steps[at][0] + [("dP", at), dp_full.nth(at)[0]]

        yield from following()
        if n:
            yield from s(0)
            yield from dp(0)
        item = 0
        for at in range(n):
            yield from following()
            if at + 1 < n:
                yield from s(at + 1)
            yield ds_full, at & 1
            if steps[at][0]:
                yield dq_empty, (item & 1) ^ 1
                item += 1
            m.queue += [("dQ", at)] + [dq_full] * steps[at][1]
            if at + 1 < n:
                yield from dp(at + 1)

    def softmax(w):
        slot = at = items_done = 0
        left, work, stores = 0, False, False
        while True:
            if work:
                yield s_full, at & 1
                m.need(("S", at))
                s_empty.arrive()
            if stores:
                yield dq_full, items_done & 1
                items_done += 1
                dq_empty.arrive()
                stores = False
            if left is None:
                assert at == n
                return
            had = work
            if work:
                left -= 1
                stores = left == 0
            if not work or left == 0:
                while True:
                    yield item_full.nth(slot)
                    left = held[slot]
                    if left is None:
                        break
                    item_empty.nth(slot)[0].arrive()
                    slot += 1
                    if left:
                        break
                work = left is not None
            if had:
                yield dp_full.nth(at)
                m.need(("dP", at))
                ds_full.arrive()
                at += 1

    return m.run({"loader": loader(), "issuer": issuer(), **{f"softmax {w}": softmax(w) for w in range(WARPS)}})


def draw(seed):
    rng = random.Random(seed)
    empty = rng.choice([0, 0.3, 0.8])
    return rng, [0 if rng.random() < empty else rng.choice([1, 1, 2, 3, 5]) for _ in range(rng.randrange(9))]


@pytest.mark.parametrize("do_stages,row_slots", [(2, 2), (3, 4)])  # heads of 128, of 64
def test_dkdv_goes_on_in_every_order(do_stages, row_slots):
    for seed in range(1500):
        rng, items = draw(seed)
        assert dkdv(rng, items, do_stages, row_slots) == [], (seed, items)


def test_dq_goes_on_in_every_order():
    for seed in range(1500):
        rng, items = draw(seed)
        assert dq(rng, items) == [], (seed, items)


def test_the_model_sees_a_ring_of_unseen_tiles_stand_still():
    """Tiles that no query sees, handed on in the ring of rows: three behind an item leave all roles waiting."""
    assert any(dkdv(random.Random(seed), [2, 0, 0, 0, 0, 1], 2, 2, through_ring=True) for seed in range(50))
    assert all(not dkdv(random.Random(seed), [2, 0, 1, 0, 1], 2, 2, through_ring=True) for seed in range(50))
