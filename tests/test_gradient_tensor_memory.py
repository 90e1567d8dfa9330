"""A model of what the roles of the block-sparse gradient kernel share, with tensor memory, run in random
orders (no GPU).

Beside the stages in shared memory (tests/test_gradient_barriers.py) it follows S and P, dP and dS, the sums
and the copies of Q and dO in tensor memory: a product may be issued once what it reads is written, by all
softmax warps, and what it overwrites has been read; sums may be read once the last product into them is
done.  At the end no copy and no product is left, as the other half of the kernel takes the same memory.
Products finish in the order issued, copies in any.

Each wait of the kernel has a name here.  With any one of them left out the model has to find a fault,
so that it sees what the waits are for.  And the waits, arrivals and commits of the source, in the order
they stand there, have to be those that the model was written from.
"""

import os
import random
import re

import pytest

from tests.test_gradient_barriers import WARPS, Bar, Ring, steps_of

SOURCE = os.path.join(os.path.dirname(__file__), "..", "selected_block_attention_gb300", "csrc", "blocksparse_backward.cu")


class Fault(Exception):
    pass


class Machine:
    def __init__(self, rng, without):
        self.rng, self.without, self.queue, self.copies, self.done = rng, without, [], [], set()
        self.asked = set()

    def wait(self, name, bar, parity):
        self.asked.add(name)
        if name != self.without:
            yield bar, parity

    def need(self, *events):
        for e in events:
            if e not in self.done:
                raise Fault(e)

    def load(self, bar, event):
        self.copies.append((bar, event))

    def run(self, roles):
        """Names of the roles that wait for ever."""
        rng, live, blocked = self.rng, dict(roles), dict.fromkeys(roles)
        speed = {k: rng.random() ** 3 + 1e-3 for k in [*roles, "tensor", "copies"]}
        while live:
            can = [k for k in live if blocked[k] is None or blocked[k][0].over(blocked[k][1])]
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
                bar, event = self.copies.pop(rng.randrange(len(self.copies)))
                self.done.add(event)
                bar.arrive()
            else:
                try:
                    blocked[k] = next(live[k])
                except StopIteration:
                    del live[k]
        if self.queue or self.copies:
            raise Fault("left behind")
        return []


ALL = range(WARPS)


def ops(name, at):
    """An event of each softmax warp; none for a step or item before the first."""
    return [(name, at, w) for w in ALL] if at >= 0 else []


def once(name, at):
    return [(name, at)] if at >= 0 else []


def dkdv(rng, items, do_stages, row_slots, without=None):
    m, steps, q_stages = Machine(rng, without), steps_of(items), 3
    n, real = len(steps), [size for size in items if size]
    k_full, k_empty, v_full, v_empty, s_full, acc_full, mma_done = (Bar() for _ in range(7))
    p_full, ds_full, acc_empty = (Bar(WARPS) for _ in range(3))
    q_full, do_full, dp_full = Ring(q_stages), Ring(do_stages), Ring(2)
    row_full, row_empty = Ring(row_slots), Ring(row_slots, WARPS)
    rows, flags = {}, {}
    last_of = [sum(real[:i + 1]) - 1 for i in range(len(real))]  # an item's last step

    def loader():
        at = 0
        for item, size in enumerate(real):
            for i in range(size):
                bar, parity = row_empty.nth(at)
                yield from m.wait("loader row_empty", bar, parity ^ 1)
                m.need(*ops("row read", at - row_slots))
                rows[at] = at
                m.load(row_full.nth(at)[0], ("row", at))
                if i == 0:
                    yield from m.wait("loader k_empty", k_empty, (item & 1) ^ 1)
                    m.need(*once("S", at - 1))
                    m.load(k_full, ("K", item))
                if do_stages == q_stages and at + 1 - do_stages >= 0:
                    yield from m.wait("loader dp_full", *dp_full.nth(at + 1 - do_stages))
                m.need(*once("S", at - q_stages), *once("dK", at - q_stages), *once("flags read", at - q_stages))
                flags[at] = at
                m.load(q_full.nth(at)[0], ("Q", at))
                if i == 0:
                    yield from m.wait("loader v_empty", v_empty, (item & 1) ^ 1)
                    m.need(*once("dP", at - 1))
                    m.load(v_full, ("V", item))
                if do_stages < q_stages and at >= 2:
                    yield from m.wait("loader dp_full", *dp_full.nth(at - 1))
                m.need(*once("dP", at - do_stages), *once("dV", at - do_stages))
                m.load(do_full.nth(at)[0], ("dO", at))
                at += 1
        bar, parity = row_empty.nth(at)
        yield from m.wait("loader row_empty", bar, parity ^ 1)
        m.need(*ops("row read", at - row_slots))
        rows[at] = None
        m.done.add(("row", at))
        row_full.nth(at)[0].arrive()
        m.need(*once("flags read", at - q_stages))
        flags[at] = None
        m.done.add(("Q", at))
        q_full.nth(at)[0].arrive()
        # drains: the last load of each barrier, but those whose phase the end's arrival ended behind them
        if real:
            yield k_full, (len(real) - 1) & 1
            yield v_full, (len(real) - 1) & 1
        for ring, stages, skip in ((q_full, q_stages, at % q_stages), (do_full, do_stages, None), (row_full, row_slots, at % row_slots)):
            for k in range(max(0, at - stages), at):
                if k % stages != skip:
                    yield ring.nth(k)

    def issuer():
        items_s = items_dp = 0

        def s(at):
            nonlocal items_s
            yield from m.wait("issuer q_full", *q_full.nth(at))
            m.need(("Q", at))
            what = flags[at]
            m.done.add(("flags read", at))
            if what is None:
                return
            if steps[at][0]:
                yield from m.wait("issuer k_full", k_full, items_s & 1)
                items_s += 1
            m.need(("K", items_s - 1), *ops("P", at - 1))  # over S and P of the step before
            m.queue += [("S", at), s_full] + [k_empty] * steps[at][1]

        def dp(at):
            nonlocal items_dp
            if steps[at][0]:
                yield from m.wait("issuer v_full", v_full, items_dp & 1)
                items_dp += 1
            yield from m.wait("issuer do_full", *do_full.nth(at))
            m.need(("V", items_dp - 1), ("dO", at), *ops("dS", at - 1))
            m.queue += [("dP", at), dp_full.nth(at)[0]] + [v_empty] * steps[at][1]

        yield from s(0)
        if n:
            yield from dp(0)
        item = -1
        for at in range(n):
            yield from m.wait("issuer p_full", p_full, at & 1)
            if steps[at][0]:
                item += 1
                yield from m.wait("issuer acc_empty", acc_empty, (item & 1) ^ 1)
            m.need(*ops("P", at), *ops("stored", item - 1))
            m.queue.append(("dV", at))
            yield from s(at + 1)
            yield from m.wait("issuer ds_full", ds_full, at & 1)
            m.need(*ops("dS", at), *ops("stored", item - 1))
            m.queue += [("dK", at)] + [acc_full] * steps[at][1]
            if at + 1 < n:
                yield from dp(at + 1)
        m.queue.append(mma_done)
        yield mma_done, 0

    def softmax(w):
        at, r, item, stores = None, 0, 0, False
        what = 0
        while True:
            if at is not None:
                yield from m.wait("softmax s_full", s_full, at & 1)
                m.need(("S", at), ("row", at))
                m.done.add(("P", at, w))
                p_full.arrive()
            if stores:
                yield from m.wait("softmax acc_full", acc_full, item & 1)
                m.need(("dV", last_of[item]), ("dK", last_of[item]))
                m.done.add(("stored", item, w))
                acc_empty.arrive()
                item, stores = item + 1, False
            if what is None:
                return
            yield from m.wait("softmax row_full", *row_full.nth(r))
            m.need(("row", r))
            before, what = at, rows[r]
            if what is not None and what != r:
                raise Fault("another step's row")
            r += 1
            if before is not None:
                yield from m.wait("softmax dp_full", *dp_full.nth(before))
                m.need(("dP", before))
                m.done.add(("dS", before, w))
                ds_full.arrive()
                m.done.add(("row read", before, w))
                row_empty.nth(before)[0].arrive()
                stores = steps[before][1]
            at = what

    return m, m.run({"loader": loader(), "issuer": issuer(), **{f"softmax {w}": softmax(w) for w in ALL}})


def dq(rng, items, without=None):
    m, steps, slots, k_stages, v_stages = Machine(rng, without), steps_of(items), 3, 3, 2
    n, real = len(steps), [size for size in items if size]
    item_full, item_empty = Ring(slots), Ring(slots, 1 + WARPS)
    q_full, q_empty, do_full, do_empty, s_full, dq_full, mma_done = (Bar() for _ in range(7))
    s_empty, ds_full, dq_empty = (Bar(WARPS) for _ in range(3))
    k_full, v_full, dp_full = Ring(k_stages), Ring(v_stages), Ring(2)
    held = {}
    last_of = [sum(real[:i + 1]) - 1 for i in range(len(real))]

    def read_item(slot, who):
        m.need(("item", slot))
        size = held[slot]
        m.done.add(("item read", slot, who))
        if size is not None:
            item_empty.nth(slot)[0].arrive()
        return size

    def loader():
        at, item = 0, 0
        for i, size in enumerate([*items, None]):
            bar, parity = item_empty.nth(i)
            yield from m.wait("loader item_empty", bar, parity ^ 1)
            if i >= slots:
                m.need(*[("item read", i - slots, who) for who in ("issuer", *ALL)])
            held[i] = size
            m.done.add(("item", i))
            item_full.nth(i)[0].arrive()
            for t in range(size or 0):
                if t == 0:
                    yield from m.wait("loader q_empty", q_empty, (item & 1) ^ 1)
                    m.need(*once("Q copied", item - 1))
                    m.load(q_full, ("Q", item))
                if at >= 2:
                    yield from m.wait("loader dp_full", *dp_full.nth(at - 2))
                m.need(*once("S", at - k_stages), *once("dQ", at - k_stages))
                m.load(k_full.nth(at)[0], ("K", at))
                if t == 0:
                    yield from m.wait("loader do_empty", do_empty, (item & 1) ^ 1)
                    m.need(*once("dO copied", item - 1))
                    m.load(do_full, ("dO", item))
                    item += 1
                m.need(*once("dP", at - v_stages))
                m.load(v_full.nth(at)[0], ("V", at))
                at += 1
        for ring, stages in ((k_full, k_stages), (v_full, v_stages)):
            for k in range(max(0, at - stages), at):
                yield ring.nth(k)
        if item:
            yield q_full, (item - 1) & 1
            yield do_full, (item - 1) & 1

    def issuer():
        slot = left = 0
        items_s = items_dp = -1

        def following():
            nonlocal slot, left
            while left == 0:
                yield from m.wait("issuer item_full", *item_full.nth(slot))
                left = read_item(slot, "issuer")
                if left is None:
                    return
                slot += 1
            left -= 1

        def s(at):
            nonlocal items_s
            if steps[at][0]:
                items_s += 1
                yield from m.wait("issuer q_full", q_full, items_s & 1)
                m.need(("Q", items_s))
            yield from m.wait("issuer k_full", *k_full.nth(at))
            yield from m.wait("issuer s_empty", s_empty, (at & 1) ^ 1)
            m.need(("K", at), *ops("S read", at - 1))
            if steps[at][0]:
                m.need(*once("S", at - 1))  # done with Q of the item before
                m.queue += [("Q copied", items_s), q_empty]
            m.queue += [("S", at), s_full]

        def dp(at):
            nonlocal items_dp
            if steps[at][0]:
                items_dp += 1
                yield from m.wait("issuer do_full", do_full, items_dp & 1)
                m.need(("dO", items_dp))
            yield from m.wait("issuer v_full", *v_full.nth(at))
            m.need(("V", at), *ops("dS", at - 1))
            if steps[at][0]:
                m.need(*once("dP", at - 1))
                m.queue += [("dO copied", items_dp), do_empty]
            m.queue += [("dP", at), dp_full.nth(at)[0]]

        yield from following()
        if n:
            yield from s(0)
            yield from dp(0)
        item = -1
        for at in range(n):
            yield from following()
            if at + 1 < n:
                yield from s(at + 1)
            yield from m.wait("issuer ds_full", ds_full, at & 1)
            if steps[at][0]:
                item += 1
                yield from m.wait("issuer dq_empty", dq_empty, (item & 1) ^ 1)
            m.need(*ops("dS", at), *ops("stored", item - 1))
            m.queue += [("dQ", at)] + [dq_full] * steps[at][1]
            if at + 1 < n:
                yield from dp(at + 1)
        m.queue.append(mma_done)
        yield mma_done, 0

    def softmax(w):
        slot = at = item = 0
        left, work, stores = 0, False, False
        while True:
            if work:
                yield from m.wait("softmax s_full", s_full, at & 1)
                m.need(("S", at))
                m.done.add(("S read", at, w))
                s_empty.arrive()
            if stores:
                yield from m.wait("softmax dq_full", dq_full, item & 1)
                m.need(("dQ", last_of[item]))
                m.done.add(("stored", item, w))
                dq_empty.arrive()
                item, stores = item + 1, False
            if left is None:
                return
            had = work
            if work:
                left -= 1
                stores = left == 0
            if not work or left == 0:
                while True:
                    yield from m.wait("softmax item_full", *item_full.nth(slot))
                    left = read_item(slot, w)
                    if left is None:
                        break
                    slot += 1
                    if left:
                        break
                work = left is not None
            if had:
                yield from m.wait("softmax dp_full", *dp_full.nth(at))
                m.need(("dP", at))
                m.done.add(("dS", at, w))
                ds_full.arrive()
                at += 1

    return m, m.run({"loader": loader(), "issuer": issuer(), **{f"softmax {w}": softmax(w) for w in ALL}})


def draw(seed):
    rng = random.Random(seed)
    empty = rng.choice([0, 0.3, 0.8])
    return rng, [0 if rng.random() < empty else rng.choice([1, 1, 2, 3, 5]) for _ in range(rng.randrange(10))]


HALVES = {"dK / dV, heads of 128": lambda rng, items, **kw: dkdv(rng, items, 2, 2, **kw),
          "dK / dV, heads of 64": lambda rng, items, **kw: dkdv(rng, items, 3, 4, **kw),
          "dQ": dq}
KV_WAITS = ["loader row_empty", "loader k_empty", "loader v_empty", "loader dp_full", "issuer q_full", "issuer k_full",
            "issuer v_full", "issuer do_full", "issuer p_full", "issuer acc_empty", "issuer ds_full", "softmax s_full",
            "softmax acc_full", "softmax row_full", "softmax dp_full"]
DQ_WAITS = ["loader item_empty", "loader q_empty", "loader do_empty", "loader dp_full", "issuer item_full", "issuer q_full",
            "issuer k_full", "issuer s_empty", "issuer do_full", "issuer v_full", "issuer ds_full", "issuer dq_empty",
            "softmax s_full", "softmax dq_full", "softmax item_full", "softmax dp_full"]
WAITS = {name: DQ_WAITS if name == "dQ" else KV_WAITS for name in HALVES}
# Waits that others imply, kept as the reason is far from them: a row's fourth next comes behind the wait for
# dP two steps on, which follows dS of the row's step; dS of an item's first step comes behind the stores of
# the item before.
IMPLIED = {("dK / dV, heads of 64", "loader row_empty"), ("dQ", "issuer dq_empty")}


@pytest.mark.parametrize("half", HALVES)
def test_no_order_finds_a_fault(half):
    asked = set()
    for seed in range(1000):
        rng, items = draw(seed)
        m, waiting = HALVES[half](rng, items)
        assert waiting == [], (seed, items)
        asked |= m.asked
    assert asked == set(WAITS[half])


def finds(half, without):
    for seed in range(1000):
        rng, items = draw(seed)
        try:
            if HALVES[half](rng, items, without=without)[1]:
                return True
        except (Fault, KeyError):
            return True
    return False


@pytest.mark.parametrize("half,without", [(half, name) for half in HALVES for name in WAITS[half]])
def test_a_wait_left_out_is_found(half, without):
    assert finds(half, without) != ((half, without) in IMPLIED)


# ------------------------------------------------------------------ the source
def roles(function):
    """Waits (?), arrivals (!), copies (<) and commits (>) of a function's roles, in the order they stand."""
    with open(SOURCE) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    text = text[text.index(f"void {function}("):]
    end = re.search(r"\n}\n", text).start()
    parts = re.split(r"(?:else )?if \(warp (?:==|>=) \d\) \{", text[:end])
    call = re.compile(r"(wait_phase|drain_wait|mbar_arrive_expect_tx|mbar_arrive|mma_commit_by)\((?:leader, )?&?(\w+)"
                      r"|(load_halves)<[^>]*>\([^,]*, [^,]*, &?(\w+)|(dp_there)\(")
    sign = dict(wait_phase="?", drain_wait="~", mbar_arrive_expect_tx="<", mbar_arrive="!", mma_commit_by=">")
    out = []
    for part in parts[1:]:
        names = []
        for m in call.finditer(part):
            names.append("? dp" if m[5] else f"< {m[4]}" if m[3] else f"{sign[m[1]]} {m[2]}")
        out.append(names)
    return out


def test_the_source_of_dkdv():
    loader, issuer, softmax = roles("dkdv_items")
    assert loader == ["? dp_full", "? row_empty", "! row_full", "! q_full", "? row_empty", "< row_full", "? k_empty",
                      "< k_full", "? dp", "< q_full", "? v_empty", "< v_full", "? dp", "< do_full", "~ k_full",
                      "~ v_full", "~ q_full", "~ do_full", "~ row_full"]
    assert issuer == ["? q_full", "? k_full", "> s_full", "> k_empty", "? v_full", "? do_full", "> dp_full", "> v_empty",
                      "? p_full", "? acc_empty", "? ds_full", "> acc_full", "> mma_done", "~ mma_done"]
    assert softmax == ["? row_full", "! row_empty", "? acc_full", "! acc_empty", "? s_full", "! p_full", "? dp_full",
                       "! ds_full"]


def test_the_source_of_dq():
    loader, issuer, softmax = roles("dq_items")
    assert loader == ["? item_empty", "! item_full", "! item_full", "? q_empty", "< q_full", "? dp_full", "< k_full",
                      "? do_empty", "< do_full", "< v_full", "~ k_full", "~ v_full", "~ q_full", "~ do_full"]
    assert issuer == ["? item_full", "! item_empty", "? q_full", "? k_full", "? s_empty", "> q_empty", "> s_full",
                      "? do_full", "? v_full", "> do_empty", "> dp_full", "? ds_full", "? dq_empty", "> dq_full",
                      "> mma_done", "~ mma_done"]
    assert softmax == ["? dq_full", "! dq_empty", "? item_full", "! item_empty", "? s_full", "! s_empty", "? dp_full",
                       "! ds_full"]
