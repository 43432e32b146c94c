"""The barriers of the bf16 linear attention kernels, walked through on the CPU.

A wait by parity is right only while at most the phase it waits for and none
after it can be over: two phases later the parity is the old one again, and
the wait runs out.  Likewise a warp may arrive for a phase only once the phase
before is over.  Timing makes most such mistakes invisible on a GPU, so the
roles are restated here as sequences of waits and arrivals, and each is held
back before each of its steps while all others run as far as they can.  They
only wait for one another, so that is the furthest they can get, whatever the
timing: what holds then holds always.  Copies and products complete at once.

What the restatement takes from the source is the number of `staged` barriers
(outputs ready in shared memory): one for both buffers of z lets the output
warps get two tiles ahead of the store warp.
"""
import os
import random
import re
from collections import defaultdict

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SOURCE = os.path.join(ROOT, "long_context_attention_causal_gb300", "csrc", "polar_linear_tc.cu")
OUT_WARPS = 4


def staged_barriers():
    text = re.search(r"struct OutBars \{(.*?)\n\};", open(SOURCE).read(), re.S).group(1)
    return int(re.search(r"\bstaged(?:\[(\d)\])?[,;]", text).group(1) or 1)


class Hazard(Exception):
    pass


class Machine:
    """roles: {name: [("wait" | "arrive", barrier, phase), ..]}; counts: the
    arrivals that end a phase of a barrier."""

    def __init__(self, roles, counts):
        self.roles, self.counts = roles, counts
        self.at = dict.fromkeys(roles, 0)
        self.arrived = defaultdict(int)

    def over(self, bar):
        return self.arrived[bar] // self.counts[bar[0]]

    def step(self, name):
        """One step of a role; False where it has to wait or is through."""
        if self.at[name] == len(self.roles[name]):
            return False
        kind, bar, phase = self.roles[name][self.at[name]]
        over = self.over(bar)
        if kind == "wait":
            if over > phase + 1:
                raise Hazard(f"{name} waits for phase {phase} of {bar}, {over} are over")
            if over <= phase:
                return False
        else:
            if over != phase:
                raise Hazard(f"{name} arrives for phase {phase} of {bar}, {over} are over")
            self.arrived[bar] += 1
        self.at[name] += 1
        return True

    def run(self, names):
        moved = True
        while moved:
            moved = False
            for n in names:
                while self.step(n):
                    moved = True

    def done(self):
        return all(self.at[n] == len(r) for n, r in self.roles.items())


def check(roles, counts):
    """Hold every role before every step, run the others, then let it go on."""
    m = Machine(roles, counts)
    m.run(list(roles))
    assert m.done(), {n: (m.at[n], len(r)) for n, r in roles.items() if m.at[n] < len(r)}
    seen = set()
    for held in roles:
        key = (held.rstrip("0123456789"), tuple(roles[held]))
        if key in seen:          # its twins do the same
            continue
        seen.add(key)
        m = Machine(roles, counts)
        others = [n for n in roles if n != held]
        while m.at[held] < len(roles[held]):
            m.run(others)
            assert m.step(held), f"{held} stands still at {roles[held][m.at[held]]}"


def state_warps(terms):
    return 16 if terms == 3 else 8


def out_roles(portions, staged, terms, apart):
    """portions: [(tiles, final state wanted, rows to zero in these tiles)];
    terms: of scaled y; apart: each has a buffer of its own."""
    tma, mma, store, out, state = [], [], [], [], []

    def two(bar, k):
        return (bar, k % 2), k // 2

    def add(role, kind, *bar_phase):
        for b, p in bar_phase:
            role.append((kind, b if isinstance(b, tuple) else (b,), p))

    def one(bar, k):
        return (bar,), k

    k = ku = kf = 0
    for live, final, ragged in portions:
        wait_ds = False
        for c in range(live):
            upd = c + 1 < live or final
            if k >= 2:
                add(tma, "wait", two("empty_x", k - 2))
            add(tma, "arrive", two("full_x", k))
            if k >= 1:
                add(tma, "wait", one("empty_y", k - 1))
            add(tma, "arrive", one("full_y", k))
            if k >= 2:
                add(tma, "wait", two("empty_z", k - 2))
            add(tma, "arrive", two("full_z", k))

            add(mma, "wait", two("full_x", k), one("full_y", k))
            if c in ragged:
                add(mma, "wait", one("fixed", kf))
            add(mma, "arrive", one("s_full", k), one("empty_y", k))
            add(mma, "wait", one("m_op", k))
            if k > 0:
                add(mma, "wait", one("o_free", k - 1))
            add(mma, "arrive", two("empty_x", k))
            add(mma, "wait", two("full_z", k))
            if upd:
                add(mma, "wait", one("first", ku))
                if not apart:
                    if terms == 3:
                        add(mma, "arrive", one("first_done", ku))
                        add(mma, "wait", one("second", ku))
                    add(mma, "wait", one("last", ku))
                add(mma, "arrive", one("ds_full", ku))
            add(mma, "wait", one("p_full", k))
            add(mma, "arrive", one("o_full", k))

            ready = two("staged", k) if staged == 2 else one("staged", k)
            add(store, "wait", ready)
            add(store, "arrive", two("empty_z", k))

            add(out, "wait", one("s_full", k), two("empty_x", k))
            add(out, "arrive", one("p_full", k))
            add(out, "wait", one("o_full", k))
            add(out, "arrive", one("o_free", k), ready)

            add(state, "wait", one("full_y", k))
            if c in ragged:
                add(state, "wait", two("full_z", k))
                add(state, "arrive", one("fixed", kf))
                kf += 1
            add(state, "arrive", one("empty_y", k))
            if wait_ds:
                add(state, "wait", one("ds_full", ku - 1))
            add(state, "arrive", one("m_op", k))
            if upd:
                add(state, "arrive", one("first", ku))
                if not apart:
                    if terms == 3:
                        add(state, "wait", one("first_done", ku))
                        add(state, "arrive", one("second", ku))
                    add(state, "wait", two("empty_x", k))
                    add(state, "arrive", one("last", ku))
                ku += 1
            else:
                add(state, "wait", two("empty_x", k))
            wait_ds = upd
            k += 1
        if final and wait_ds:
            add(state, "wait", one("ds_full", ku - 1))
    roles = {"tma": tma, "mma": mma, "store": store}
    roles.update({f"out{i}": out for i in range(OUT_WARPS)})
    roles.update({f"state{i}": state for i in range(state_warps(terms))})
    counts = dict.fromkeys("full_x full_z empty_x empty_z full_y s_full o_full ds_full first_done"
                           .split(), 1)
    counts.update(dict.fromkeys("p_full o_free staged".split(), OUT_WARPS))
    counts.update(dict.fromkeys("m_op first second last fixed".split(), state_warps(terms)))
    counts["empty_y"] = 1 + state_warps(terms)
    return roles, counts


def state_roles(tiles, stages, terms):
    tma, mma, work = [], [], []

    def ring(bar, c):
        return (bar, c % stages), c // stages

    for c in range(tiles):
        if c >= stages:
            tma.append(("wait", *ring("empty", c - stages)))
        tma.append(("arrive", *ring("full", c)))
        mma.append(("wait", *ring("first", c)))
        if terms == 3:
            mma.append(("arrive", ("first_done",), c))
        mma.append(("wait", ("second",), c))
        if terms == 3:
            mma.append(("wait", ("third",), c))
        mma += [("arrive", ("sums",), c), ("arrive", *ring("empty", c))]
        work += [("wait", *ring("full", c)), ("arrive", *ring("first", c))]
        if c:
            work.append(("wait", ("sums",), c - 1))
        work.append(("arrive", ("second",), c))
        if terms == 3:
            work += [("wait", ("first_done",), c), ("arrive", ("third",), c)]
    if tiles:
        work.append(("wait", ("sums",), tiles - 1))
    roles = {"tma": tma, "mma": mma, **{f"work{i}": work for i in range(state_warps(terms))}}
    counts = dict.fromkeys("full empty sums first_done".split(), 1)
    counts.update(dict.fromkeys("first second third".split(), state_warps(terms)))
    return roles, counts


def walks():
    yield [(1, False, ())] * 6
    yield [(1, True, ())] * 6
    yield [(9, False, ())]
    yield [(9, True, (8,))]
    yield [(0, True, ()), (1, False, (0,)), (0, False, ()), (2, True, (1,))] * 2
    rng = random.Random(7)
    for _ in range(40):
        yield [(n := rng.choice([0, 1, 1, 2, 3, 5]), rng.random() < 0.5,
                (n - 1,) if n and rng.random() < 0.5 else ()) for _ in range(rng.randint(1, 6))]


@pytest.mark.parametrize("terms", [2, 3])
@pytest.mark.parametrize("apart", [False, True])
def test_output_kernel(terms, apart):
    for portions in walks():
        check(*out_roles(portions, staged_barriers(), terms, apart))


def test_one_staged_barrier_would_not_do():
    with pytest.raises(Hazard, match="store waits"):
        check(*out_roles([(9, False, ())], 1, 2, False))


@pytest.mark.parametrize("stages", [3, 6])
@pytest.mark.parametrize("terms", [2, 3])
def test_state_kernel(stages, terms):
    for tiles in (0, 1, 2, 3, 7, 20):
        check(*state_roles(tiles, stages, terms))
