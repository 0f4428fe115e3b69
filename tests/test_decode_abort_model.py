"""The decode kernel's expired waits, over every interleaving on the CPU.

Every wait of the ring is bounded: once its limit passes, or once another warp
gave up, a role stops waiting and runs on.  The model has the producer warp and
two consumer warps (a stage is handed back by all of them), lets any role give
up at any wait whose event has not happened, at any moment, and any copy land
at any moment, and checks that
  * no stage is armed while its last copy is in flight (its barrier would count
    two copies in one phase);
  * no copy is in flight once every role has ended (the CTA's shared memory then
    belongs to another one);
  * no role is left at a barrier, and while nobody has given up every tile is
    taken after it landed.
The consumers' barrier within a tile has no limit: each of them reaches it for
every tile.  Two facts that the checks rest on are read from the kernel's source:
whether a consumer that gave up still hands a stage back, and whether the
producer waits for its last copies in every case; so is the number of stages."""
import re
from pathlib import Path

import pytest

SOURCE = (Path(__file__).resolve().parents[1] / "attention_forward_fa_gb300/csrc/fa_decode.cuh").read_text()


def facts():
    """(consumers that gave up hand back stages, the producer always drains)."""
    arrive = re.findall(r"if \(lane == 0([^)]*)\) mbar_arrive\(EMPTY\(st\)\);", SOURCE)
    drain = re.findall(r"if \(([^)]*)\)\s*for \(int i = max\(0, it - NS\); i < it; \+\+i\) "
                       r"drain_bar\(FULL\(i % NS\), \(i / NS\) & 1, wc\.timeout\);", SOURCE)
    assert len(arrive) == 1 and len(drain) == 1, "the ring's hand-back or drain is written in another way"
    return "!dead" not in arrive[0], "dead" not in drain[0]


def stages(D):
    m = re.search(r"kStages = (\d+) \* \((\d+) / D\);", SOURCE)
    return int(m[1]) * (int(m[2]) // D)


def explore(ns, tiles, hands_back_dead, always_drains, consumers=2, may_give_up=True):
    """Faults that some interleaving reaches."""
    # producer: (place, tile, drained up to, dead); place: wait, arm, drain, end
    # consumer: (place, tile, dead); place: wait, sync, back, end
    start = (("wait", 0, 0, False), tuple(("wait", 0, False) for _ in range(consumers)),
             tuple([0] * ns),                       # completed phases of FULL
             tuple([(0, 0)] * ns),                  # EMPTY: completed phases, arrivals
             frozenset(), False)                    # copies in flight (tiles), the abort flag
    seen, todo, bad, ends = {start}, [start], set(), 0
    while todo:
        state = todo.pop()
        prod, cons, full, empty, flying, abort = state
        after = []

        def passes(count, n):                       # try_wait on the parity of phase n
            return count % 2 != n % 2

        place, it, drained, dead = prod
        if place == "wait":
            st, n = it % ns, it // ns
            if it == tiles:
                first = max(0, it - ns)
                to = ("drain", it, first, dead) if always_drains or dead else ("end", it, 0, dead)
                after.append((to, cons, full, empty, flying, abort))
            elif n == 0 or passes(empty[st][0], n - 1):
                after.append((("arm", it, 0, dead), cons, full, empty, flying, abort))
            elif may_give_up or abort:              # its limit, or the flag
                after.append((("drain", it, max(0, it - ns), True), cons, full, empty, flying, True))
        elif place == "arm":
            st = it % ns
            if any(x % ns == st for x in flying) or full[st] != it // ns:
                bad.add("armed with a copy in flight")
            else:
                after.append((("wait", it + 1, 0, dead), cons, full, empty, flying | {it}, abort))
        elif place == "drain":
            if drained == it:
                after.append((("end", it, 0, dead), cons, full, empty, flying, abort))
            elif passes(full[drained % ns], drained // ns):
                after.append((("drain", it, drained + 1, dead), cons, full, empty, flying, abort))
        for x in flying:                            # a copy lands
            f = list(full)
            f[x % ns] += 1
            after.append((prod, cons, tuple(f), empty, flying - {x}, abort))
        for i, (place, at, gone) in enumerate(cons):
            def to(new, **kw):
                d = dict(empty=empty, abort=abort)
                d.update(kw)
                return (prod, cons[:i] + (new,) + cons[i + 1:], full, d["empty"], flying, d["abort"])

            if place == "wait":
                if at == tiles:
                    after.append(to(("end", at, gone)))
                elif gone:
                    after.append(to(("sync", at, True)))
                else:
                    st, n = at % ns, at // ns
                    if passes(full[st], n):
                        if not abort and full[st] != n + 1:
                            bad.add("taken before it landed")
                        after.append(to(("sync", at, False)))
                    elif may_give_up or abort:
                        after.append(to(("sync", at, True), abort=True))
            elif place == "back":
                e = empty
                if hands_back_dead or not gone:
                    st = at % ns
                    phases, here = e[st]
                    here += 1
                    if here == consumers:
                        phases, here = phases + 1, 0
                    e = e[:st] + ((phases, here),) + e[st + 1:]
                after.append(to(("wait", at + 1, gone), empty=e))
        if all(c[0] == "sync" for c in cons):       # the consumers' barrier
            assert len({c[1] for c in cons}) == 1
            after.append((prod, tuple(("back",) + c[1:] for c in cons), full, empty, flying, abort))
        if prod[0] == "end" and all(c[0] == "end" for c in cons):
            ends += 1
            if flying:
                bad.add("in flight at the end")
            continue
        if not after and not bad:
            bad.add("stuck")
        for s in after:
            if s not in seen:
                seen.add(s)
                todo.append(s)
    assert ends or bad
    return bad


@pytest.mark.parametrize("D", [64, 128])
def test_expired_waits_leave_nothing_in_flight(D):
    ns = stages(D)
    for tiles in (1, ns - 1, ns, ns + 1, 2 * ns + 1):
        assert explore(ns, tiles, *facts()) == set()


@pytest.mark.parametrize("D", [64, 128])
def test_without_expired_waits_every_tile_is_taken(D):
    ns = stages(D)
    for tiles in (1, ns, 2 * ns + 1, 3 * ns):
        assert explore(ns, tiles, *facts(), may_give_up=False) == set()


def test_three_consumers():
    assert explore(2, 5, *facts(), consumers=3) == set()


def test_the_model_sees_a_stage_handed_back_by_a_warp_that_gave_up():
    assert "armed with a copy in flight" in explore(2, 5, True, True)


def test_the_model_sees_a_missing_drain():
    assert "in flight at the end" in explore(2, 2, False, False)
