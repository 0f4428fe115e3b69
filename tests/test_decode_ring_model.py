"""CPU model of the decode kernel's tile ring: one producer, consumer teams that
take the tiles in turn, full / empty barriers that are waited on by the parity
of a phase, copies that may land in any order.  Every interleaving is visited.
A wait on parity P passes whenever the barrier's current phase has the other
parity, so a waiter that is two phases ahead passes too early.  The kernel has
one team, which is sound with any number of stages; with two that happens
unless each stage stays with one of them."""
import pytest


def faults(stages, tiles, teams=2):
    """Faults that some interleaving reaches: a consumer that takes a tile which
    has not landed, or a copy into a stage whose barrier is still armed."""
    start = (0, tuple([0] * stages), tuple([0] * stages), frozenset(), tuple(range(teams)))
    seen, todo, bad, done = {start}, [start], set(), 0
    while todo:
        issued, full, empty, flying, at = todo.pop()
        after = []
        if issued < tiles:
            st, n = issued % stages, issued // stages
            if n == 0 or empty[st] % 2 != (n - 1) % 2:
                if any(x % stages == st for x in flying):
                    bad.add("armed twice")
                else:
                    after.append((issued + 1, full, empty, flying | {issued}, at))
        for x in flying:                                    # any copy may land next
            f = list(full)
            f[x % stages] += 1
            after.append((issued, tuple(f), empty, flying - {x}, at))
        for team, i in enumerate(at):
            if i >= tiles:
                continue
            st, n = i % stages, i // stages
            if full[st] % 2 != n % 2:                       # the wait passes
                if full[st] != n + 1:
                    bad.add("taken too early")
                    continue
                e = list(empty)
                e[st] += 1
                after.append((issued, full, tuple(e), flying, at[:team] + (i + teams,) + at[team + 1:]))
        if not after and issued == tiles and not flying and all(i >= tiles for i in at):
            done += 1
        elif not after and not bad:
            bad.add("stuck")
        for s in after:
            if s not in seen:
                seen.add(s)
                todo.append(s)
    assert done == 1 or bad
    return bad


@pytest.mark.parametrize("stages", [2, 3, 4, 6])
def test_one_team_is_sound(stages):
    for tiles in (1, stages, 2 * stages + 1, 3 * stages + 1):
        assert faults(stages, tiles, teams=1) == set()


@pytest.mark.parametrize("stages", [2, 4, 6])
def test_a_stage_that_stays_with_its_team_is_sound(stages):
    for tiles in (1, stages, 2 * stages + 1, 2 * stages + 4):
        assert faults(stages, tiles) == set()


@pytest.mark.parametrize("stages", [3, 5])
def test_a_stage_that_changes_teams_is_not(stages):
    assert "taken too early" in faults(stages, 3 * stages)
