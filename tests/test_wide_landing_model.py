"""CPU model of fa_wide_kernel's loads: copies that land in any order, converters of K and of V that
each see every other one, and commits of the tensor cores that arrive in any order.

A wait on a phase's parity passes while the barrier's current phase has the other one, so that it
also passes two phases early: whoever waits for a phase has to know that the one before is over.
Two kinds of waiters that share the barriers of a ring with an odd number of stages do not know it.
The model's producer, memory, converters, issuer, tensor cores and softmax warps wait on the
barriers that the source names; a tile is read only from the stage that holds it, landed and whole.
(tests/test_wide_protocol_model.py has the other hand-offs; its copies land as they are issued.)"""
import random
import re

import pytest

from tests.test_wide_protocol_model import SOURCE, Bar, cpp, stages


def barriers(D, eight, split):
    """Barriers of the ring of operand tiles and of that of codes."""
    ST, RS = stages(D, eight, split)
    got = []
    for name in ("kOpBars", "kRawBars"):
        e = re.search(rf"int {name} = ([^;]+);", SOURCE)[1]
        e = re.sub(r"\bkStages\b", str(ST), re.sub(r"\bkRawStages\b", str(RS), e)).replace("&&", "and")
        got.append(cpp(e, D, eight, split))
    return got


def test_the_model_follows_the_source():
    for line in ("constexpr int R = EIGHT ? RS : ST, B = EIGHT ? RB : NS;",
                 "auto there = [&](int ld) { return EIGHT ? RFULL(ld % B) : FULL(ld % B); };",
                 "const int st = (ld + B - R) % B, n = (ld + B - R) / B;",
                 "ok = wait_bar(EIGHT ? REMPTY(st) : EMPTY(st), (n - 1) & 1, wc);",
                 "const uint32_t bar = there(ld), to = ld % R;",
                 "wait_bar(RFULL(ld % RB), (ld / RB) & 1, wc)",
                 "if (!dead && ld >= ST && !__all_sync(0xffffffffu, wait_bar(EMPTY((ld - ST) % NS), ((ld - ST) / NS) & 1, wc)))",
                 "mbar_arrive(FULL(ld % NS));", "mbar_arrive(REMPTY(ld % RB));", "if (last) mma_commit_if(EMPTY(ld % NS), lead);",
                 "wait_bar(FULL(ld % NS), (ld / NS) & 1, wc)", "mbar_init(RFULL(s), 1);", "mbar_init(REMPTY(s), kWideConverters);",
                 "mbar_init(FULL(s), EIGHT ? kWideConverters : 1);", "rs = ld % RS, st = ld % ST;"):
        assert line in SOURCE, line
    for D in (64, 128):
        for split in (False, True):
            for eight in (False, True):
                ST, RS = stages(D, eight, split)
                NS, RB = barriers(D, eight, split)
                assert NS % ST == 0 and (RS == 0 or RB % RS == 0)
                if eight:                        # every barrier belongs to K or to V
                    assert NS % 2 == 0 and RB % 2 == 0


def run(pieces, ST, NS, RS, RB, split, seed):
    """One random schedule; an AssertionError says what went wrong."""
    rng = random.Random(seed)
    eight = RS > 0
    full = [Bar(2 if eight else 1) for _ in range(NS)]
    empty = [Bar(1) for _ in range(NS)]
    rfull = [Bar(1) for _ in range(RB)]
    rempty = [Bar(2) for _ in range(RB)]
    sfull, pready = [Bar(1), Bar(1)], [Bar(1), Bar(1)]
    op, raw = [None] * ST, [None] * RS           # the load that a stage holds, landed
    parts, readers = [0] * ST, [0] * ST
    flying, queue, commits = [], [], []          # copies, tensor core work, commits on their way
    total = sum(pieces)
    loads, issued = 2 * total, [0]

    def put(st, ld):
        assert readers[st] == 0, "a stage is overwritten under its readers"
        op[st] = ld

    def producer():
        R, B = (RS, RB) if eight else (ST, NS)
        for ld in range(loads):
            st, n = (ld + B - R) % B, (ld + B - R) // B
            if n > 0:
                bar = (rempty if eight else empty)[st]
                yield lambda: bar.passed((n - 1) & 1)
            if eight:
                assert raw[ld % R] is None, "codes are overwritten"
            else:
                put(ld % R, None)
            flying.append(ld)
            issued[0] += 1
            yield None

    def memory():
        while True:
            yield lambda: flying or issued[0] == loads
            if not flying:
                return
            ld = flying.pop(rng.randrange(len(flying)))
            if eight:
                raw[ld % RS] = ld
                rfull[ld % RB].arrive()
            else:
                op[ld % ST] = ld
                full[ld % NS].arrive()

    def converter(kind):
        for tile in range(total):
            ld = 2 * tile + kind
            rs, st = ld % RS, ld % ST
            yield lambda: rfull[ld % RB].passed((ld // RB) & 1)
            if ld >= ST:
                yield lambda: empty[(ld - ST) % NS].passed(((ld - ST) // NS) & 1)
            assert raw[rs] == ld, "codes that have not landed, or another load's"
            if parts[st] == 0:
                put(st, None)
            parts[st] += 1
            yield None
            assert raw[rs] == ld, "codes change under a converter"
            if parts[st] == 2:
                parts[st] = 0
                put(st, ld)
            full[ld % NS].arrive()
            if rempty[ld % RB].here == 1:
                raw[rs] = None
            rempty[ld % RB].arrive()

    ended = [0]

    def tensor_cores():
        while True:
            yield lambda: queue
            work = queue.pop(0)
            if work is None:
                ended[0] = 1
                return
            if isinstance(work, Bar):
                commits.append(work)
                continue
            st = work[1] % ST
            assert op[st] == work[1], "the stage holds another tile"
            readers[st] -= 1

    def arrivals():                              # of commits: behind all before them, in any order of their own
        while True:
            yield lambda: commits or ended[0]
            if not commits:
                return
            commits.pop(rng.randrange(len(commits))).arrive()

    def issuer():
        made, first = [0, 0], 0

        def issue(ld, *bars):
            readers[ld % ST] += 1
            queue.append(("mma", ld))
            queue.extend(bars)

        def landed(ld):
            return lambda: full[ld % NS].passed((ld // NS) & 1)

        for nt in pieces:
            yield landed(2 * first)
            e = empty[(2 * first) % NS]
            if split:
                issue(2 * first, sfull[0], e)
                if nt > 1:
                    yield landed(2 * first + 2)
                    issue(2 * first + 2, sfull[1], empty[(2 * first + 2) % NS])
            else:
                issue(2 * first, sfull[0])
                issue(2 * first, sfull[1], e)
            for j in range(nt):
                tile = first + j
                yield landed(2 * tile + 1)
                for t in ([j & 1] if split else [0, 1]):
                    yield lambda: pready[t].passed(made[t] & 1)
                    made[t] += 1
                    last = [empty[(2 * tile + 1) % NS]] if split or t == 1 else []
                    issue(2 * tile + 1, *last)
                    step = 2 if split else 1
                    if j + step < nt:
                        k = 2 * (tile + step)
                        if split or t == 0:
                            yield landed(k)
                        issue(k, sfull[t], *([empty[k % NS]] if split or t == 1 else []))
            first += nt
        queue.append(None)

    def softmax(t):
        made = first = 0
        for nt in pieces:
            for j in range(t if split else 0, nt, 2 if split else 1):
                yield lambda: sfull[t].passed(made & 1)
                made += 1
                if not eight and rng.random() < 0.5:     # a masked tile: rows of V become 0
                    ld = 2 * (first + j) + 1
                    yield lambda: full[ld % NS].passed((ld // NS) & 1)
                    assert op[ld % ST] == ld, "V has not landed"
                yield None
                pready[t].arrive()
            first += nt

    roles = [producer(), memory(), tensor_cores(), arrivals(), issuer(), softmax(0), softmax(1)]
    if eight:
        roles += [converter(k) for k in (0, 0, 1, 1)]
    rng.shuffle(roles)
    slow = rng.choice(roles)                     # one role takes its turn rarely, so that others run ahead
    waits = {r: next(r, StopIteration) for r in roles}
    live = [r for r in roles if waits[r] is not StopIteration]
    while live:
        able = [r for r in live if waits[r] is None or waits[r]()]
        assert able, "stuck"
        quick = [r for r in able if r is not slow]
        r = rng.choice(quick if quick and rng.random() < 0.9 else able)
        waits[r] = next(r, StopIteration)
        if waits[r] is StopIteration:
            live.remove(r)
    assert not queue and not commits and not flying


CASES = [[1], [2], [3], [1, 1, 1, 1], [2, 1, 3, 1, 2], [7, 1, 4], [1, 6, 2, 2, 5], [15]]


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("eight", [False, True])
@pytest.mark.parametrize("split", [False, True])
def test_copies_may_land_in_any_order(D, eight, split):
    ST, RS = stages(D, eight, split)
    NS, RB = barriers(D, eight, split)
    for i, pieces in enumerate(CASES):
        for seed in range(60):
            run(pieces, ST, NS, RS, RB, split, 1000 * i + seed)


@pytest.mark.parametrize("split", [False, True])
def test_the_model_sees_a_barrier_per_stage_of_an_odd_ring(split):
    """K's and V's converters taking turns at three barriers read codes that have not landed."""
    ST, _ = stages(128, True, split)
    with pytest.raises(AssertionError, match="codes|stuck|stage"):
        for seed in range(400):
            run([15], ST, 2 * ST if ST % 2 else ST, 3, 3, split, seed)


def test_the_model_sees_an_odd_ring_of_operand_tiles():
    """Three operand stages with a barrier each: a converter takes a stage under its readers, once
    commits may arrive in any order."""
    with pytest.raises(AssertionError):
        for seed in range(2000):
            run([15], 3, 3, 4, 4, False, seed)
