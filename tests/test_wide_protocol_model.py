"""CPU model of the hand-offs of fa_wide_kernel: producer, converters, issuer, the tensor
cores, and two groups of softmax warps, each as the kernel's loops produce its waits and
arrivals, under random schedules.

A barrier counts arrivals per phase; a wait on a parity passes while the barrier's current
phase has the other one (so a waiter two phases off passes too early or never).  Tensor
core work runs in order of issue, some time after it, and a commit arrives once everything
before it has run.  Checked at every step: a tile is read from the stage that holds it, no
stage, S, O or Q is overwritten before its last reader is done, the keys and scales of a
tile are still those of the tile when their last reader leaves, the second group's O and
sums stay until the first has joined them; and every role ends.

Stages, the depth of the ring of keys and scales and which loads go where are read from the
source.  Each group of softmax warps is two warps here (four there), each half of the
converters two (three there)."""
import random
import re
from pathlib import Path

import pytest

SOURCE = (Path(__file__).resolve().parents[1] / "attention_forward_fa_gb300/csrc/fa_wide.cuh").read_text()


def cpp(expr, D, eight, split):
    """A chain of C++ conditionals over D, EIGHT and SPLIT."""
    expr = re.sub(r"\bEIGHT\b", str(int(eight)), expr)
    expr = re.sub(r"\bSPLIT\b", str(int(split)), expr)
    expr = re.sub(r"\bD\b", str(D), expr).replace("!", "not ")

    def pick(e):
        e = e.strip()
        while e.startswith("(") and closing(e) == len(e) - 1:
            e = e[1:-1].strip()
        depth = 0
        for i, ch in enumerate(e):
            depth += (ch == "(") - (ch == ")")
            if ch == "?" and depth == 0:
                level, inner = 0, 0
                for j in range(i + 1, len(e)):
                    inner += (e[j] == "(") - (e[j] == ")")
                    if inner == 0 and e[j] == "?":
                        level += 1
                    if inner == 0 and e[j] == ":":
                        if level == 0:
                            return pick(e[i + 1:j]) if eval(e[:i]) else pick(e[j + 1:])
                        level -= 1
        return int(eval(e))

    def closing(e):
        depth = 0
        for i, ch in enumerate(e):
            depth += (ch == "(") - (ch == ")")
            if depth == 0:
                return i

    return pick(expr)


def stages(D, eight, split):
    ops = re.search(r"int kStages = ([^;]+);", SOURCE)[1]
    raw = re.search(r"int kRawStages = ([^;]+);", SOURCE)[1]
    return cpp(ops, D, eight, split), cpp(raw, D, eight, split)


INFO = int(re.search(r"constexpr int kWideInfo = (\d+);", SOURCE)[1])


def test_the_model_follows_the_source():
    assert stages(128, False, False) == (5, 0) and stages(64, False, True) == (10, 0)
    assert stages(128, True, True)[1] > 0
    for line in ("if (SPLIT && t == 1 && piece > 0 && !__all_sync(0xffffffffu, wait_bar(QREADY, (piece - 1) & 1, wc))) break;",
                 "const int ld = 2 * tile + kind;", "if (last) mma_commit_if(EMPTY(ld % NS), lead);", "mbar_init(QREADY, 8);",
                 "mbar_init(JOIN, 4);", "mbar_init(PREADY(t), 4);", "mbar_init(EMPTY(s), 1);",
                 "ok = wait_bar(EIGHT ? REMPTY(st) : EMPTY(st), (n - 1) & 1, wc);"):
        assert line in SOURCE, line


class Bar:
    def __init__(self, count):
        self.count, self.here, self.phase = count, 0, 0

    def arrive(self):
        self.here += 1
        if self.here == self.count:
            self.here, self.phase = 0, self.phase + 1

    def passed(self, parity):
        return self.phase % 2 != parity


def run(pieces, NS, RS, split, info, seed, planted=None):
    """Runs one random schedule; an AssertionError says what went wrong."""
    rng = random.Random(seed)
    eight = RS > 0
    full = [Bar(2 if eight else 1) for _ in range(NS)]
    empty = [Bar(1) for _ in range(NS)]
    rfull = [Bar(1) for _ in range(RS)]
    rempty = [Bar(2) for _ in range(RS)]
    sfull, pready, ofull = ([Bar(n) for _ in range(2)] for n in (1, 2, 1))
    qready, join = Bar(4), Bar(2)
    op, raw = [None] * NS, [None] * RS           # the load that a stage holds
    parts = [0] * NS                             # converters that have written it
    readers = [0] * NS                           # tensor core work in flight on it
    meta = [None] * info
    S = ["free", "free"]                         # of a group: free, ("S", tile), ("P", tile)
    half = [0, 0]                                # softmax warps that have made P of it
    O, done = [None, None], [0, 0]               # the piece that an accumulator belongs to; that it is answered up to
    Q = [None, None]
    s_in_flight = 0
    ml = None
    queue = []
    firsts = [sum(pieces[:i]) for i in range(len(pieces))]
    total = sum(pieces)

    def put(st, ld):
        assert readers[st] == 0, "a stage is overwritten under the tensor cores"
        op[st] = ld

    def producer():
        n_ring = RS if eight else NS
        for tile in range(total):
            for kind in range(2):
                ld = 2 * tile + kind
                st, n = ld % n_ring, ld // n_ring
                if n > 0:
                    bar = rempty[st] if eight else empty[st]
                    yield lambda: bar.passed((n - 1) & 1)
                if kind == 0:
                    meta[tile % info] = tile
                yield None
                if eight:
                    assert raw[st] is None, "codes are overwritten"
                    raw[st] = ld
                    rfull[st].arrive()
                else:
                    put(st, ld)
                    full[st].arrive()

    def converter(kind):
        for tile in range(total):
            ld = 2 * tile + kind
            rs, st = ld % RS, ld % NS
            yield lambda: rfull[rs].passed((ld // RS) & 1)
            if ld >= NS and planted != "no wait for the stage":
                yield lambda: empty[st].passed((ld // NS - 1) & 1)
            assert raw[rs] == ld and meta[tile % info] == tile
            if parts[st] == 0:
                put(st, None)
            parts[st] += 1
            yield None
            assert raw[rs] == ld and meta[tile % info] == tile
            if parts[st] == 2:
                parts[st] = 0
                put(st, ld)
            full[st].arrive()
            if rempty[rs].here == 1:
                raw[rs] = None
            rempty[rs].arrive()

    def tensor_cores():
        nonlocal s_in_flight
        while True:
            yield lambda: queue
            work = queue.pop(0)
            if work is None:
                return
            if work[0] == "commit":
                work[1].arrive()
                continue
            _, t, tile, piece = work
            st = (2 * tile + (work[0] == "PV")) % NS
            assert op[st] == 2 * tile + (work[0] == "PV"), "the stage holds another tile"
            if work[0] == "S":
                assert S[t] == "free", "S is written over P that is still wanted"
                assert Q[0 if split else t] == piece, "Q of another piece"
                S[t] = ("S", tile)
                s_in_flight -= 1
            else:
                assert S[t] == ("P", tile)
                if O[t] != piece:
                    assert O[t] is None or done[t] > O[t], "O is overwritten before its answer has left"
                    O[t] = piece
                S[t] = "free"
            readers[st] -= 1

    def issuer():
        nonlocal s_in_flight
        made = [0, 0]

        def issue(what, t, tile, piece):
            nonlocal s_in_flight
            readers[(2 * tile + (what == "PV")) % NS] += 1
            s_in_flight += what == "S"
            queue.append((what, t, tile, piece))

        def scores(t, tile, piece, last):
            issue("S", t, tile, piece)
            queue.append(("commit", sfull[t]))
            if last:
                queue.append(("commit", empty[(2 * tile) % NS]))

        def landed(ld):
            return lambda: full[ld % NS].passed((ld // NS) & 1)

        for piece, nt in enumerate(pieces):
            tile = firsts[piece]
            yield lambda: qready.passed(piece & 1)
            yield landed(2 * tile)
            if split:
                scores(0, tile, piece, True)
                if nt > 1:
                    yield landed(2 * tile + 2)
                    scores(1, tile + 1, piece, True)
            else:
                scores(0, tile, piece, False)
                scores(1, tile, piece, True)
            for j in range(nt):
                tile = firsts[piece] + j
                yield landed(2 * tile + 1)
                for t in ([j & 1] if split else [0, 1]):
                    yield lambda: pready[t].passed(made[t] & 1)
                    made[t] += 1
                    issue("PV", t, tile, piece)
                    if split or t == 1:
                        queue.append(("commit", empty[(2 * tile + 1) % NS]))
                    step = 2 if split else 1
                    if j + step < nt:
                        if split or t == 0:
                            yield landed(2 * (tile + step))
                        scores(t, tile + step, piece, split or t == 1)
                    else:
                        queue.append(("commit", ofull[t]))
        queue.append(None)

    qrows = [0, 0]                               # warps that have written their rows of a Q

    def softmax(t):
        nonlocal ml
        made = pieces_of = joins = 0
        for piece, nt in enumerate(pieces):
            q = 0 if split else t
            if split and t == 1 and piece and planted != "no wait at Q":
                yield lambda: qready.passed((piece - 1) & 1)
            if not split or t == 0:
                assert not any(w and w[0] == "S" and (split or w[1] == t) for w in queue), "Q is overwritten under S"
                qrows[q] += 1
                if qrows[q] == 2:
                    qrows[q], Q[q] = 0, piece
            yield None
            qready.arrive()
            n = 0
            for j in range(t if split else 0, nt, 2 if split else 1):
                tile = firsts[piece] + j
                yield lambda: sfull[t].passed(made & 1)
                made += 1
                n += 1
                assert S[t] in (("S", tile),), "another tile's S"
                assert meta[tile % info] == tile, "the keys of another tile"
                yield None
                assert meta[tile % info] == tile, "the keys changed under a reader"
                half[t] += 1
                if half[t] == 2:
                    half[t], S[t] = 0, ("P", tile)
                pready[t].arrive()
                while S[t] == ("S", tile):       # (a warp's own P does not let the next S in by itself)
                    yield None
            if n:
                yield lambda: ofull[t].passed(pieces_of & 1)
                pieces_of += 1
                assert O[t] == piece
            if split and t == 1:
                if n:
                    ml = piece
                    yield None
                    join.arrive()
                continue
            if split and nt > 1 and planted != "no wait for the other group":
                yield lambda: ofull[1].passed(joins & 1)
                yield lambda: join.passed(joins & 1)
                joins += 1
            if split and nt > 1:
                assert O[1] == piece and ml == piece, "the second group's part is not there"
                yield None
                assert O[1] == piece and ml == piece, "the second group's part is gone"
                done[1] = piece + 1
            yield None
            assert O[t] == piece
            answered[t] += 1
            if answered[t] == 2:
                answered[t] = 0
                done[t] = piece + 1

    answered = [0, 0]
    roles = [producer(), issuer(), tensor_cores()] + [softmax(t) for t in (0, 0, 1, 1)]
    if eight:
        roles += [converter(k) for k in (0, 0, 1, 1)]
    waits = {}
    for r in roles:
        waits[r] = next(r, StopIteration)
    live = [r for r in roles if waits[r] is not StopIteration]
    while live:
        able = [r for r in live if waits[r] is None or waits[r]()]
        assert able, "stuck"
        r = rng.choice(able)
        waits[r] = next(r, StopIteration)
        if waits[r] is StopIteration:
            live.remove(r)
    assert not queue


CASES = [[1], [2], [3], [1, 1, 1, 1], [2, 1, 3, 1, 2], [7, 1, 4], [1, 6, 2, 2, 5], [15]]


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("eight", [False, True])
@pytest.mark.parametrize("split", [False, True])
def test_every_hand_off_holds(D, eight, split):
    NS, RS = stages(D, eight, split)
    for i, pieces in enumerate(CASES):
        for seed in range(60):
            run(pieces, NS, RS, split, INFO, 1000 * i + seed)


@pytest.mark.parametrize("split", [False, True])
def test_the_model_sees_a_shorter_ring_of_keys(split):
    with pytest.raises(AssertionError):
        for seed in range(300):
            run([15], *stages(64, False, split), split, 2, seed)


def test_the_model_sees_a_group_that_stands_for_the_other():
    """Pieces of one tile leave the second group nothing to wait for."""
    with pytest.raises(AssertionError):
        for seed in range(300):
            run([1, 1, 1], *stages(128, False, True), True, INFO, seed, planted="no wait at Q")


def test_the_model_sees_a_stage_taken_too_early():
    with pytest.raises(AssertionError):
        for seed in range(300):
            run([9], *stages(128, True, True), True, INFO, seed, planted="no wait for the stage")


def test_the_model_sees_a_join_that_does_not_wait():
    with pytest.raises(AssertionError):
        for seed in range(300):
            run([2, 3, 2], *stages(128, False, True), True, INFO, seed, planted="no wait for the other group")
