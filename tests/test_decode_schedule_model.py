"""CPU model of the decode kernels' schedule: the units of all sequences, charged
a fixed number of tiles each, are cut into equal ranges, one per CTA; every CTA
finds its start by a search over the lengths and walks on by itself, and the
join kernel works out anew which CTAs hold a row's pieces and in which slots.
Checked here: every tile is taken once, a CTA writes a slot once, and the join
reads exactly the slots that were written, in the order of the keys."""
import numpy as np
import pytest

CHARGE = 2      # tiles that a unit costs by itself
CHUNKS = 8


def first_of(total, n, c):
    return total * c // n


def owner(total, n, t):
    return ((t + 1) * n - 1) // total


def start_of(charges, units, start):
    """(sequence, unit, offset) by the kernel's search: chunks of 32 whole sequences
    are passed, the last with at most `start` charged tiles before it is the one."""
    B, first, before, base = len(charges), start // units, 0, 0
    while True:
        for i in range(CHUNKS):
            c = charges[base + 32 * i:base + 32 * i + 32]
            if before + sum(c) <= first and base + 32 * (i + 1) < B:
                before += sum(c)
                continue
            inc = np.cumsum(c)
            here = [k for k in range(len(c)) if before + inc[k] - c[k] <= first]
            k = here[-1]
            off = start - (before + int(inc[k]) - c[k]) * units
            return base + 32 * i + k, off // c[k], off % c[k]
        base += 32 * CHUNKS


def run(tiles, units, ctas):
    charges = [t + CHARGE for t in tiles]
    total = sum(charges) * units
    n = min(ctas, total)
    written, taken = {}, {}
    for cta in range(n):
        start, end = first_of(total, n, cta), first_of(total, n, cta + 1)
        assert end > start
        b, unit, off = start_of(charges, units, start)
        left = end - start
        while left > 0:
            take = min(charges[b] - off, left)
            t0 = max(0, off - CHARGE)
            nt = max(0, off + take - CHARGE) - t0
            left -= take
            if nt:
                taken.setdefault((b, unit), []).append((t0, nt))
                if not (t0 == 0 and nt == tiles[b]):
                    slot = 2 * cta + (1 if t0 == 0 else 0)
                    assert slot not in written
                    written[slot] = (b, unit, t0, nt)
            off = 0
            unit += 1
            if unit == units:
                unit, b = 0, b + 1
    read = set()
    before = 0
    for b, t in enumerate(tiles):
        for unit in range(units):
            pieces = sorted(taken[(b, unit)])
            at = 0
            for t0, nt in pieces:
                assert t0 == at
                at += nt
            assert at == t
            base = before * units + unit * (t + CHARGE) + CHARGE
            c0, c1 = owner(total, n, base), owner(total, n, base + t - 1)
            assert (c0 == c1) == (len(pieces) == 1)
            if c0 != c1:
                got = [written[2 * c + (1 if c == c0 else 0)] for c in range(c0, c1 + 1)]
                assert [g[:2] for g in got] == [(b, unit)] * len(got)
                assert [g[2:] for g in got] == pieces
                read |= {2 * c + (1 if c == c0 else 0) for c in range(c0, c1 + 1)}
        before += t + CHARGE
    assert read == set(written)


@pytest.mark.parametrize("B,units,ctas", [(1, 1, 304), (1, 8, 304), (4, 8, 304), (33, 2, 304), (64, 8, 304),
                                          (257, 3, 304), (600, 1, 304), (5, 7, 13), (40, 16, 1)])
def test_every_tile_once_and_every_piece_joined(B, units, ctas):
    rng = np.random.default_rng(B * 1000 + units)
    for most in (1, 2, 9, 200, 3000):
        tiles = [int(x) for x in rng.integers(1, most + 1, B)]
        run(tiles, units, ctas)
        run([1] * (B - 1) + [most], units, ctas)
