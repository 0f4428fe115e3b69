"""The decode kernels' schedule in the kernel's own arithmetic: quotients by the
upper half of a product with ceil(2^64 / d), 32-bit ones where both numbers
fit, the search of a CTA's start for up to 32 sequences and for more, and the
join's sums over the lengths.  Each is compared with plain whole numbers, and
what tests/test_decode_schedule_model.py takes for granted (a unit's charge,
sequences per look-up) is read from the source."""
import re
from pathlib import Path

import numpy as np
import pytest

from tests import test_decode_schedule_model as model

CSRC = Path(__file__).resolve().parents[1] / "attention_forward_fa_gb300/csrc"
SOURCE = (CSRC / "fa_decode.cuh").read_text()
HOST = (CSRC / "fa_paged.cu").read_text()
M64 = 2 ** 64 - 1


def constant(name):
    return int(re.search(rf"constexpr int {name} = (\d+);", SOURCE)[1])


CHARGE, CHUNKS = constant("kUnitTiles"), constant("kChunks")


def test_the_models_follow_the_source():
    assert (model.CHARGE, model.CHUNKS) == (CHARGE, CHUNKS)
    assert "d == 1 ? 0ull : ~0ull / d + 1" in HOST
    assert "return inv ? (long long)__umul64hi((unsigned long long)a, inv) : a;" in SOURCE
    assert "return total <= p.ctas ? c : times_inverse(total * c, p.ctas_inv);" in SOURCE
    assert "return (int)quotient((t + 1) * n - 1, total);" in SOURCE


def inverse(d):
    return 0 if d == 1 else (M64 // d + 1) & M64


def times_inverse(a, inv):
    return (a * inv) >> 64 if inv else a


def quotient(a, b):
    return a // b if (a | b) >> 32 else (a & 0xFFFFFFFF) // (b & 0xFFFFFFFF)


@pytest.mark.parametrize("d", [1, 2, 3, 7, 8, 13, 48, 304, 305, 1000, 65535, 65537, 2 ** 20 - 3])
def test_quotients_by_inverses_are_exact(d):
    """While a * d < 2^64: at multiples of d, next to them, and at random."""
    rng = np.random.default_rng(d)
    most = M64 // d
    inv = inverse(d)
    for a in [0, 1, d - 1, d, d + 1, most - 1, most // d * d, most // d * d - 1] + [
            int(x) for s in (8, 20, 40, 60) for x in rng.integers(0, min(2 ** s, most), 2000)]:
        assert times_inverse(a, inv) == a // d and quotient(a, d) == a // d


def start_of(charges, units, start):
    """(sequence, unit, offset) of charged tile `start`, as the kernel finds it."""
    B, first = len(charges), times_inverse(start, inverse(units))
    if B <= 32:
        at, before, mine = 0, 0, charges + [0] * (32 - B)
    else:
        at, before, base = -1, 0, 0
        while at < 0:
            for i in range(CHUNKS):
                if at >= 0:
                    break
                c = charges[base + 32 * i:base + 32 * i + 32]
                c = c + [0] * (32 - len(c))
                if before + sum(c) > first or base + 32 * (i + 1) >= B:
                    at, mine = base + 32 * i, c
                else:
                    before += sum(c)
            base += 32 * CHUNKS
    inc = np.cumsum(mine)
    lane = max(k for k in range(32) if mine[k] > 0 and before + int(inc[k]) - mine[k] <= first)
    off = start - (before + int(inc[lane]) - mine[lane]) * units
    unit = quotient(off, mine[lane])
    return at + lane, unit, off - unit * mine[lane]


def join_sums(charges, block, warps, wpr, per_b):
    """(sequence, charges before it) per row of a join block, as its warps add them up."""
    B, out = len(charges), []
    total = per_b * B
    for w in range(warps):
        row = block * (warps // wpr) + w // wpr
        if row >= total:
            continue
        b = row // per_b
        if B <= 32 * CHUNKS:
            before = sum(charges[:b])
        else:
            b0 = block * (warps // wpr) // per_b
            before = sum(sum(charges[base + j] for j in range(32 * CHUNKS) if base + j < min(b0, B))
                         for v in range(warps) for base in range(32 * CHUNKS * v, B, 32 * CHUNKS * warps))
            assert b - b0 < 32
            before += sum(charges[b0 + lane] for lane in range(32) if b0 + lane < b)
        out.append((b, before))
    return out


@pytest.mark.parametrize("B,units", [(1, 1), (1, 8), (31, 3), (32, 8), (33, 8), (256, 2), (257, 1), (700, 5)])
@pytest.mark.parametrize("most", [1, 40, 2 ** 25])
def test_starts_and_joins(B, units, most):
    rng = np.random.default_rng(B * units)
    charges = [int(x) + CHARGE for x in rng.integers(1, most + 1, B)]
    total, ctas = sum(charges) * units, 304
    n = min(ctas, total)
    ends = np.cumsum([0] + charges)
    inv = inverse(ctas)
    for c in range(0, n, 1 if B < 300 else 13):
        start = c if total <= ctas else times_inverse(total * c, inv)
        assert start == (c if total <= ctas else total * c // ctas)
        b = int(np.searchsorted(ends * units, start, side="right")) - 1
        off = start - int(ends[b]) * units
        assert start_of(charges, units, start) == (b, off // charges[b], off % charges[b])
        assert quotient((start + 1) * n - 1, total) == c       # the owner of its first tile
        if start:
            assert quotient(start * n - 1, total) == c - 1
    for wpr, warps in ((1, 8), (8, 8), (32, 32)):
        for per_b in (1, 3, 40):
            rows = per_b * B
            blocks = -(-rows // (warps // wpr))
            for block in range(0, blocks, max(1, blocks // 40)):
                for b, before in join_sums(charges, block, warps, wpr, per_b):
                    assert before == int(ends[b])
