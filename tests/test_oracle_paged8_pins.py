"""Pins of the fp64 reference of the 8-bit cache and of drafting (oracle/paged.py):
closed forms, the other functions of the reference and torch's casts, no GPU."""
import numpy as np
import pytest
import torch

from oracle import fp8 as F
from oracle import paged as P

FMT = ["e4m3fn", "e5m2"]


@pytest.mark.parametrize("fmt", FMT)
def test_the_scale_is_the_least_that_holds_the_row(fmt):
    top = F.FORMATS[fmt][2]
    rng = np.random.default_rng(0)
    x = rng.standard_normal((500, 16)) * 2.0 ** rng.integers(-60, 60, (500, 1))
    e = P.exponent(x, fmt)
    a = np.abs(x).max(-1)
    assert (a <= top * 2.0 ** e).all() and (a > top * 2.0 ** (e - 1)).all()
    one = np.array([[top], [np.nextafter(top, np.inf)], [top / 2], [0.0], [1e-40], [top * 2.0 ** -80]])
    assert P.exponent(one, fmt).tolist() == [0, 1, -1, -80, -80, -80]


@pytest.mark.parametrize("fmt", FMT)
def test_codes_are_the_casts_of_torch(fmt):
    rng = np.random.default_rng(1)
    x = rng.standard_normal((300, 64)).astype(np.float32) * (2.0 ** rng.integers(-20, 20, (300, 1))).astype(np.float32)
    codes, e = P.quantise(x.astype(np.float64), fmt)
    t = torch.ldexp(torch.from_numpy(x), -torch.from_numpy(e)[:, None].int())
    cast = t.to(torch.float8_e4m3fn if fmt == "e4m3fn" else torch.float8_e5m2)
    assert np.array_equal(cast.double().numpy(), codes)
    assert (np.abs(codes).max(-1) > F.FORMATS[fmt][2] / 2 * 0.9).all()
    err = np.abs(np.ldexp(codes, e[:, None]) - x)
    half = {"e4m3fn": (2.0 ** -4, 2.0 ** -10), "e5m2": (2.0 ** -3, 2.0 ** -17)}[fmt]
    assert (err <= np.maximum(half[0] * np.abs(x), half[1] * 2.0 ** e[:, None])).all()


def _pool(rng, B, H, page, per, D):
    num = B * per + 2
    table = rng.permutation(num)[:B * per].reshape(B, per).astype(np.int32)
    return rng.standard_normal((num, H, page, D)), rng.standard_normal((num, H, page, D)), table


def test_a_chain_is_the_newest_tokens():
    """A tree in which every draft sees those before it and itself."""
    rng = np.random.default_rng(2)
    k, v, table = _pool(rng, 2, 2, 16, 4, 8)
    q = rng.standard_normal((2, 4, 5, 8))
    chain = np.tril(np.ones((5, 5), dtype=bool))[None].repeat(2, 0)
    a = P.decode(q, k, v, table, [50, 5], 0.3)
    b = P.decode(q, k, v, table, [50, 5], 0.3, tree=(chain, [5, 5]))
    assert all(np.array_equal(x, y) for x, y in zip(a, b))


def test_a_branch_is_the_sequence_it_spells():
    """Row i of a tree answers as the last token of a text without the other branches."""
    rng = np.random.default_rng(3)
    k, v, table = _pool(rng, 1, 1, 16, 3, 8)
    parent = [-1, 0, 0, 1, -1, 2, 4]
    anc = np.zeros((1, 7, 7), dtype=bool)
    for i, p in enumerate(parent):
        anc[0, i] = anc[0, p] if p >= 0 else False
        anc[0, i, i] = True
    n = 30
    q = rng.standard_normal((1, 1, 7, 8))
    O, L, *_ = P.decode(q, k, v, table, [n], 0.4, tree=(anc, [7]))
    for i in range(7):
        path = np.flatnonzero(anc[0, i])
        (k2, v2), _, _ = P.keep([k, v], table, [n - 7], path[None], [len(path)], 16)
        o, l, *_ = P.decode(q[:, :, i:i + 1], k2, v2, table, [n - 7 + len(path)], 0.4)
        assert np.allclose(O[0, 0, i], o[0, 0, 0], atol=1e-13) and np.allclose(L[0, 0, i], l[0, 0, 0], atol=1e-13)
    # padding rows see the tokens before the drafts, and a row that sees nothing is empty
    O, L, *_ = P.decode(q, k, v, table, [n], 0.4, tree=(anc, [3]))
    o, l, *_ = P.decode(q[:, :, 5:6], k, v, table, [n - 3], 0.4)
    assert np.allclose(O[0, 0, 5], o[0, 0, 0], atol=1e-13)
    O, L, *_ = P.decode(q, k, v, table, [7], 0.4, tree=(np.zeros_like(anc), [7]))
    assert (O == 0).all() and np.isposinf(L).all()


def test_reading_and_keeping():
    rng = np.random.default_rng(4)
    k, v, table = _pool(rng, 2, 3, 16, 4, 8)
    ko, vo = rng.standard_normal((2, 2, 3, 40, 8))
    a, b = P.read(k, v, table, [5, 0], [40, 17], ko, vo)
    flat = k[table[0]].transpose(1, 0, 2, 3).reshape(3, 64, 8)
    assert np.array_equal(a[0], flat[:, 5:45]) and np.array_equal(b[1, :, 17:], vo[1, :, 17:])
    lo, hi = k.min(2), k.max(2)
    idx = np.array([[1, 2, 9], [0, 1, -1]])
    (k2, v2), lo2, hi2 = P.keep([k, v], table, [15, 20], idx, [3, 2], 16, k, lo, hi)
    f2 = k2[table[0]].transpose(1, 0, 2, 3).reshape(3, 64, 8)
    assert np.array_equal(f2[:, 15:18], flat[:, [16, 17, 24]]) and np.array_equal(f2[:, :15], flat[:, :15])
    assert np.array_equal(f2[:, 18:], flat[:, 18:])
    p0, p1 = table[0, 0], table[0, 1]
    assert np.array_equal(lo2[p0], np.minimum(lo[p0], flat[:, 16]))            # widened
    assert np.array_equal(hi2[p1], np.maximum(flat[:, 17], flat[:, 24]))       # slot 0 moved into: anew
    others = [p for p in range(k.shape[0]) if p not in (p0, p1)]
    assert np.array_equal(k2[others], k[others]) and np.array_equal(lo2[others], lo[others])


def test_turning_by_given_positions():
    rng = np.random.default_rng(5)
    k, v, table = _pool(rng, 1, 1, 16, 2, 16)
    a = np.arange(40)[:, None] * 10000.0 ** (-np.arange(0, 16, 2) / 16)
    x = rng.standard_normal((1, 1, 3, 16))
    kp = P.append(k, v, table, [4], x, x, [3], np.cos(a), np.sin(a), positions=np.array([[9, 9, 30]]))[0]
    want = P.rotate(x[0], np.array([9, 9, 30]), np.cos(a), np.sin(a), False)
    assert np.allclose(kp[table[0, 0], :, 4:7], want)
