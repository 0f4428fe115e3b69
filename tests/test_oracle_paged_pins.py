"""Pins of the fp64 reference of the paged operators (oracle/paged.py): closed
forms and the dense reference, no GPU."""
import numpy as np
import pytest

from oracle import attention as A
from oracle import paged as P


def _tables(n, r):
    a = np.arange(n)[:, None] * 10000.0 ** (-np.arange(0, r, 2) / r)
    return np.cos(a), np.sin(a)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_keeps_lengths_and_depends_on_distance(interleaved):
    rng = np.random.default_rng(0)
    cos, sin = _tables(200, 32)
    x, y = rng.standard_normal((2, 1, 64))
    rx = P.rotate(x, np.array([7]), cos, sin, interleaved)
    assert np.allclose((rx ** 2).sum(), (x ** 2).sum(), rtol=1e-14)
    assert np.array_equal(rx[:, 32:], x[:, 32:])            # channels past the rotated ones
    d = [float((P.rotate(x, np.array([t]), cos, sin, interleaved)
                * P.rotate(y, np.array([t + 13]), cos, sin, interleaved)).sum()) for t in (0, 50, 180)]
    assert np.allclose(d, d[0], rtol=1e-12)
    a, b = (0, 1) if interleaved else (0, 16)               # the fastest pair turns by one radian a step
    assert np.allclose(P.rotate(x, np.array([1]), cos, sin, interleaved)[0, a],
                       x[0, a] * np.cos(1) - x[0, b] * np.sin(1))


def _scatter(k, v, page, num, rng):
    B, H, S, D = k.shape
    per = -(-S // page)
    table = rng.permutation(num)[:B * per].reshape(B, per).astype(np.int32)
    kp, vp = np.full((2, num, H, page, D), np.nan)
    for b in range(B):
        for t in range(S):
            kp[table[b, t // page], :, t % page] = k[b, :, t]
            vp[table[b, t // page], :, t % page] = v[b, :, t]
    return kp, vp, table


def test_decode_over_all_pages_is_the_dense_reference():
    rng = np.random.default_rng(1)
    B, Hq, Hkv, S, D, Sq = 2, 4, 2, 37, 8, 3
    k, v = rng.standard_normal((2, B, Hkv, S, D))
    q = rng.standard_normal((B, Hq, S, D))
    kp, vp, table = _scatter(k, v, 16, 9, rng)
    O, L, _, _, _ = P.decode(q[:, :, S - Sq:], kp, vp, table, [S, S], 0.3)
    for b in range(B):
        for h in range(Hq):
            Od, Ld = A.attention_fwd(q[b:b + 1, h:h + 1], k[b:b + 1, h // 2:h // 2 + 1],
                                     v[b:b + 1, h // 2:h // 2 + 1], 0.3, mask=1)[:2]
            assert np.allclose(O[b, h], Od[0, 0, S - Sq:], atol=1e-12)
            assert np.allclose(L[b, h], Ld[0, 0, S - Sq:], atol=1e-12)


def test_decode_limits():
    rng = np.random.default_rng(2)
    k, v = rng.standard_normal((2, 1, 1, 40, 8))
    q = rng.standard_normal((1, 1, 2, 8))
    kp, vp, table = _scatter(k, v, 16, 5, rng)
    O, L, _, _, _ = P.decode(q, kp, vp, table, [1], 1.0)         # row 0 lies before the first token
    assert np.all(O[0, 0, 0] == 0) and np.isposinf(L[0, 0, 0])
    assert np.allclose(O[0, 0, 1], v[0, 0, 0])                # a single key
    O, L, _, _, _ = P.decode(q, kp, vp, table, [0], 1.0)
    assert np.all(O == 0) and np.isposinf(L).all()
    O, _, _, _, _ = P.decode(q, kp, vp, table, [40], 1.0, pre_tokens=0)
    assert np.allclose(O[0, 0], v[0, 0, 38:40])               # each row sees itself alone
    O, _, _, _, _ = P.decode(0 * q, kp, vp, table, [40], 1.0, page_idx=np.array([[[1, -1, 1, 9]]]))
    assert np.allclose(O[0, 0, 0], v[0, 0, 16:32].mean(0))    # listed twice, invalid slots
    O, _, _, _, _ = P.decode(0 * q, kp, vp, table, [40], 1.0, page_idx=np.array([[[1, -1, 9, 0]]]))
    assert np.allclose(O[0, 0, 0], v[0, 0, 16:32].mean(0))    # three pages: the fourth entry is not read


def test_append_then_decode_and_bounds():
    rng = np.random.default_rng(3)
    cos, sin = _tables(64, 16)
    k, v = rng.standard_normal((2, 1, 2, 20, 16))
    kp = np.full((4, 2, 16, 16), np.nan)
    lo, hi = np.full((4, 2, 16), np.nan), np.full((4, 2, 16), np.nan)
    table = np.array([[2, 0, 3]], dtype=np.int32)
    kp2, vp2, lo, hi = P.append(kp, kp, table, [0], k[:, :, :7], v[:, :, :7], [7], cos, sin, k_min=lo, k_max=hi)
    kp2, vp2, lo, hi = P.append(kp2, vp2, table, [7], k[:, :, 7:], v[:, :, 7:], [13], cos, sin, k_min=lo, k_max=hi)
    kr = P.rotate(k[0], np.arange(20), cos, sin, False)
    assert np.allclose(kp2[2], kr[:, :16]) and np.allclose(kp2[0][:, :4], kr[:, 16:])
    assert np.isnan(kp2[0][:, 4:]).all() and np.isnan(kp2[[1, 3]]).all()
    assert np.allclose(lo[2], kr[:, :16].min(1)) and np.allclose(hi[0], kr[:, 16:].max(1))
    assert np.allclose(vp2[0][:, :4], v[0, :, 16:])


def test_scores_bound_every_key_of_the_page():
    rng = np.random.default_rng(4)
    k = rng.standard_normal((6, 1, 16, 8))
    q = rng.standard_normal((1, 2, 1, 8))
    table = rng.permutation(6)[None].astype(np.int32)
    lo, hi = k.min(2), k.max(2)
    got = P.select(q, lo, hi, table, [96], 16, 3, first=1, last=1)[0, 0]
    assert list(got) == sorted(set(got)) and 0 in got and 5 in got
    bound = np.stack([np.maximum(q[0, g, 0] * lo[:, 0], q[0, g, 0] * hi[:, 0]).sum(-1) for g in range(2)]).max(0)
    assert (bound >= np.stack([(k[:, 0] @ q[0, g, 0]).max(-1) for g in range(2)]).max(0)).all()
    third = [p for p in got if p not in (0, 5)][0]
    assert bound[table[0, third]] == bound[table[0, 1:5]].max()
    assert list(P.select(q, lo * 0, hi * 0, table, [96], 16, 4)[0, 0]) == [0, 1, 2, 5]   # ties: lower page
    assert list(P.select(q, lo, hi, table, [17], 16, 4)[0, 0]) == [0, 1, -1, -1]
    assert list(P.select(q, lo, hi, table, [0], 16, 4)[0, 0]) == [-1] * 4
