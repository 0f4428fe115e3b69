"""GPU parity of the 8-bit cache and of drafting over a paged cache (fa_kv_append_ext,
fa_decode_ext, fa_kv_read, fa_kv_keep) against the fp64 reference of oracle/paged.py.

Bounds, with u the type's half step (2^-8 bf16, 2^-11 fp16) and c the format's (2^-4
e4m3, 2^-3 e5m2; of its subnormals 2^-10 and 2^-17 in units of a row's scale):
  * a rotated channel x is off by r = 3 2^-24 (|a cos| + |b sin|) in fp32, so
    that a stored key is within max(c |x|, subnormal half step 2^e) + (1 + c) r of it (and
    a row's scale is that of its largest channel as computed, up to r of it);
  * a score is an fp32 sum of D <= 128 exact products: its error is at most
    e_s = 2^-16 X with X = max_j scale sum_d |q_d k_jd|; the key's scale and the
    value's exponent E are put on it with two fp32 roundings of X + |E| each;
  * a probability is off by the error of its score, of the subtraction of the
    reference (2^-22 of what is subtracted) and the exponential (2^-16 with all that is
    relative); it enters as one fp16, 2^-11 of it, or, of small ones, 2^-25 where
    the largest weight of a code, 2^(s + e) at most, is at least 2^7.  So
    |O - ref| <= (2 e_s + 2^-20 (X + E) + 2^-15 + 2^-11) A + 2^-32 W + (u + 2^-20) |ref|
    with A = sum_j p_j |v_j|, W = max_j(p_j 2^e_j) sum_j |code_j|;
  * |LSE - ref| <= e_s + 2^-21 (X + E) + 2^-20 (1 + |ref| + E).
Bounds over a 16-bit cache are those of tests/test_gpu_paged.py.  Whole numbers, moved
rows and untouched memory are equal bit for bit."""
import math

import numpy as np
import pytest

from oracle import fp8 as F
from oracle import paged as P
from tests.test_gpu_paged import SUB, U, Cache, _check, _dev, _host, _round, _status, _tables, _torch_type

pytestmark = pytest.mark.gpu

HALF = {"e4m3fn": (2.0 ** -4, 2.0 ** -10), "e5m2": (2.0 ** -3, 2.0 ** -17)}


@pytest.fixture(scope="module", autouse=True)
def built():
    from attention_forward_fa_gb300 import build
    build.build()


def _codes(x, fmt):
    """float64 codes as a float8 tensor on the GPU."""
    import torch
    return torch.from_numpy(np.ascontiguousarray(x)).float().to(torch.float8_e4m3fn if fmt == "e4m3fn" else torch.float8_e5m2).cuda()


class Cache8:
    """A random 8-bit cache on both sides: codes, exponents and values (pages in random order)."""

    def __init__(self, seed, dtype, fmt, B, Hkv, D, page, cap, layout="hnd", spare=3, bounds=False, stale=False,
                 spread=0.0):
        import torch
        import attention_forward_fa_gb300 as fa
        self.rng = rng = np.random.default_rng(seed)
        self.dtype, self.fmt, self.B, self.Hkv, self.D, self.page = dtype, fmt, B, Hkv, D, page
        need = [-(-c // page) for c in cap]
        num = sum(need) + spare
        order = rng.permutation(num)
        self.table = np.full((B, max(max(need), 1)), -1, dtype=np.int32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = order[at:at + n]
            at += n
        shape = (num, Hkv, page, D)
        size = lambda: 2.0 ** (spread * rng.standard_normal(shape[:3])).round()[..., None] if spread else 1.0
        (self.kc, self.ke), (self.vc, self.ve) = (P.quantise(rng.standard_normal(shape) * s, fmt) for s in (1.0, size()))
        self.k, self.v = np.ldexp(self.kc, self.ke[..., None]), np.ldexp(self.vc, self.ve[..., None])
        tk, tv = _codes(self.kc, fmt).view(torch.uint8), _codes(self.vc, fmt).view(torch.uint8)
        sk, sv = (_dev((e + 127).astype(np.uint8)) for e in (self.ke, self.ve))
        if stale:                     # what no sequence sees: NaN codes, scales of 2^128 (NaN) and 2^-127
            unseen = np.ones(shape[:3], dtype=bool)
            for b in range(B):
                for t in range(cap[b]):
                    unseen[self.table[b, t // page], :, t % page] = False
            m = torch.from_numpy(unseen).cuda()
            tk[m], tv[m] = 0x7F, 0xFF
            sk[m], sv[m] = 255, 0
            sv[m.logical_and(torch.rand(m.shape, device="cuda") < 0.5)] = 255
        if layout == "nhd":           # [num, page, Hkv, D] pools
            tk, tv = (t.transpose(1, 2).contiguous().transpose(1, 2) for t in (tk, tv))
        elif layout == "halves":      # K and V of a page side by side in one pool, rows padded by 16
            both = torch.zeros(num, 2, Hkv, page, D + 16, dtype=tk.dtype, device="cuda")
            both[:, 0, ..., :D], both[:, 1, ..., :D] = tk, tv
            tk, tv = both[:, 0, ..., :D], both[:, 1, ..., :D]
        self.bk, self.bv, self.sk, self.sv = tk, tv, sk, sv
        kind = torch.float8_e4m3fn if fmt == "e4m3fn" else torch.float8_e5m2
        self.lo = self.hi = self.tlo = self.thi = None
        if bounds:
            self.lo, self.hi = _round(self.k.min(2), dtype), _round(self.k.max(2), dtype)
            self.tlo, self.thi = _dev(self.lo, dtype), _dev(self.hi, dtype)
        self.obj = fa.PagedKV(tk.view(kind), tv.view(kind), _dev(self.table), self.tlo, self.thi, k_scale=sk, v_scale=sv,
                              dtype=_torch_type(dtype))

    def ints(self, x):
        return _dev(np.asarray(x, dtype=np.int32))

    def stored(self):
        """(k codes, k exponents, v codes, v exponents) on the device now, on the host."""
        import torch
        kind = torch.float8_e4m3fn if self.fmt == "e4m3fn" else torch.float8_e5m2
        got = []
        for t, s in ((self.bk, self.sk), (self.bv, self.sv)):
            got += [t.contiguous().view(kind).double().cpu().numpy(), s.cpu().numpy().astype(np.int64) - 127]
        return got

    def values(self):
        kc, ke, vc, ve = self.stored()
        with np.errstate(invalid="ignore", over="ignore"):
            return np.ldexp(kc, ke[..., None]), np.ldexp(vc, ve[..., None])


def _spread(c, q, table, lens, scale, tree=None, pre=None, idx=None):
    """W and E of the bound: per output max_j(p_j 2^e_j) sum_j |code_j|, and the largest |e| of a value seen."""
    B, Hq, Sq, D = q.shape
    O1, L, A, X, V = P.decode(q, c.k, np.broadcast_to(np.exp2(c.ve.astype(float))[..., None], c.v.shape), table, lens, scale, pre, idx, tree)
    # sum_j p_j 2^e_j is at least the largest term: an upper bound of it
    W1 = O1[..., :1]
    C = P.decode(q, c.k, c.vc, table, lens, scale, pre, idx, tree)[4]
    return W1 * C, float(np.abs(c.ve).max())


def _check8(got_o, got_l, ref, W, E, dtype, where=""):
    O, L, A, X, V = ref
    o, l = _host(got_o), _host(got_l)
    u = U[dtype]
    empty = np.isposinf(L)
    assert np.array_equal(np.isposinf(l), empty), f"{where}: rows without keys"
    assert (o[empty] == 0).all()
    es = 2.0 ** -16 * X
    lim = (2 * es + 2.0 ** -20 * (X + E) + 2.0 ** -15 + 2.0 ** -11)[..., None] * A + 2.0 ** -32 * W
    lim += (u + 2.0 ** -20) * np.abs(O) + SUB[dtype]
    err = np.abs(o - O)
    assert (err <= lim).all(), f"{where}: O off by {(err / np.maximum(lim, 1e-30)).max():.3g} of its bound"
    le = np.abs(l[~empty] - L[~empty])
    ll = (es + 2.0 ** -21 * (X + E))[~empty] + 2.0 ** -20 * (1 + np.abs(L[~empty]) + E)
    assert (le <= ll).all(), f"{where}: LSE off by {(le / ll).max():.3g} of its bound"


def _trees(rng, B, S, wide=4):
    """Random trees bool [B, S, S] (itself seen) and depths [B, S]."""
    anc = np.zeros((B, S, S), dtype=bool)
    for b in range(B):
        for i in range(S):
            p = i - 1 - int(rng.integers(wide))
            if p >= 0:
                anc[b, i] = anc[b, p]
            anc[b, i, i] = True
    return anc, anc.sum(-1).astype(np.int32) - 1


# ------------------------------------------------------------------ append
APPEND = [
    # dtype, fmt, B, Hq, Hkv, D, page, S, old, new, rot, interleaved, layout, given positions
    ("bf16", "e4m3fn", 1, 4, 1, 128, 64, 1, [0], [1], 128, False, "hnd", False),
    ("bf16", "e4m3fn", 3, 32, 8, 128, 64, 1, [63, 64, 517], [1, 1, 1], 128, False, "nhd", True),
    ("fp16", "e5m2", 5, 6, 6, 64, 16, 1, [0, 15, 16, 17, 300], [1, 0, 1, 1, 1], 32, True, "halves", False),
    ("bf16", "e5m2", 2, 8, 2, 64, 32, 2, [31, 5], [2, 1], 64, True, "hnd", True),
    ("fp16", "e4m3fn", 3, 40, 5, 128, 16, 37, [0, 3, 15], [37, 20, 0], 64, False, "nhd", True),
    ("bf16", "e4m3fn", 2, 3, 3, 128, 256, 300, [250, 0], [300, 257], 128, True, "hnd", False),
    ("bf16", "e5m2", 2, 16, 16, 64, 128, 129, [100, 127], [129, 65], 0, False, "halves", True),
    ("fp16", "e4m3fn", 1, 33, 1, 64, 64, 70, [7], [70], 16, False, "hnd", False),
    ("bf16", "e4m3fn", 1, 72, 9, 128, 32, 3, [30], [3], 112, True, "nhd", True),
    # much room, few tokens: a block looks for its pieces
    ("bf16", "e4m3fn", 16, 1, 1, 64, 16, 4096, [5, 0] + [100] * 14, [900, 0, 4096, 33] + [1] * 12, 64, False, "hnd", False),
    ("fp16", "e5m2", 26, 1, 1, 128, 16, 2048, [15] * 25 + [0], [2, 2048] + [1, 0] * 12, 32, True, "nhd", True),
]


def _turned(x, old, new, rot, inter, cos, sin, pos):
    """(x rotated in 64 bits, |a cos| + |b sin|) of the tokens of each sequence."""
    y, mag = np.array(x), np.zeros_like(x)
    if rot:
        ia = np.arange(0, rot, 2) if inter else np.arange(rot // 2)
        ib = ia + (1 if inter else rot // 2)
        for b in range(x.shape[0]):
            p = pos[b, :new[b]] if pos is not None else old[b] + np.arange(new[b])
            y[b][:, :new[b]] = P.rotate(x[b][:, :new[b]], p, cos, sin, inter)
            cc, ss = np.abs(cos[p]).astype(float), np.abs(sin[p]).astype(float)
            a, d = np.abs(x[b][:, :new[b]][..., ia]), np.abs(x[b][:, :new[b]][..., ib])
            m = np.zeros_like(x[b][:, :new[b]])
            m[..., ia], m[..., ib] = a * cc + d * ss, a * ss + d * cc
            mag[b][:, :new[b]] = m
    return y, mag


@pytest.mark.parametrize("case", APPEND, ids=lambda c: "-".join(map(str, c[:8])))
@pytest.mark.parametrize("form", ["plain", "fused_in_place"])
def test_append8(case, form):
    import attention_forward_fa_gb300 as fa
    dtype, fmt, B, Hq, Hkv, D, page, S, old, new, rot, inter, layout, placed = case
    c = Cache8(1, dtype, fmt, B, Hkv, D, page, [o + n for o, n in zip(old, new)], layout, bounds=True)
    rng = c.rng
    q, k, v = (_round(rng.standard_normal((B, h, S, D)), dtype) for h in (Hq, Hkv, Hkv))
    most = max(o + n for o, n in zip(old, new)) + 1
    cos, sin = _tables(most, rot) if rot else (None, None)
    kw = dict(cos=_dev(cos), sin=_dev(sin)) if rot else {}
    pos = rng.integers(0, most, (B, S)).astype(np.int32) if placed else None
    if placed:
        for b in range(B):
            pos[b, new[b]:] = -7         # padding: not read
        kw["positions"] = _dev(pos)
    if form == "plain":
        tq, tk, tv = _dev(q, dtype), _dev(k, dtype), _dev(v, dtype)
        mark = _round(rng.standard_normal(q.shape), dtype)
        qo = _dev(mark, dtype)
    else:
        x = _dev(np.concatenate((q, k, v), 1), dtype).transpose(1, 2).contiguous().transpose(1, 2)
        tq, tk, tv = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
        mark, qo = q, tq
    was = c.stored()
    got = fa.paged_kv_append(c.obj, c.ints(old), tk, tv, new_lens=c.ints(new), q=tq, q_out=qo, interleaved=inter, **kw)
    assert got is qo and _status() == 0
    kc, ke, vc, ve = c.stored()
    ek, mk = _turned(k, old, new, rot, inter, cos, sin, pos)
    zeros = np.zeros_like(c.k)
    full = lambda x: P.append(zeros, zeros, c.table, old, x, x, new)[0]
    ek, mk, ev = full(ek), full(mk), full(v)
    wrote = np.zeros(c.k.shape[:3], dtype=bool)
    for b in range(B):
        for t in range(old[b], old[b] + new[b]):
            wrote[c.table[b, t // page], :, t % page] = True
    for a, b in zip(was, (kc, ke, vc, ve)):
        assert np.array_equal(a[~wrote], b[~wrote])
    # values: the very codes and scales of the reference
    rc, re = P.quantise(ev[wrote], fmt)
    assert np.array_equal(vc[wrote], rc) and np.array_equal(ve[wrote], re)
    # keys: within half a code of the rotated key, by a scale that its largest channel needs
    r = 3 * 2.0 ** -24 * mk[wrote]
    x, half = ek[wrote], HALF[fmt]
    top = np.abs(x).max(-1) * (1 + 2.0 ** -22) + r.max(-1), np.abs(x).max(-1) * (1 - 2.0 ** -22) - r.max(-1)
    e = ke[wrote]
    assert (e <= P.exponent(top[0][:, None], fmt)).all() and (e >= P.exponent(np.maximum(top[1], 0)[:, None], fmt)).all()
    err = np.abs(np.ldexp(kc[wrote], e[:, None]) - x)
    assert (err <= np.maximum(half[0] * np.abs(x), half[1] * 2.0 ** e[:, None]) + (1 + half[0]) * r).all()
    # queries as with a 16-bit cache
    eq, mq = _turned(q, old, new, rot, inter, cos, sin, pos)
    gq, u = _host(qo), U[dtype]
    for b in range(B):
        n = new[b]
        lim = u * np.abs(eq[b][:, :n]) + (1 + u) * 3 * 2.0 ** -24 * mq[b][:, :n] + SUB[dtype]
        assert (np.abs(gq[b][:, :n] - eq[b][:, :n]) <= (lim if rot else 0)).all()
        assert np.array_equal(gq[b][:, n:], mark[b][:, n:])
    # bounds of the touched pages: those of the keys as stored (of fp16 next below and above)
    gk = np.ldexp(kc, ke[..., None])
    lo, hi = c.lo.copy(), c.hi.copy()
    for b in range(B):
        for p in range(old[b] // page, -(-(old[b] + new[b]) // page)):
            a, z = max(old[b], p * page) - p * page, min(old[b] + new[b], (p + 1) * page) - p * page
            if z > a:
                i = c.table[b, p]
                l, h = gk[i, :, a:z].min(1), gk[i, :, a:z].max(1)
                lo[i], hi[i] = (l, h) if a == 0 else (np.minimum(l, lo[i]), np.maximum(h, hi[i]))
    gl, gh = _host(c.tlo), _host(c.thi)
    if dtype == "bf16":
        assert np.array_equal(gl, lo) and np.array_equal(gh, hi)
    else:
        assert (gl <= lo).all() and (gh >= hi).all()
        step = np.maximum(2.0 ** -10 * np.abs(lo), 2.0 ** -24), np.maximum(2.0 ** -10 * np.abs(hi), 2.0 ** -24)
        assert (lo - gl < step[0]).all() and (gh - hi < step[1]).all()


@pytest.mark.parametrize("fmt", ["e4m3fn", "e5m2"])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_append8_scales_and_codes_at_their_borders(dtype, fmt):
    """Rows whose largest channel is at, next above and below 1.75 * 2^x; zeros; the
    least and largest rows; channels half way between two codes."""
    import attention_forward_fa_gb300 as fa
    rng = np.random.default_rng(2)
    D, rows = 64, []
    for x in (-14, -3, 0, 7):
        for top in (1.75, 1.75 + 2.0 ** (-7 if dtype == "bf16" else -10), 1.75 - 2.0 ** (-7 if dtype == "bf16" else -10), 1.0):
            r = _round(rng.uniform(-1, 1, D) * 2.0 ** (x - rng.integers(0, 12, D)), dtype)
            r[3] = top * 2.0 ** x * (-1) ** len(rows)
            rows.append(r)
    ties = np.arange(D) % 16 + 0.5 + 16          # halves between codes of 4 bits, and of 3
    rows += [ties, -2 * ties, np.zeros(D), np.full(D, 2.0 ** -24), -np.full(D, 2.0 ** -14)]
    if dtype == "bf16":
        rows += [np.full(D, 2.0 ** -100), np.full(D, 2.0 ** -133), np.full(D, 1.75 * 2.0 ** 127), -np.full(D, (2 - 2.0 ** -7) * 2.0 ** 127),
                 np.full(D, 2.0 ** -80) * np.arange(D)]
    else:
        rows += [np.full(D, 65504.0), np.arange(D) * 2.0 ** -24]
    x = np.array(rows)[None, None]
    assert np.array_equal(_round(x, dtype), x)
    n = x.shape[2]
    c = Cache8(3, dtype, fmt, 1, 1, D, 16, [n])
    fa.paged_kv_append(c.obj, c.ints([0]), _dev(x, dtype), _dev(-x, dtype))
    assert _status() == 0
    kc, ke, vc, ve = c.stored()
    for t in range(n):
        p, s = c.table[0, t // 16], t % 16
        for sign, codes, e in ((1, kc, ke), (-1, vc, ve)):
            rc, re = P.quantise(sign * x[0, 0, t], fmt)
            assert np.array_equal(codes[p, 0, s], rc) and e[p, 0, s] == re, (t, sign)


def test_append8_rows_that_are_not_finite():
    """Such a row becomes NaN, the others are as they would be, the status says so."""
    import torch
    import attention_forward_fa_gb300 as fa
    for bad in (math.inf, -math.inf, math.nan):
        c = Cache8(4, "bf16", "e4m3fn", 1, 2, 128, 16, [40], bounds=True)
        x = _round(c.rng.standard_normal((1, 2, 40, 128)), "bf16")
        y = x.copy()
        x[0, 1, 17, 100], y[0, 0, 3, 5] = bad, bad
        fa.paged_kv_append(c.obj, c.ints([0]), _dev(x, "bf16"), _dev(y, "bf16"))
        assert _status() == fa.FA_ERR_RANGE and _status() == 0
        kc, ke, vc, ve = c.stored()
        p, s = c.table[0, 1], 1
        assert ke[p, 1, s] == 128 and (kc[p, 1, s] == 0).all() and ve[c.table[0, 0], 0, 3] == 128
        out = fa.paged_kv_read(c.obj, c.ints([40]), size=40)
        k, v = (_host(t) for t in out)
        assert np.isnan(k[0, 1, 17]).all() and np.isnan(v[0, 0, 3]).all()
        k[0, 1, 17], v[0, 0, 3] = 0, 0
        assert np.isfinite(k).all() and np.isfinite(v).all()
        assert bool(torch.isfinite(c.tlo).all()) and bool(torch.isfinite(c.thi).all())
        assert (np.abs(k - np.where(np.isfinite(x), x, 0))[0, 0] <= np.maximum(2.0 ** -4 * np.abs(x), 2.0 ** -10 * 2.0 ** -6)[0, 0]).all()


def test_append_at_given_positions():
    """A 16-bit cache: the same rows turned by positions as by their places, and a
    position without a row left out."""
    import torch
    import attention_forward_fa_gb300 as fa
    for dtype, D, inter in (("bf16", 128, False), ("fp16", 64, True)):
        a, b = (Cache(5, dtype, 3, 2, D, 16, [60] * 3, bounds=True) for _ in range(2))
        x = _dev(_round(a.rng.standard_normal((3, 8, 20, D)), dtype), dtype)
        cos, sin = (_dev(t) for t in _tables(64, D))
        old, new = a.ints([0, 7, 31]), a.ints([20, 11, 0])
        kw = dict(new_lens=new, cos=cos, sin=sin, interleaved=inter)
        qa = fa.paged_kv_append(a.obj, old, x[:, 4:6], x[:, 6:], q=x[:, :4], q_out=torch.zeros_like(x[:, :4]), **kw)
        pos = (old[:, None] + torch.arange(20, device="cuda", dtype=torch.int32)).contiguous()
        qb = fa.paged_kv_append(b.obj, old, x[:, 4:6], x[:, 6:], q=x[:, :4], q_out=torch.zeros_like(x[:, :4]), positions=pos, **kw)
        assert _status() == 0
        for s, t in ((qa, qb), (a.tk, b.tk), (a.tv, b.tv), (a.tlo, b.tlo), (a.thi, b.thi)):
            assert torch.equal(s, t)
        pos[:, 1] = pos[:, 0]            # two drafts of one depth
        pos[1, 3], pos[0, 5] = 64, -1
        was = b.tk.clone(), b.tv.clone()
        q = torch.zeros_like(x[:, :4])
        fa.paged_kv_append(b.obj, old, x[:, 4:6] + 1, x[:, 6:] + 1, q=x[:, :4], q_out=q, positions=pos, **kw)
        assert _status() == fa.FA_ERR_INDEX and _status() == 0
        for seq, i in ((1, 3), (0, 5)):
            t = int(old[seq]) + i
            p = b.table[seq, t // 16]
            assert torch.equal(b.tk[p, :, t % 16], was[0][p, :, t % 16]) and torch.equal(b.tv[p, :, t % 16], was[1][p, :, t % 16])
            assert bool((q[seq, :, i] == 0).all()) and bool((q[seq, :, i + 1] != 0).any())


def test_append_at_given_positions_of_more_pieces_than_blocks():
    """Room for more pieces than blocks: a block looks for its pieces; the same bits as without positions."""
    import torch
    import attention_forward_fa_gb300 as fa
    B, S, D = 26, 2048, 128
    old, new = [15] * 25 + [0], [2, 2048] + [1, 0] * 12
    a, b = (Cache(32, "bf16", B, 1, D, 16, [o + n for o, n in zip(old, new)], bounds=True) for _ in range(2))
    x = _dev(_round(a.rng.standard_normal((B, 3, S, D)), "bf16"), "bf16")
    cos, sin = (_dev(t) for t in _tables(2100, D))
    to, tn = a.ints(old), a.ints(new)
    kw = dict(new_lens=tn, cos=cos, sin=sin)
    qa = fa.paged_kv_append(a.obj, to, x[:, 1:2], x[:, 2:], q=x[:, :1], q_out=torch.zeros_like(x[:, :1]), **kw)
    pos = (to[:, None] + torch.arange(S, device="cuda", dtype=torch.int32)).contiguous()
    qb = fa.paged_kv_append(b.obj, to, x[:, 1:2], x[:, 2:], q=x[:, :1], q_out=torch.zeros_like(x[:, :1]), positions=pos, **kw)
    assert _status() == 0
    for s, t in ((qa, qb), (a.tk, b.tk), (a.tv, b.tv), (a.tlo, b.tlo), (a.thi, b.thi)):
        assert torch.equal(s, t)


# ------------------------------------------------------------------ decode
DECODE = [
    # dtype, fmt, B, Hq, Hkv, D, page, Sq, lens, pre, layout
    ("bf16", "e4m3fn", 1, 1, 1, 128, 16, 1, [1], None, "hnd"),
    ("bf16", "e4m3fn", 4, 8, 2, 128, 64, 1, [0, 1, 63, 64], None, "hnd"),
    ("fp16", "e5m2", 3, 4, 4, 64, 16, 1, [15, 17, 1000], None, "nhd"),
    ("bf16", "e4m3fn", 2, 32, 8, 128, 64, 1, [517, 3001], None, "halves"),
    ("bf16", "e5m2", 1, 12, 4, 64, 256, 1, [777], None, "hnd"),
    ("fp16", "e4m3fn", 2, 40, 8, 128, 32, 1, [129, 31], None, "nhd"),
    ("bf16", "e4m3fn", 2, 24, 2, 128, 128, 1, [700, 5], None, "hnd"),
    ("bf16", "e4m3fn", 3, 32, 1, 128, 64, 1, [900, 64, 1], None, "hnd"),
    ("fp16", "e4m3fn", 1, 71, 1, 64, 16, 1, [530], None, "halves"),
    ("bf16", "e5m2", 3, 8, 2, 128, 64, 5, [700, 3, 66], None, "hnd"),
    ("fp16", "e4m3fn", 2, 16, 2, 64, 16, 7, [6, 515], None, "nhd"),
    ("bf16", "e4m3fn", 2, 6, 6, 128, 32, 2, [65, 1], None, "hnd"),
    ("bf16", "e4m3fn", 3, 8, 2, 128, 64, 1, [700, 64, 3], 100, "hnd"),
    ("bf16", "e4m3fn", 3, 8, 2, 64, 16, 5, [700, 128, 3], 100, "hnd"),
    ("fp16", "e5m2", 2, 4, 1, 128, 128, 3, [1000, 130], 0, "nhd"),
    ("bf16", "e4m3fn", 1, 4, 1, 128, 64, 1, [20000], None, "hnd"),
    ("bf16", "e4m3fn", 2, 64, 1, 128, 64, 1, [300, 33], None, "hnd"),
    ("fp16", "e4m3fn", 1, 16, 2, 128, 32, 8, [260], None, "nhd"),
    ("fp16", "e4m3fn", 2, 56, 1, 64, 16, 1, [300, 17], None, "hnd"),
    ("bf16", "e4m3fn", 1, 8, 1, 64, 128, 17, [150], 40, "halves"),
    ("bf16", "e4m3fn", 1, 128, 1, 128, 256, 1, [500], None, "hnd"),
    ("fp16", "e5m2", 2, 16, 16, 64, 16, 1, [5000, 4999], 4097, "hnd"),
    ("bf16", "e4m3fn", 3, 8, 2, 128, 64, 150, [400, 151, 100], None, "nhd"),       # a chunk of a prompt
    ("fp16", "e4m3fn", 1, 6, 2, 64, 32, 333, [333], 64, "hnd"),
]


def _decode8(c, q, lens, where="", scale=None, **kw):
    import attention_forward_fa_gb300 as fa
    scale = c.D ** -0.5 if scale is None else scale
    o, l = fa.flash_attention_decode(_dev(q, c.dtype), c.obj, c.ints(lens), scale=scale,
                                     **{k: _dev(x) if k == "page_idx" else x for k, x in kw.items()})
    assert _status() == 0
    a = (c.table, lens, scale)
    pre, idx = kw.get("pre_tokens"), kw.get("page_idx")
    W, E = _spread(c, q, *a, None, pre, idx)
    _check8(o, l, P.decode(q, c.k, c.v, *a, pre, idx), W, E, c.dtype, where)


@pytest.mark.parametrize("case", DECODE, ids=lambda c: "-".join(map(str, c[:8])) + ("" if c[9] is None else f"-w{c[9]}"))
def test_decode8(case):
    dtype, fmt, B, Hq, Hkv, D, page, Sq, lens, pre, layout = case
    c = Cache8(6, dtype, fmt, B, Hkv, D, page, lens, layout, stale=True)
    q = _round(c.rng.standard_normal((B, Hq, Sq, D)), dtype)
    _decode8(c, q, lens, str(case), pre_tokens=pre)


@pytest.mark.parametrize("dtype,fmt,D", [("bf16", "e4m3fn", 128), ("fp16", "e4m3fn", 64), ("fp16", "e5m2", 128)])
@pytest.mark.parametrize("spread", [3.0, 12.0])
@pytest.mark.parametrize("Sq", [1, 12, 24, 40])
def test_decode8_values_of_any_size(dtype, fmt, D, spread, Sq):
    """Values whose rows differ by many powers of two: small ones with large
    probabilities beside large ones with small, rows of zeros among them."""
    lens = [700, 33, 130]
    for scale in (0.05, D ** -0.5, 1.0):
        c = Cache8(7, dtype, fmt, 3, 2, D, 32, lens, spread=spread)
        if dtype == "fp16":              # (the answers must fit: 448 * 2^4, 57344 * 2^0)
            shift = max(0, int(c.ve.max()) - (4 if fmt == "e4m3fn" else 0))
            c.ve -= shift
        zero = c.rng.random(c.ve.shape) < 0.1
        c.vc[zero], c.ve[zero] = 0, P.LEAST
        c.ve = np.maximum(c.ve, P.LEAST)
        c.v = np.ldexp(c.vc, c.ve[..., None])
        c.bv.copy_(_codes(c.vc, fmt).view(c.bv.dtype))
        c.sv.copy_(_dev((c.ve + 127).astype(np.uint8)))
        q = _round(c.rng.standard_normal((3, 8, Sq, D)), dtype)
        _decode8(c, q, lens, f"spread {spread} scale {scale}", scale=scale)


def test_decode8_all_values_zero_and_queries_of_any_size():
    import attention_forward_fa_gb300 as fa
    lens = [300]
    c = Cache8(8, "bf16", "e4m3fn", 1, 1, 128, 64, lens)
    q = _round(c.rng.standard_normal((1, 8, 1, 128)) * 2.0 ** np.array([0, -10, 10, -40, 3, -70, 1, 0])[None, :, None, None], "bf16")
    q[0, 6] = 0
    for h, scale in ((0, 0.1), (2, 1e-4), (3, 1e10), (5, 1e20), (6, 3.0)):
        _decode8(c, q[:, h:h + 1], lens, f"row {h}", scale=scale)
    _decode8(c, q[:, [0, 1, 3, 7]], lens, "rows together", scale=0.1)
    o = fa.flash_attention_decode(_dev(np.where(np.arange(8)[:, None, None] == 1, np.nan, q), "bf16"), c.obj, c.ints(lens), scale=0.1)[0]
    good = [0, 1 + 1, 3, 7]
    want = fa.flash_attention_decode(_dev(q, "bf16"), c.obj, c.ints(lens), scale=0.1)[0]
    assert np.array_equal(_host(o)[:, good], _host(want)[:, good])      # a NaN query reaches no other row
    c.vc[:], c.ve[:], c.v[:] = 0, P.LEAST, 0
    c.bv.zero_()
    c.sv.fill_(P.LEAST + 127)
    _decode8(c, q[:, :1], lens, "zeros", scale=0.1)
    assert _status() == 0


@pytest.mark.parametrize("dtype,fmt,B,Hq,Hkv,D,page,Sq,lens,sel", [
    ("bf16", "e4m3fn", 3, 8, 2, 128, 64, 1, [1000, 130, 5], 4),
    ("fp16", "e5m2", 2, 6, 3, 64, 16, 3, [500, 40], 12),
    ("bf16", "e4m3fn", 1, 4, 1, 128, 256, 2, [1500], 3),
    ("bf16", "e4m3fn", 70, 2, 2, 64, 32, 1, [100] * 70, 64),
    ("bf16", "e4m3fn", 3, 8, 2, 128, 64, 10, [1000, 130, 5], 4),
    ("fp16", "e5m2", 2, 6, 1, 64, 16, 30, [500, 40], 12),
    ("bf16", "e4m3fn", 2, 8, 1, 128, 64, 10, [700, 140], 6),
])
def test_decode8_listed_pages(dtype, fmt, B, Hq, Hkv, D, page, Sq, lens, sel):
    c = Cache8(9, dtype, fmt, B, Hkv, D, page, lens, stale=True)
    q = _round(c.rng.standard_normal((B, Hq, Sq, D)), dtype)
    idx = np.full((B, Hkv, sel), -1, dtype=np.int32)
    for b in range(B):
        n = -(-lens[b] // page)
        for h in range(Hkv):
            take = c.rng.permutation(n)[:min(sel, n)]
            idx[b, h, :len(take)] = take
    _decode8(c, q, lens, "listed", page_idx=idx)
    idx[0, 0, :2] = idx[0, 0, 0]          # a page listed twice counts twice
    _decode8(c, q, lens, "twice", page_idx=idx)


@pytest.mark.parametrize("D", [64, 128])
def test_decode8_growing_scores_and_subnormal_codes(D):
    """Keys of ever larger scores move every reference many times; keys and values made
    of the format's subnormals."""
    for dtype, fmt, step in (("bf16", "e4m3fn", 0.02), ("fp16", "e4m3fn", 0.3), ("bf16", "e5m2", -0.05)):
        lens = [1500]
        c = Cache8(10, dtype, fmt, 1, 1, D, 64, lens)
        k = c.k[c.table[0], 0].reshape(-1, D)
        k[:, 0] = np.arange(k.shape[0]) * step
        kc, ke = P.quantise(k.reshape(-1, 64, D), fmt)
        c.kc[c.table[0], 0], c.ke[c.table[0], 0] = kc, ke
        c.k = np.ldexp(c.kc, c.ke[..., None])
        c.bk.copy_(_codes(c.kc, fmt).view(c.bk.dtype))
        c.sk.copy_(_dev((c.ke + 127).astype(np.uint8)))
        q = _round(0.1 * c.rng.standard_normal((1, 4, 1, D)), dtype)
        q[..., 0] = np.array([1.0, 0.5, -1.0, 0.0])[None, :, None]
        _decode8(c, q, lens, f"{dtype} {step}", scale=1.0)
        least = HALF[fmt][1] * 2
        for x in (c.kc, c.vc):
            x[:] = c.rng.integers(-7 if fmt == "e4m3fn" else -3, 8 if fmt == "e4m3fn" else 4, x.shape) * least
        c.ke[:], c.ve[:] = 9 if fmt == "e4m3fn" else 15, 3
        c.k, c.v = np.ldexp(c.kc, c.ke[..., None]), np.ldexp(c.vc, c.ve[..., None])
        for t, s, x, e in ((c.bk, c.sk, c.kc, c.ke), (c.bv, c.sv, c.vc, c.ve)):
            t.copy_(_codes(x, fmt).view(t.dtype))
            s.copy_(_dev((e + 127).astype(np.uint8)))
        _decode8(c, q, lens, f"{dtype} subnormal codes", scale=0.2)


@pytest.mark.parametrize("B,Hq,Hkv,page,Sq", [(300, 1, 1, 16, 1), (513, 5, 1, 16, 1), (40, 8, 8, 32, 2)])
def test_decode8_many_sequences(B, Hq, Hkv, page, Sq):
    rng = np.random.default_rng(11)
    lens = [int(x) for x in rng.integers(0, 400, B)]
    c = Cache8(12, "bf16", "e4m3fn", B, Hkv, 64, page, lens, stale=True)
    _decode8(c, _round(rng.standard_normal((B, Hq, Sq, 64)), "bf16"), lens, "many")


@pytest.mark.parametrize("Sq", [1, 20, 40])
def test_decode8_leaves_out_bad_pages(Sq):
    import attention_forward_fa_gb300 as fa
    lens = [200, 200, 200]
    c = Cache8(13, "bf16", "e4m3fn", 3, 2, 128, 16, lens)
    q = _round(c.rng.standard_normal((3, 4, Sq, 128)), "bf16")
    c.table[0, 2], c.table[1, 12] = c.k.shape[0], -1
    c.obj.page_table.copy_(_dev(c.table))
    o, l = fa.flash_attention_decode(_dev(q, "bf16"), c.obj, c.ints(lens))
    assert _status() == fa.FA_ERR_INDEX and _status() == 0
    idx = np.tile(np.arange(13, dtype=np.int32), (3, 2, 1))
    idx[0, :, 2], idx[1, :, 12] = -1, -1
    a = (c.table, lens, 128 ** -0.5)
    W, E = _spread(c, q, *a, idx=idx)
    _check8(o, l, P.decode(q, c.k, c.v, *a, None, idx), W, E, "bf16")
    o, l = fa.flash_attention_decode(_dev(q, "bf16"), c.obj, c.ints([-3, 200000, 200]))
    assert _status() == fa.FA_ERR_INDEX
    assert bool((o[:2] == 0).all()) and bool((l[:2] == math.inf).all())


@pytest.mark.parametrize("dtype,fmt,G,Sq,n,grow", [
    ("fp16", "e4m3fn", 5, 16, 20000, 0.0), ("bf16", "e5m2", 4, 40, 9000, 0.0), ("fp16", "e4m3fn", 70, 1, 26000, 2e-3),
    ("bf16", None, 3, 13, 20000, 0.0), ("fp16", None, 5, 30, 17000, 3e-3),
])
def test_many_rows_over_long_pieces(dtype, fmt, G, Sq, n, grow):
    """More tiles of one unit in one CTA than add up in the accumulator, with scores that
    grow along the keys too: 160 sequences over the same pages, the same queries."""
    import torch
    import attention_forward_fa_gb300 as fa
    B, page, D = 160, 64, 64
    c = Cache(30, dtype, 1, 1, D, page, [n]) if fmt is None else Cache8(30, dtype, fmt, 1, 1, D, page, [n], spread=2.0)
    if grow:
        k = c.k[c.table[0], 0].reshape(-1, D)
        k[:, 0] = np.arange(k.shape[0]) * grow
        if fmt is None:
            c.k[c.table[0], 0] = _round(k, dtype).reshape(-1, page, D)
            c.tk.copy_(_dev(c.k, dtype))
        else:
            c.kc[c.table[0], 0], c.ke[c.table[0], 0] = P.quantise(k.reshape(-1, page, D), fmt)
            c.k = np.ldexp(c.kc, c.ke[..., None])
            c.bk.copy_(_codes(c.kc, fmt).view(c.bk.dtype))
            c.sk.copy_(_dev((c.ke + 127).astype(np.uint8)))
    q = _round(c.rng.standard_normal((1, G, Sq, D)), dtype)
    q[..., 0] = np.abs(q[..., 0])
    anc, _ = _trees(c.rng, 1, Sq)
    table = c.obj.page_table.expand(B, -1).contiguous()
    many = (fa.PagedKV(c.obj.k_pages, c.obj.v_pages, table) if fmt is None else
            fa.PagedKV(c.obj.k_pages, c.obj.v_pages, table, k_scale=c.sk, v_scale=c.sv, dtype=_torch_type(dtype)))
    o, l = fa.flash_attention_decode_tree(_dev(q, dtype).expand(B, -1, -1, -1).contiguous(), many,
                                          torch.full((B,), n, dtype=torch.int32, device="cuda"), _dev(anc[0]))
    assert _status() == 0
    a = (c.table, [n], D ** -0.5)
    ref = P.decode(q, c.k, c.v, *a, tree=(anc, [Sq]))
    for b in (0, 1, 77, 151, 152, 159):
        if fmt is None:
            _check(o[b:b + 1], l[b:b + 1], ref, dtype, f"sequence {b}")
        else:
            _check8(o[b:b + 1], l[b:b + 1], ref, *_spread(c, q, *a, (anc, [Sq])), dtype, f"sequence {b}")


# ------------------------------------------------------------------ trees
TREE = [
    # dtype, fmt or None, B, Hq, Hkv, D, page, S, lens (drafts included), drafts, one tree for all
    ("bf16", None, 1, 4, 1, 128, 64, 1, [1], [1], False),
    ("bf16", None, 3, 8, 2, 128, 64, 8, [517, 8, 70], [8, 8, 3], False),
    ("fp16", None, 2, 16, 2, 64, 16, 13, [200, 40], [13, 0], False),
    ("bf16", None, 2, 4, 4, 128, 16, 64, [64, 900], [64, 61], False),
    ("fp16", None, 2, 3, 1, 64, 256, 33, [300, 33], [33, 33], True),
    ("bf16", None, 1, 8, 1, 128, 32, 100, [2100], [100], False),
    ("bf16", None, 40, 2, 2, 64, 16, 5, list(range(5, 45)), [5] * 40, True),
    ("bf16", "e4m3fn", 1, 4, 1, 128, 64, 1, [1], [1], False),
    ("bf16", "e4m3fn", 3, 8, 2, 128, 64, 8, [517, 8, 70], [8, 8, 3], False),
    ("fp16", "e5m2", 2, 16, 2, 64, 16, 13, [200, 40], [13, 0], False),
    ("bf16", "e4m3fn", 2, 4, 4, 128, 16, 64, [64, 900], [64, 61], False),
    ("fp16", "e4m3fn", 2, 3, 1, 64, 256, 33, [300, 33], [33, 33], True),
    ("bf16", "e4m3fn", 1, 8, 1, 128, 32, 150, [2100], [147], False),
    # sequences without tokens or drafts, by warps and by tcgen05
    ("bf16", None, 4, 48, 1, 128, 16, 1, [0, 1, 300, 129], [0, 1, 1, 0], True),
    ("fp16", "e4m3fn", 4, 72, 1, 64, 32, 2, [0, 2, 300, 129], [0, 2, 1, 0], False),
    ("bf16", "e4m3fn", 4, 12, 4, 128, 32, 2, [0, 2, 300, 129], [0, 2, 1, 0], False),
    ("bf16", "e5m2", 3, 140, 1, 128, 128, 2, [2, 0, 260], [2, 0, 2], False),
    # many units of one tile or two per CTA, and two passes of rows
    ("bf16", None, 420, 4, 1, 64, 16, 10, [10 + 7 * b % 150 for b in range(420)], [10] * 420, True),
    ("bf16", "e4m3fn", 420, 4, 1, 64, 32, 20, [20 + 7 * b % 150 for b in range(420)], [20 - b % 3 for b in range(420)], False),
    ("bf16", "e4m3fn", 20, 4, 1, 128, 32, 12, [12 + 7 * b % 450 for b in range(20)], [12 - b % 3 for b in range(20)], False),
    ("fp16", "e4m3fn", 90, 66, 6, 128, 64, 4, [4 + 11 * b % 300 for b in range(90)], [4] * 90, True),
]


@pytest.mark.parametrize("case", TREE, ids=lambda c: "-".join(map(str, c[:8])))
@pytest.mark.parametrize("kind", ["tree", "blind"])
def test_tree(case, kind):
    """Random trees; blind: rows that do not see themselves, or any draft, and
    columns past the drafts set."""
    import torch
    import attention_forward_fa_gb300 as fa
    dtype, fmt, B, Hq, Hkv, D, page, S, lens, drafts, shared = case
    c = Cache(14, dtype, B, Hkv, D, page, lens) if fmt is None else Cache8(14, dtype, fmt, B, Hkv, D, page, lens, stale=True)
    anc, _ = _trees(c.rng, 1 if shared else B, S)
    if kind == "blind":
        anc[:, ::3] = False
        anc |= c.rng.random(anc.shape) < 0.1
        anc[0, 0] = False
    q = _round(c.rng.standard_normal((B, Hq, S, D)), dtype)
    for b in range(B):
        q[b, :, drafts[b]:] *= 3
    q = _round(q, dtype)                  # (what the device gets)
    ta = _dev(anc[0] if shared else anc) if kind == "tree" else _dev((anc[0] if shared else anc).astype(np.uint8) * 200)
    full = np.broadcast_to(anc, (B, S, S))
    n = c.ints(drafts)
    o, l = fa.flash_attention_decode_tree(_dev(q, dtype), c.obj, c.ints(lens), ta, new_lens=n)
    assert _status() == 0
    a = (c.table, lens, D ** -0.5)
    ref = P.decode(q, c.k, c.v, *a, tree=(full, drafts))
    if fmt is None:
        _check(o, l, ref, dtype, str(case))
    else:
        _check8(o, l, ref, *_spread(c, q, *a, (full, drafts)), dtype, str(case))
    if all(d == S for d in drafts):       # new_lens left out, and trees of any stride
        o2, l2 = fa.flash_attention_decode_tree(_dev(q, dtype), c.obj, c.ints(lens),
                                                _dev(np.repeat(full, 2, 0))[::2] if not shared else ta.expand(B, S, S))
        assert torch.equal(o, o2) and torch.equal(l, l2)
    bad = _dev(np.where(np.arange(S)[:, None] >= np.asarray(drafts)[:, None, None, None], np.nan, q), dtype)
    o3, l3 = fa.flash_attention_decode_tree(bad, c.obj, c.ints(lens), ta, new_lens=n)
    for b in range(B):                    # padding reaches no other row
        assert torch.equal(o[b, :, :drafts[b]], o3[b, :, :drafts[b]]) and torch.equal(l[b, :, :drafts[b]], l3[b, :, :drafts[b]])
    assert _status() == 0


@pytest.mark.parametrize("dtype,fmt,Hq,S", [("bf16", None, 2, 6), ("fp16", None, 8, 20), ("bf16", None, 40, 11), ("bf16", "e4m3fn", 2, 6),
                                            ("fp16", "e5m2", 8, 20), ("bf16", "e4m3fn", 40, 11)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_tree_scales_and_unseen_places(dtype, fmt, Hq, S, bad):
    """Scales from flat to one-hot and a negative one; keys and values behind a sequence's tokens, in its own
    pages too, are anything."""
    import torch
    import attention_forward_fa_gb300 as fa
    lens, drafts, D, page = [333, 40, S], [S, S - 2, S], 64, 32
    cap = [-(-n // page) * page for n in lens]
    c = Cache(33, dtype, 3, 1, D, page, cap) if fmt is None else Cache8(33, dtype, fmt, 3, 1, D, page, cap)
    for b, n in enumerate(lens):
        for t in range(n, cap[b]):
            p, s = int(c.table[b, t // page]), t % page
            if fmt is None:
                c.tk[p, :, s] = bad
                c.tv[p, :, s] = -bad
            else:
                c.bk[p, :, s], c.bv[p, :, s] = 0x7F, 0xFE
                c.sk[p, :, s], c.sv[p, :, s] = 255, 255 if t % 2 else 0
    anc, _ = _trees(c.rng, 3, S)
    q = _round(c.rng.standard_normal((3, Hq, S, D)), dtype)
    for scale in (0.0, -0.2, 0.125, 3.0):
        o, l = fa.flash_attention_decode_tree(_dev(q, dtype), c.obj, c.ints(lens), _dev(anc), new_lens=c.ints(drafts), scale=scale)
        assert _status() == 0
        a = (c.table, lens, scale)
        ref = P.decode(q, c.k, c.v, *a, tree=(anc, drafts))
        if fmt is None:
            _check(o, l, ref, dtype, f"scale {scale}")
        else:
            _check8(o, l, ref, *_spread(c, q, *a, (anc, drafts)), dtype, f"scale {scale}")


@pytest.mark.parametrize("fmt", [None, "e4m3fn"])
def test_trees_on_two_streams_at_once(fmt):
    """Calls with many rows on two streams beside a matrix product of torch's on a third: each has scratch and
    accumulators of its own."""
    import torch
    import attention_forward_fa_gb300 as fa
    lens, S = [2000, 700], 24
    cs = [Cache(34 + i, "bf16", 2, 4, 128, 64, lens) if fmt is None else Cache8(34 + i, "bf16", fmt, 2, 4, 128, 64, lens) for i in range(2)]
    qs = [_dev(_round(c.rng.standard_normal((2, (16, 32)[i], S, 128)), "bf16"), "bf16") for i, c in enumerate(cs)]
    anc = [_dev(_trees(c.rng, 2, S)[0]) for c in cs]
    n = cs[0].ints(lens)
    want = [fa.flash_attention_decode_tree(q, c.obj, n, a) for q, c, a in zip(qs, cs, anc)]
    m = torch.randn(1024, 1024, device="cuda", dtype=torch.bfloat16)
    prod = m @ m
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(3)], [[], []]
    for _ in range(20):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                got[i].append(fa.flash_attention_decode_tree(qs[i], cs[i].obj, n, anc[i]))
        with torch.cuda.stream(streams[2]):
            other = m @ m
    torch.cuda.synchronize()
    for i in range(2):
        for o, l in got[i]:
            assert torch.equal(o, want[i][0]) and torch.equal(l, want[i][1])
    assert torch.equal(other, prod) and _status() == 0


@pytest.mark.parametrize("fmt", [None, "e4m3fn"])
def test_a_chain_of_drafts_is_decode(fmt):
    import torch
    import attention_forward_fa_gb300 as fa
    lens, S = [300, 40, 7], 7
    c = Cache(15, "bf16", 3, 2, 128, 32, lens) if fmt is None else Cache8(15, "bf16", fmt, 3, 2, 128, 32, lens)
    q = _dev(_round(c.rng.standard_normal((3, 8, S, 128)), "bf16"), "bf16")
    chain = torch.ones(S, S, dtype=torch.bool, device="cuda").tril()
    for x, y in zip(fa.flash_attention_decode_tree(q, c.obj, c.ints(lens), chain), fa.flash_attention_decode(q, c.obj, c.ints(lens))):
        assert torch.equal(x, y)
    assert _status() == 0


def test_tree_reports_what_does_not_fit():
    import attention_forward_fa_gb300 as fa
    lens, S = [50, 3, 50, 50], 6
    c = Cache(16, "bf16", 4, 2, 64, 16, [50] * 4)
    q = _round(c.rng.standard_normal((4, 4, S, 64)), "bf16")
    anc, _ = _trees(c.rng, 4, S)
    o, l = fa.flash_attention_decode_tree(_dev(q, "bf16"), c.obj, c.ints(lens), _dev(anc), new_lens=c.ints([6, 5, -1, 9]))
    assert _status() == fa.FA_ERR_INDEX and _status() == 0
    _check(o, l, P.decode(q, c.k, c.v, c.table, lens, 0.125, tree=(anc, [6, 3, 0, 6])), "bf16")
    fa.flash_attention_decode_tree(_dev(q, "bf16"), c.obj, c.ints(lens), _dev(anc))        # 6 drafts of 3 tokens
    assert _status() == fa.FA_ERR_INDEX and _status() == 0
    o, l = fa.flash_attention_decode_tree(_dev(q, "bf16"), c.obj, c.ints([50, 0, -5, 1000]), _dev(anc), new_lens=c.ints([2, 0, 2, 2]))
    assert _status() == fa.FA_ERR_INDEX
    assert bool((o[1:] == 0).all()) and bool((l[1:] == math.inf).all())


# ------------------------------------------------------------------ reading back
READ = [
    # dtype, fmt or None, B, Hkv, D, page, S, starts, lens, layout
    ("bf16", None, 1, 1, 128, 64, 1, [0], [1], "hnd"),
    ("fp16", None, 3, 5, 64, 16, 70, [3, 0, 100], [70, 0, 41], "nhd"),
    ("bf16", "e4m3fn", 2, 8, 128, 64, 333, [0, 63], [333, 130], "hnd"),
    ("fp16", "e5m2", 3, 3, 64, 16, 65, None, [65, 1, 64], "halves"),
    ("fp16", "e4m3fn", 1, 2, 128, 256, 1000, [777], [1000], "nhd"),
    ("bf16", "e5m2", 2, 1, 64, 128, 129, [128, 127], [129, 128], "hnd"),
]


@pytest.mark.parametrize("case", READ, ids=lambda c: "-".join(map(str, c[:7])))
@pytest.mark.parametrize("form", ["dense", "strided"])
def test_read(case, form):
    import torch
    import attention_forward_fa_gb300 as fa
    dtype, fmt, B, Hkv, D, page, S, starts, lens, layout = case
    first = starts or [0] * B
    cap = [s + n for s, n in zip(first, lens)]
    c = Cache(17, dtype, B, Hkv, D, page, cap, layout) if fmt is None else Cache8(17, dtype, fmt, B, Hkv, D, page, cap, layout, stale=True)
    mk, mv = (_round(c.rng.standard_normal((B, Hkv, S, D)), dtype) for _ in range(2))
    ek, ev = P.read(c.k, c.v, c.table, first, lens, mk, mv)
    if form == "dense":
        k, v = _dev(mk, dtype), _dev(mv, dtype)
    else:                                # [B, S, 2, Hkv, D + 8]
        both = torch.zeros(B, S, 2, Hkv, D + 8, dtype=_torch_type(dtype), device="cuda")
        k, v = (both[:, :, i, :, :D].transpose(1, 2) for i in range(2))
        k.copy_(_dev(mk, dtype)), v.copy_(_dev(mv, dtype))
    kw = {} if starts is None else dict(starts=c.ints(starts))
    got = fa.paged_kv_read(c.obj, c.ints(lens), k_out=k, v_out=v, **kw)
    assert got[0] is k and got[1] is v and _status() == 0
    assert np.array_equal(_host(k), _round(ek, dtype)) and np.array_equal(_host(v), _round(ev, dtype))
    if form == "strided":
        assert bool((both[..., D:] == 0).all())
    k2, v2 = fa.paged_kv_read(c.obj, c.ints(lens), size=S, **kw)
    for b in range(B):
        assert torch.equal(k2[b, :, :lens[b]], k[b, :, :lens[b]]) and torch.equal(v2[b, :, :lens[b]], v[b, :, :lens[b]])


def test_read_leaves_out_what_is_not_there():
    import attention_forward_fa_gb300 as fa
    for c in (Cache(18, "bf16", 5, 2, 64, 16, [64] * 5), Cache8(18, "bf16", "e4m3fn", 5, 2, 64, 16, [64] * 5)):
        c.table[1, 1] = c.k.shape[0]
        c.obj.page_table.copy_(_dev(c.table))
        mk = _round(c.rng.standard_normal((5, 2, 40, 64)), "bf16")
        k, v = _dev(mk, "bf16"), _dev(mk, "bf16")
        fa.paged_kv_read(c.obj, c.ints([40, 40, 50, 40, -2]), starts=c.ints([0, 0, 10, 30, 0]), k_out=k, v_out=v)
        assert _status() == fa.FA_ERR_INDEX and _status() == 0
        t = c.table.copy()
        t[1, 1] = 0
        ek, _ = P.read(c.k, c.v, t, [0, 0, 10, 0, 0], [40, 40, 40, 0, 0], mk, mk)
        ek[1, :, 16:32] = mk[1, :, 16:32]
        assert np.array_equal(_host(k), _round(ek, "bf16"))


# ------------------------------------------------------------------ keeping
KEEP = [
    # dtype, fmt or None, B, Hkv, D, page, S, old, idx, layout
    ("bf16", None, 1, 1, 128, 64, 4, [517], [[1, 3]], "hnd"),
    ("fp16", None, 3, 5, 64, 16, 20, [0, 15, 31], [[0, 1, 2, 7, 19], [1, 17], []], "nhd"),
    ("bf16", "e4m3fn", 2, 8, 128, 64, 70, [60, 0], [list(range(0, 70, 2)), list(range(1, 70))], "hnd"),
    ("fp16", "e5m2", 3, 3, 64, 16, 30, [16, 3, 100], [[29], [0], [2, 3, 5, 7, 11, 13, 17, 19, 23, 29]], "halves"),
    ("bf16", "e4m3fn", 1, 40, 128, 256, 100, [250], [list(range(3, 100))], "nhd"),
    ("bf16", None, 2, 17, 128, 32, 40, [31, 32], [list(range(1, 40)), list(range(40))], "halves"),
]


@pytest.mark.parametrize("case", KEEP, ids=lambda c: "-".join(map(str, c[:7])))
def test_keep(case):
    import attention_forward_fa_gb300 as fa
    dtype, fmt, B, Hkv, D, page, S, old, paths, layout = case
    cap = [o + S for o in old]
    c = (Cache(19, dtype, B, Hkv, D, page, cap, layout, bounds=True) if fmt is None else
         Cache8(19, dtype, fmt, B, Hkv, D, page, cap, layout, bounds=True))
    M = max(len(p) for p in paths) + 1
    idx = np.full((B, M), -3, dtype=np.int32)
    for b, p in enumerate(paths):
        idx[b, :len(p)] = p
    n = [len(p) for p in paths]
    fa.paged_kv_keep(c.obj, c.ints(old), c.ints(idx), c.ints(n))
    assert _status() == 0
    pools = [c.k, c.v] if fmt is None else [c.kc, c.vc, c.ke, c.ve]
    want, lo, hi = P.keep(pools, c.table, old, idx, n, page, c.k, c.lo, c.hi)
    if fmt is None:
        got = [_host(c.tk), _host(c.tv)]
    else:
        kc, ke, vc, ve = c.stored()
        got = [kc, vc, ke, ve]
    assert all(np.array_equal(a, b) for a, b in zip(got, want))
    gl, gh = _host(c.tlo), _host(c.thi)
    if fmt is None or dtype == "bf16":
        assert np.array_equal(gl, lo) and np.array_equal(gh, hi)
    else:
        assert (gl <= lo + 2.0 ** -11 * np.abs(lo)).all() and (gh >= hi - 2.0 ** -11 * np.abs(hi)).all()
        assert (np.abs(gl - lo) <= 2.0 ** -10 * np.abs(lo) + 2.0 ** -24).all() and (np.abs(gh - hi) <= 2.0 ** -10 * np.abs(hi) + 2.0 ** -24).all()


def test_keep_ends_a_path_at_what_does_not_fit():
    import attention_forward_fa_gb300 as fa
    for c in (Cache(20, "bf16", 6, 2, 64, 16, [48] * 6), Cache8(20, "bf16", "e4m3fn", 6, 2, 64, 16, [48] * 6)):
        c.table[3, 2] = -4
        c.obj.page_table.copy_(_dev(c.table))
        old = [10, 10, 10, 10, 10, -1]
        idx = np.array([[1, 3, 3, 5], [2, 1, 5, 6], [1, 4, 38, 39], [1, 2, 23, 30], [-1, 2, 3, 4], [1, 2, 3, 4]], dtype=np.int32)
        fa.paged_kv_keep(c.obj, c.ints(old), c.ints(idx), c.ints([4, 4, 4, 4, 4, 4]))
        assert _status() == fa.FA_ERR_INDEX and _status() == 0
        n = [2, 1, 2, 2, 0, 0]
        eight = isinstance(c, Cache8)
        want, _, _ = P.keep([c.kc, c.ke] if eight else [c.k], c.table, old, idx, n, 16)
        got = c.stored()[:2] if eight else [_host(c.tk)]
        assert all(np.array_equal(a, b) for a, b in zip(got, want))
        was = c.obj.k_pages.view(dtype=__import__("torch").uint8).clone()
        fa.paged_kv_keep(c.obj, c.ints([10] * 6), c.ints(idx), c.ints([0, 0, 0, 0, -1, 0]))
        assert _status() == fa.FA_ERR_INDEX
        assert bool((was == c.obj.k_pages.view(dtype=was.dtype)).all())


# ------------------------------------------------------------------ together
@pytest.mark.parametrize("dtype,fmt,D,page,inter", [("bf16", "e4m3fn", 128, 64, False), ("fp16", "e5m2", 64, 16, True),
                                                    ("bf16", None, 128, 16, False)])
def test_drafting_run(dtype, fmt, D, page, inter):
    """Prompts into the cache; then steps of a tree of drafts each (appended by depth, attended over,
    a path of it kept); a token by token step and chosen pages last; and the cache read back."""
    import torch
    import attention_forward_fa_gb300 as fa
    B, Hq, Hkv, S = 3, 8, 2, 9
    prompt, total = [100, 1, 333], 420
    c = (Cache(21, dtype, B, Hkv, D, page, [total] * B, bounds=True) if fmt is None else
         Cache8(21, dtype, fmt, B, Hkv, D, page, [total] * B, bounds=True))
    cos, sin = _tables(total, D)
    kw = dict(cos=_dev(cos), sin=_dev(sin), interleaved=inter)
    lens = np.zeros(B, dtype=np.int64)

    def append(S, new, **more):
        x = _dev(_round(c.rng.standard_normal((B, Hq + 2 * Hkv, S, D)), dtype), dtype)
        return fa.paged_kv_append(c.obj, c.ints(lens), x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], new_lens=c.ints(new),
                                  q=x[:, :Hq], q_out=torch.zeros_like(x[:, :Hq]), **kw, **more)

    def check(o, l, q, lens, tree=None, idx=None):
        if fmt is None:
            k, v = _host(c.tk), _host(c.tv)
            _check(o, l, P.decode(_host(q), k, v, c.table, lens, D ** -0.5, None, idx, tree), dtype)
        else:
            c.kc, c.ke, c.vc, c.ve = c.stored()
            c.k, c.v = c.values()
            _check8(o, l, P.decode(_host(q), c.k, c.v, c.table, lens, D ** -0.5, None, idx, tree),
                    *_spread(c, _host(q), c.table, lens, D ** -0.5, tree, None, idx), dtype)

    append(333, prompt)
    lens += prompt
    for step in range(4):
        drafts = [S, S - 3, 1 + step]
        anc, depth = _trees(c.rng, B, S)
        pos = (lens[:, None] + depth).astype(np.int32)
        q = append(S, drafts, positions=_dev(pos))
        both = lens + drafts
        o, l = fa.flash_attention_decode_tree(q, c.obj, c.ints(both), _dev(anc), new_lens=c.ints(drafts))
        check(o, l, q, both, (anc, drafts))
        # the way to some draft of each sequence
        idx, n = np.full((B, S), -1, dtype=np.int32), []
        for b in range(B):
            path = np.flatnonzero(anc[b, c.rng.integers(drafts[b])])
            idx[b, :len(path)] = path
            n.append(len(path))
        fa.paged_kv_keep(c.obj, c.ints(lens), c.ints(idx), c.ints(n))
        lens += n
    assert _status() == 0
    q = append(1, [1] * B)
    lens += 1
    o, l = fa.flash_attention_decode(q, c.obj, c.ints(lens))
    check(o, l, q, lens)
    idx = fa.select_kv_pages(q, c.obj, c.ints(lens), 3)
    ref = P.select(_host(q), _host(c.tlo), _host(c.thi), c.table, lens, page, 3)
    assert np.array_equal(idx.cpu().numpy(), ref)
    o, l = fa.flash_attention_decode(q, c.obj, c.ints(lens), page_idx=idx)
    check(o, l, q, lens, None, ref)
    # the bounds bound what the cache holds
    k = _host(c.tk) if fmt is None else c.values()[0]
    for b in range(B):
        for p in range(-(-int(lens[b]) // page)):
            i, z = c.table[b, p], min(page, int(lens[b]) - p * page)
            assert (_host(c.tlo)[i][:, None] <= k[i, :, :z]).all() and (_host(c.thi)[i][:, None] >= k[i, :, :z]).all()
    rk, rv = fa.paged_kv_read(c.obj, c.ints(lens), size=total)
    k, v = (_host(c.tk), _host(c.tv)) if fmt is None else c.values()
    ek, ev = P.read(k, v, c.table, [0] * B, lens, np.zeros(rk.shape), np.zeros(rk.shape))
    for b in range(B):
        assert np.array_equal(_host(rk)[b, :, :lens[b]], _round(ek, dtype)[b, :, :lens[b]])
        assert np.array_equal(_host(rv)[b, :, :lens[b]], _round(ev, dtype)[b, :, :lens[b]])
    assert _status() == 0


def test_read_back_feeds_the_forward():
    """The prefix of a prompt out of an 8-bit cache, and the dense forward over it."""
    import torch
    import attention_forward_fa_gb300 as fa
    n, D = 300, 128
    c = Cache8(22, "bf16", "e4m3fn", 1, 2, D, 64, [n])
    k, v = fa.paged_kv_read(c.obj, c.ints([n]), size=n)
    q = _dev(_round(c.rng.standard_normal((1, 8, n, D)), "bf16"), "bf16")
    o, l = fa.flash_attention_forward(q, k, v, causal=True)
    od, ld = fa.flash_attention_decode(q, c.obj, c.ints([n]))
    W, E = _spread(c, _host(q), c.table, [n], D ** -0.5)
    ref = P.decode(_host(q), c.k, c.v, c.table, [n], D ** -0.5)
    _check8(od, ld, ref, W, E, "bf16")
    assert (np.abs(_host(o) - ref[0]) <= 1e-4 + 7.8125e-3 * np.abs(ref[0])).all()
    assert _status() == 0


def test_streams_and_graphs():
    """A step of drafts captured whole (append by depth, tree attention, keep, read), replayed on a
    stream while eager calls run on another; streams given by handle."""
    import torch
    import attention_forward_fa_gb300 as fa
    B, Hq, Hkv, D, page, S = 2, 8, 2, 128, 64, 6
    cos, sin = (_dev(x) for x in _tables(1100, D))

    def state(seed):
        c = Cache8(seed, "bf16", "e4m3fn", B, Hkv, D, page, [1000, 300], bounds=True)
        x = _dev(_round(c.rng.standard_normal((B, Hq + 2 * Hkv, S, D)), "bf16"), "bf16")
        anc, depth = _trees(c.rng, B, S)
        lens = c.ints([900, 200])
        s = dict(c=c, x=x, anc=_dev(anc), lens=lens, both=lens + S, pos=(lens[:, None] + _dev(depth)).contiguous(),
                 idx=c.ints([[1, 3, 5], [0, 2, -1]]), n=c.ints([3, 2]), q=torch.zeros(B, Hq, S, D, dtype=torch.bfloat16, device="cuda"),
                 o=torch.zeros(B, Hq, S, D, dtype=torch.bfloat16, device="cuda"), l=torch.zeros(B, Hq, S, device="cuda"),
                 k=torch.zeros(B, Hkv, 910, D, dtype=torch.bfloat16, device="cuda"), v=torch.zeros(B, Hkv, 910, D, dtype=torch.bfloat16, device="cuda"))
        return s

    def step(s, stream=None):
        kw = dict(stream=stream)
        fa.paged_kv_append(s["c"].obj, s["lens"], s["x"][:, Hq:Hq + Hkv], s["x"][:, Hq + Hkv:], q=s["x"][:, :Hq], q_out=s["q"],
                           cos=cos, sin=sin, positions=s["pos"], **kw)
        fa.flash_attention_decode_tree(s["q"], s["c"].obj, s["both"], s["anc"], out=s["o"], lse=s["l"], **kw)
        fa.paged_kv_keep(s["c"].obj, s["lens"], s["idx"], s["n"], **kw)
        fa.paged_kv_read(s["c"].obj, s["n"], starts=s["lens"], k_out=s["k"], v_out=s["v"], **kw)

    names = ("q", "o", "l", "k", "v")
    want = {}
    for seed in (23, 24, 25):
        s = state(seed)
        step(s)
        torch.cuda.synchronize()
        want[seed] = [s[x].clone() for x in names]
    a, b, d = state(23), state(24), state(25)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    step(d, stream=side)
    side.synchronize()
    assert all(torch.equal(d[x], w) for x, w in zip(names, want[25]))
    step(d, stream=side.cuda_stream)
    side.synchronize()
    assert all(torch.equal(d[x], w) for x, w in zip(names, want[25]))
    graphs = []
    for s in (a, b):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step(s)
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(10):
        for s in (a, b):
            for x in names:
                s[x].zero_()
        torch.cuda.synchronize()
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                for _ in range(3):
                    g.replay()
        step(d)
        torch.cuda.synchronize()
        for s, seed in ((a, 23), (b, 24), (d, 25)):
            assert all(torch.equal(s[x], w) for x, w in zip(names, want[seed])), seed
    assert _status() == 0


def test_beyond_32_bit_offsets():
    """An 8-bit pool of more than 2^32 codes; the sequence's pages lie at its end."""
    import torch
    import attention_forward_fa_gb300 as fa
    Hkv, page, D = 8, 64, 128
    num = 2 ** 32 // (Hkv * page * D) + 40
    k = torch.empty(num, Hkv, page, D, dtype=torch.uint8, device="cuda")
    v = torch.empty_like(k)
    sk, sv = (torch.zeros(num, Hkv, page, dtype=torch.uint8, device="cuda") for _ in range(2))
    rng = np.random.default_rng(26)
    table = np.arange(num - 1, num - 21, -1, dtype=np.int32)[None]
    cache = fa.PagedKV(k.view(torch.float8_e4m3fn), v.view(torch.float8_e4m3fn), _dev(table), k_scale=sk, v_scale=sv)
    x, y = (_round(rng.standard_normal((1, Hkv, 20 * page, D)), "bf16") for _ in range(2))
    fa.paged_kv_append(cache, _dev(np.zeros(1, dtype=np.int32)), _dev(x, "bf16"), _dev(y, "bf16"))
    n = _dev(np.array([1250], dtype=np.int32))
    q = _round(rng.standard_normal((1, 16, 1, D)), "bf16")
    o, l = fa.flash_attention_decode(_dev(q, "bf16"), cache, n)

    class Small:
        fmt, D = "e4m3fn", 128
    s = Small()
    split = lambda z: np.ascontiguousarray(z[0].reshape(Hkv, 20, page, D).transpose(1, 0, 2, 3))
    (s.kc, s.ke), (s.vc, s.ve) = P.quantise(split(x), "e4m3fn"), P.quantise(split(y), "e4m3fn")
    s.k, s.v = np.ldexp(s.kc, s.ke[..., None]), np.ldexp(s.vc, s.ve[..., None])
    flat = np.arange(20, dtype=np.int32)[None]
    _check8(o, l, P.decode(q, s.k, s.v, flat, [1250], D ** -0.5), *_spread(s, q, flat, [1250], D ** -0.5), "bf16")
    idx = _dev(np.array([[3, 6]], dtype=np.int32))
    fa.paged_kv_keep(cache, n, idx, _dev(np.array([2], dtype=np.int32)))
    kk, vv = fa.paged_kv_read(cache, n, starts=_dev(np.array([2], dtype=np.int32)), size=1250)
    (s.kc, s.vc, s.ke, s.ve), _, _ = P.keep([s.kc, s.vc, s.ke, s.ve], flat, [1250], np.array([[3, 6]]), [2], page)
    s.k, s.v = np.ldexp(s.kc, s.ke[..., None]), np.ldexp(s.vc, s.ve[..., None])
    ek, ev = P.read(s.k, s.v, flat, [2], [1250], np.zeros(kk.shape), np.zeros(kk.shape))
    assert np.array_equal(_host(kk), ek) and np.array_equal(_host(vv), ev)
    assert _status() == 0


def test_steps_in_flight8():
    """Many steps with nothing between their calls: the same bits as with a wait after every call."""
    import torch
    import attention_forward_fa_gb300 as fa
    B, Hq, Hkv, D, page, S, steps = 5, 8, 2, 128, 16, 4, 40
    cos, sin = (_dev(x) for x in _tables(400, D))
    rng = np.random.default_rng(27)
    xs = [_dev(_round(rng.standard_normal((B, Hq + 2 * Hkv, S, D)), "bf16"), "bf16") for _ in range(steps)]
    anc, depth = _trees(rng, B, S, 2)
    anc, depth = _dev(anc), _dev(depth)
    idx, n = _dev(np.tile(np.array([[1, 3, -1]], dtype=np.int32), (B, 1))), _dev(np.full(B, 2, dtype=np.int32))
    lens = [_dev(np.arange(B, dtype=np.int32) * 7 + 2 * i) for i in range(steps + 1)]
    both, pos = [x + S for x in lens], [(x[:, None] + depth).contiguous() for x in lens]

    def run(wait):
        c = Cache8(28, "bf16", "e4m3fn", B, Hkv, D, page, [200] * B, bounds=True)
        outs = [(torch.empty(B, Hq, S, D, dtype=torch.bfloat16, device="cuda"), torch.empty(B, Hq, S, D, dtype=torch.bfloat16, device="cuda"),
                 torch.empty(B, Hq, S, device="cuda"), *(torch.zeros(B, Hkv, 200, D, dtype=torch.bfloat16, device="cuda") for _ in range(2)))
                for _ in range(steps)]
        torch.cuda.synchronize()
        for i, (q, o, l, k, v) in enumerate(outs):
            x = xs[i]
            for call in (lambda: fa.paged_kv_append(c.obj, lens[i], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], q=x[:, :Hq], q_out=q, cos=cos, sin=sin, positions=pos[i]),
                         lambda: fa.flash_attention_decode_tree(q, c.obj, both[i], anc, out=o, lse=l),
                         lambda: fa.paged_kv_keep(c.obj, lens[i], idx, n),
                         lambda: fa.paged_kv_read(c.obj, lens[i + 1], k_out=k, v_out=v)):
                call()
                if wait:
                    torch.cuda.synchronize()
        torch.cuda.synchronize()
        return [t for ts in outs for t in ts] + [c.bk, c.bv, c.sk, c.sv, c.tlo, c.thi]

    want = run(True)
    for _ in range(4):
        for i, (a, b) in enumerate(zip(run(False), want)):
            assert torch.equal(a, b), f"output {i}"
    assert _status() == 0


@pytest.mark.parametrize("fmt,D,B,G,n", [("e4m3fn", 128, 304, 1, 131072), ("e5m2", 64, 100, 8, 131072)])
def test_decode8_long_sums_lose_nothing(fmt, D, B, G, n):
    """Equal values behind equal keys: the answer is the value, whatever the length and the split."""
    import torch
    import attention_forward_fa_gb300 as fa
    page, one = 64, 17
    k = torch.zeros(one, 1, page, D, dtype=torch.uint8, device="cuda")
    v = torch.full((one, 1, page, D), 0x3F if fmt == "e4m3fn" else 0x3E, dtype=torch.uint8, device="cuda")     # 1.875, 1.5
    value = 1.875 if fmt == "e4m3fn" else 1.5
    sk, sv = (torch.full((one, 1, page), x, dtype=torch.uint8, device="cuda") for x in (127, 124))
    kind = torch.float8_e4m3fn if fmt == "e4m3fn" else torch.float8_e5m2
    table = (torch.arange(n // page, device="cuda", dtype=torch.int32) % one).expand(B, -1).contiguous()
    c = fa.PagedKV(k.view(kind), v.view(kind), table, k_scale=sk, v_scale=sv, dtype=torch.float16)
    q = torch.randn(B, G, 1, D, device="cuda").half()
    o, l = fa.flash_attention_decode(q, c, torch.full((B,), n, device="cuda", dtype=torch.int32))
    assert _status() == 0
    # the sums' own roundings: 2^-24 for each of the 1024 tiles, of numerator and denominator
    assert float((o.double() - value / 8).abs().max()) <= (2.0 ** -13 + 2.0 ** -11) * value / 8
    assert float((l.double() - math.log(n)).abs().max()) <= 2.0 ** -13 + 2.0 ** -20 * math.log(n)


def test_wrappers_refuse_what_does_not_fit8():
    import torch
    import attention_forward_fa_gb300 as fa
    c = Cache8(29, "bf16", "e4m3fn", 2, 2, 64, 16, [40, 40])
    n = c.ints([40, 40])
    q = torch.zeros(2, 4, 3, 64, dtype=torch.bfloat16, device="cuda")
    anc = torch.ones(2, 3, 3, dtype=torch.bool, device="cuda")
    x = q[:, :2].contiguous()
    k8 = c.obj.k_pages
    for a, kw in (((k8, k8, c.obj.page_table), {}), ((k8, k8, c.obj.page_table), dict(k_scale=c.sk)),
                  ((k8, k8, c.obj.page_table), dict(k_scale=c.sk, v_scale=c.sk[:-1])),
                  ((k8, k8, c.obj.page_table), dict(k_scale=c.sk, v_scale=c.sk.int())),
                  ((k8, k8.view(torch.float8_e5m2), c.obj.page_table), dict(k_scale=c.sk, v_scale=c.sv)),
                  ((x, x, c.obj.page_table), dict(k_scale=c.sk, v_scale=c.sv)),
                  ((k8, k8, c.obj.page_table, torch.zeros(k8.shape[0], 2, 64, device="cuda"), torch.zeros(k8.shape[0], 2, 64, device="cuda")),
                   dict(k_scale=c.sk, v_scale=c.sv))):
        with pytest.raises(ValueError):
            fa.PagedKV(*a, **kw)
    with pytest.raises(TypeError):
        fa.PagedKV(k8, k8, c.obj.page_table, k_scale=c.sk, v_scale=c.sv, dtype=torch.float32)
    for bad in (anc.float(), anc.cpu(), anc[:1], anc[:, :2], anc.transpose(1, 2)[:, :, :2], anc[0, 0]):
        with pytest.raises(ValueError):
            fa.flash_attention_decode_tree(q, c.obj, n, bad)
    for bad in (q.half(), q[:, :, ::2], q[:, :3]):
        with pytest.raises(ValueError):
            fa.flash_attention_decode_tree(bad, c.obj, n, anc)
    for bad in (n.long(), n[:1], n.cpu()):
        with pytest.raises(ValueError):
            fa.flash_attention_decode_tree(q, c.obj, n, anc, new_lens=bad)
        with pytest.raises(ValueError):
            fa.paged_kv_read(c.obj, bad, size=3)
        with pytest.raises(ValueError):
            fa.paged_kv_read(c.obj, n, starts=bad, size=3)
        with pytest.raises(ValueError):
            fa.paged_kv_keep(c.obj, bad, c.ints([[0], [0]]), n)
        with pytest.raises(ValueError):
            fa.paged_kv_keep(c.obj, n, c.ints([[0], [0]]), bad)
    with pytest.raises(ValueError):
        fa.paged_kv_append(c.obj, n, x, x, positions=c.ints([0, 1]))
    with pytest.raises(ValueError):
        fa.paged_kv_keep(c.obj, n, c.ints([0, 0]), n)
    for kw in ({}, dict(size=3, k_out=x, v_out=x), dict(k_out=x), dict(k_out=x.half(), v_out=x.half()), dict(k_out=x[:1], v_out=x[:1]),
               dict(k_out=x, v_out=x[:, :, :2])):
        with pytest.raises(ValueError):
            fa.paged_kv_read(c.obj, n, **kw)
    with pytest.raises(fa.FaError):
        fa.paged_kv_read(c.obj, n, size=0)
    with pytest.raises(fa.FaError):
        fa.paged_kv_keep(c.obj, n, torch.zeros(2, 0, dtype=torch.int32, device="cuda"), n)
    pool = torch.zeros(8 * 2 * 16 * 64 + 8, dtype=torch.uint8, device="cuda")[8:].view(8, 2, 16, 64).view(torch.float8_e4m3fn)
    s8 = torch.zeros(8, 2, 16, dtype=torch.uint8, device="cuda")
    with pytest.raises(fa.FaError) as e:
        fa.flash_attention_decode(q, fa.PagedKV(pool, pool, c.obj.page_table, k_scale=s8, v_scale=s8), n)
    assert e.value.code == fa.FA_ERR_ALIGN
    assert _status() == 0


def test_front_page_tree_runs():
    """The front page's step over an 8-bit cache, behind the blocks before it, as written there."""
    import re
    from pathlib import Path
    import torch
    import attention_forward_fa_gb300 as fa
    text = (Path(__file__).resolve().parents[1] / "README.md").read_text()
    blocks = [b for b in re.findall(r"```python\n(.*?)```", text, re.S) if "paged_kv_append" in b]
    env = {"torch": torch, "fa": fa}
    torch.manual_seed(31)
    for i, b in enumerate(blocks):
        if "paged_kv_keep" in b:
            b, rest = b.split("path = ")
            exec(compile(b, f"serving-example-{i}", "exec"), env)

            class Now:
                fmt, D = "e4m3fn", 128
            c = Now()
            (c.kc, c.vc), (c.ke, c.ve) = ([_host(t) for t in env["codes"]], [t.cpu().numpy().astype(np.int64) - 127 for t in env["scales"]])
            c.k, c.v = np.ldexp(c.kc, c.ke[..., None]), np.ldexp(c.vc, c.ve[..., None])
            t, q = env["table"].cpu().numpy(), _host(env["qt"])
            tree = (env["sees"].cpu().numpy()[None].repeat(2, 0), [8, 8])
            a = (t, [1008, 45], 128 ** -0.5)
            _check8(env["ot"], env["lt"], P.decode(q, c.k, c.v, *a, tree=tree), *_spread(c, q, *a, tree), "bf16")
            exec(compile("path = " + rest, f"serving-example-{i}", "exec"), env)
            (c.k, c.v), _, _ = P.keep([c.k, c.v], t, [1000, 37], env["path"].cpu().numpy(), [3, 2], 64)
            k, v = P.read(c.k, c.v, t, [0, 0], [1003, 39], *(np.zeros((2, 8, 1003, 128)) for _ in range(2)))
            for seq, n in ((0, 1003), (1, 39)):
                assert np.array_equal(_host(env["k16"])[seq, :, :n], k[seq, :, :n])
                assert np.array_equal(_host(env["v16"])[seq, :, :n], v[seq, :, :n])
        else:
            exec(compile(b, f"serving-example-{i}", "exec"), env)
