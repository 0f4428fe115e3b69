"""GPU parity of the operators over a paged key-value cache (fa_kv_append,
fa_decode, fa_select_pages) against the fp64 reference of oracle/paged.py.

Bounds, with u the type's half step (2^-8 bf16, 2^-11 fp16; relative to the
value at most):
  * a rotated channel a cos - b sin is three fp32 roundings, so that
    |x - ref| <= u |ref| + (1 + u) 3 2^-24 (|a cos| + |b sin|), plus half the
    smallest subnormal of fp16;
  * a score is an fp32 sum of D <= 128 products: its error is at most
    e_s = 2^-16 X with X = max_j scale sum_d |q_d k_jd| (128 steps of 2^-23
    each: the tensor core may truncate);
  * a probability is off by the error of its score, of the running maximum's
    subtraction (2^-22 of the largest |score|, itself <= X) and of the
    exponential and the hi + lo split of P (2^-16 together), so that
    |O - ref| <= (2 e_s + 2^-20 X + 2^-15) A + (u + 2^-20) |ref| with
    A = sum_j p_j |v_j| (numerator and denominator: twice).  An fp16 P has an
    absolute error of up to 2^-25 besides (its subnormals), where the largest P
    of the row is at least 2^7: 2^-32 sum_j |v_j| more;
  * |LSE - ref| <= e_s + 2^-21 X + 2^-20 (1 + |ref|).
Whole numbers and untouched memory are equal bit for bit."""
import math

import numpy as np
import pytest

from oracle import paged as P

pytestmark = pytest.mark.gpu

U = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11}
SUB = {"bf16": 0.0, "fp16": 2.0 ** -25}


@pytest.fixture(scope="module", autouse=True)
def built():
    from attention_forward_fa_gb300 import build
    build.build()


def _torch_type(dtype):
    import torch
    return torch.bfloat16 if dtype == "bf16" else torch.float16


def _dev(x, dtype=None):
    """float64 values, representable in `dtype`, on the GPU (int arrays as they are)."""
    import torch
    t = torch.from_numpy(np.ascontiguousarray(x)).cuda()
    return t if dtype is None else t.to(_torch_type(dtype))


def _round(x, dtype):
    import torch
    return torch.from_numpy(np.ascontiguousarray(x)).to(torch.float32).to(_torch_type(dtype)).double().numpy()


def _host(t):
    return t.double().cpu().numpy()


def _status():
    import attention_forward_fa_gb300 as fa
    return fa.fa_check_status()


class Cache:
    """A random cache on both sides: pools (pages in random order), table, lengths."""

    def __init__(self, seed, dtype, B, Hkv, D, page, cap, layout="hnd", spare=3, bounds=False, stale=0.0):
        import torch
        import attention_forward_fa_gb300 as fa
        self.rng = rng = np.random.default_rng(seed)
        self.dtype, self.B, self.Hkv, self.D, self.page = dtype, B, Hkv, D, page
        need = [-(-c // page) for c in cap]
        num = sum(need) + spare
        order = rng.permutation(num)
        self.table = np.full((B, max(max(need), 1)), -1, dtype=np.int32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = order[at:at + n]
            at += n
        self.k = _round(rng.standard_normal((num, Hkv, page, D)), dtype)
        self.v = _round(rng.standard_normal((num, Hkv, page, D)), dtype)
        if stale:                     # what no sequence owns
            self.k[order[at:]] = stale
            self.v[order[at:]] = stale
        tk, tv = _dev(self.k, dtype), _dev(self.v, dtype)
        if layout == "nhd":           # [num, page, Hkv, D] pools
            tk, tv = (t.transpose(1, 2).contiguous().transpose(1, 2) for t in (tk, tv))
        elif layout == "halves":      # K and V of a page side by side in one pool, rows padded by 8
            both = torch.zeros(num, 2, Hkv, page, D + 8, dtype=tk.dtype, device="cuda")
            both[:, 0, ..., :D], both[:, 1, ..., :D] = tk, tv
            tk, tv = both[:, 0, ..., :D], both[:, 1, ..., :D]
        self.tk, self.tv = tk, tv
        self.lo = self.hi = self.tlo = self.thi = None
        if bounds:
            self.lo, self.hi = self.k.min(2), self.k.max(2)
            self.tlo, self.thi = _dev(self.lo, dtype), _dev(self.hi, dtype)
        self.obj = fa.PagedKV(tk, tv, _dev(self.table), self.tlo, self.thi)

    def ints(self, x):
        return _dev(np.asarray(x, dtype=np.int32))


def _tables(n, r):
    a = np.arange(n)[:, None] * 10000.0 ** (-np.arange(0, r, 2) / r)
    return np.cos(a).astype(np.float32), np.sin(a).astype(np.float32)


# ------------------------------------------------------------------ append
APPEND = [
    # dtype, B, Hq, Hkv, D, page, S, old, new, rot, interleaved, layout
    ("bf16", 1, 4, 1, 128, 64, 1, [0], [1], 128, False, "hnd"),
    ("bf16", 3, 32, 8, 128, 64, 1, [63, 64, 517], [1, 1, 1], 128, False, "nhd"),
    ("fp16", 5, 6, 6, 64, 16, 1, [0, 15, 16, 17, 300], [1, 0, 1, 1, 1], 32, True, "halves"),
    ("bf16", 2, 8, 2, 64, 32, 2, [31, 5], [2, 1], 64, True, "hnd"),
    ("fp16", 3, 40, 5, 128, 16, 37, [0, 3, 15], [37, 20, 0], 64, False, "nhd"),
    ("bf16", 2, 3, 3, 128, 256, 300, [250, 0], [300, 257], 128, True, "hnd"),
    ("bf16", 2, 16, 16, 64, 128, 129, [100, 127], [129, 65], 0, False, "halves"),
    ("fp16", 1, 33, 1, 64, 64, 70, [7], [70], 16, False, "hnd"),
    ("bf16", 1, 72, 9, 128, 32, 3, [30], [3], 112, True, "nhd"),
    # much room, few tokens: a block looks for its pieces
    ("bf16", 16, 1, 1, 64, 16, 4096, [5, 0] + [100] * 14, [900, 0, 4096, 33] + [1] * 12, 64, False, "hnd"),
    ("fp16", 26, 1, 1, 128, 16, 2048, [15] * 25 + [0], [2, 2048] + [1, 0] * 12, 32, True, "nhd"),
]


@pytest.mark.parametrize("case", APPEND, ids=lambda c: "-".join(map(str, c[:7])))
@pytest.mark.parametrize("form", ["plain", "fused_in_place"])
def test_append(case, form):
    import torch
    import attention_forward_fa_gb300 as fa
    dtype, B, Hq, Hkv, D, page, S, old, new, rot, inter, layout = case
    c = Cache(1, dtype, B, Hkv, D, page, [o + n for o, n in zip(old, new)], layout, bounds=True)
    rng = c.rng
    q, k, v = (_round(rng.standard_normal((B, h, S, D)), dtype) for h in (Hq, Hkv, Hkv))
    cos, sin = _tables(max(o + n for o, n in zip(old, new)) + 1, rot) if rot else (None, None)
    kw = dict(cos=_dev(cos), sin=_dev(sin)) if rot else {}
    lens, n = c.ints(old), c.ints(new)
    if form == "plain":
        tq, tk, tv = _dev(q, dtype), _dev(k, dtype), _dev(v, dtype)
        mark = _round(rng.standard_normal(q.shape), dtype)
        qo = _dev(mark, dtype)
    else:   # one [B, S, heads, D] projection; queries rotated in place
        x = _dev(np.concatenate((q, k, v), 1), dtype).transpose(1, 2).contiguous().transpose(1, 2)
        tq, tk, tv = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
        mark, qo = q, tq
    got = fa.paged_kv_append(c.obj, lens, tk, tv, new_lens=n, q=tq, q_out=qo, interleaved=inter, **kw)
    assert got is qo and _status() == 0
    # what the roundings see, and what bounds their errors
    ek, ev, _, _ = P.append(c.k, c.v, c.table, old, k, v, new, cos, sin, inter)
    mag = {}
    for name, x in (("q", q), ("k", k)):
        m = np.zeros_like(x)
        if rot:
            ia = np.arange(0, rot, 2) if inter else np.arange(rot // 2)
            ib = ia + (1 if inter else rot // 2)
            for b in range(B):
                p = np.minimum(old[b] + np.arange(S), cos.shape[0] - 1)
                cc, ss = np.abs(cos[p]), np.abs(sin[p])
                a, d = np.abs(x[b][..., ia]), np.abs(x[b][..., ib])
                m[b][..., ia], m[b][..., ib] = a * cc + d * ss, a * ss + d * cc
        mag[name] = m
    mk = P.append(np.zeros_like(c.k), np.zeros_like(c.v), c.table, old, mag["k"], v, new)[0]
    u = U[dtype]
    gk, gv = _host(c.tk), _host(c.tv)
    assert np.array_equal(gv, ev)
    wrote = np.zeros(c.k.shape, dtype=bool)
    for b in range(B):
        for t in range(old[b], old[b] + new[b]):
            wrote[c.table[b, t // page], :, t % page] = True
    assert np.array_equal(gk[~wrote], c.k[~wrote])
    bound = u * np.abs(ek) + (1 + u) * 3 * 2.0 ** -24 * mk + SUB[dtype]
    assert (np.abs(gk - ek) <= bound)[wrote].all()
    gq = _host(qo)
    for b in range(B):
        p = old[b] + np.arange(new[b])
        ref = P.rotate(q[b][:, :new[b]], p, cos, sin, inter) if rot else q[b][:, :new[b]]
        lim = u * np.abs(ref) + (1 + u) * 3 * 2.0 ** -24 * mag["q"][b][:, :new[b]] + SUB[dtype]
        assert (np.abs(gq[b][:, :new[b]] - ref) <= (lim if rot else 0)).all()
        assert np.array_equal(gq[b][:, new[b]:], mark[b][:, new[b]:])       # padding rows as they were
    # bounds of the touched pages: those of the keys as stored; the others as they were
    lo, hi = c.lo.copy(), c.hi.copy()
    for b in range(B):
        for p in range(old[b] // page, -(-(old[b] + new[b]) // page)):
            a, z = max(old[b], p * page) - p * page, min(old[b] + new[b], (p + 1) * page) - p * page
            if z <= a:
                continue
            i = c.table[b, p]
            l, h = gk[i, :, a:z].min(1), gk[i, :, a:z].max(1)
            lo[i], hi[i] = (l, h) if a == 0 else (np.minimum(l, lo[i]), np.maximum(h, hi[i]))
    assert np.array_equal(_host(c.tlo), lo) and np.array_equal(_host(c.thi), hi)
    torch.cuda.synchronize()


def test_append_without_queries_bounds_or_lengths():
    import attention_forward_fa_gb300 as fa
    c = Cache(2, "bf16", 2, 2, 64, 16, [20, 20])
    k, v = (_round(c.rng.standard_normal((2, 2, 20, 64)), "bf16") for _ in range(2))
    assert fa.paged_kv_append(c.obj, c.ints([0, 0]), _dev(k, "bf16"), _dev(v, "bf16")) is None
    assert _status() == 0
    ek, ev, _, _ = P.append(c.k, c.v, c.table, [0, 0], k, v, [20, 20])
    assert np.array_equal(_host(c.tk), ek) and np.array_equal(_host(c.tv), ev)


def test_append_leaves_out_what_has_no_place():
    """A page id outside the pool, a position past the table or the angles, a
    length outside: those tokens are left out, the others written, and the
    status says so."""
    import attention_forward_fa_gb300 as fa
    c = Cache(3, "bf16", 4, 1, 64, 16, [32, 32, 32, 32], bounds=True)
    num = c.k.shape[0]
    c.table[1, 1] = num          # one past the pool
    c.table[2, 1] = -5
    c.obj.page_table.copy_(_dev(c.table))
    k, v = (_round(c.rng.standard_normal((4, 1, 20, 64)), "bf16") for _ in range(2))
    old = [0, 0, 0, 25]          # the last: tokens 25..44 in a table of 32
    fa.paged_kv_append(c.obj, c.ints(old), _dev(k, "bf16"), _dev(v, "bf16"))
    assert _status() == fa.FA_ERR_INDEX and _status() == 0
    ek, ev, _, _ = P.append(c.k, c.v, c.table, old, k, v, [20, 16, 16, 7])
    assert np.array_equal(_host(c.tk), ek) and np.array_equal(_host(c.tv), ev)
    cos, sin = _tables(10, 64)
    c = Cache(4, "bf16", 3, 1, 64, 16, [32, 32, 32])
    x = _dev(k[:3], "bf16")
    fa.paged_kv_append(c.obj, c.ints([0, 9, 30]), x, x, new_lens=c.ints([20, 25, -1]), cos=_dev(cos), sin=_dev(sin))
    assert _status() == fa.FA_ERR_INDEX
    ek, ev, _, _ = P.append(c.k, c.v, c.table, [0, 9, 30], k[:3], k[:3], [10, 1, 0], cos, sin)
    assert np.array_equal(_host(c.tv), ev)
    assert np.abs(_host(c.tk) - ek).max() <= 2.0 ** -8 * np.abs(ek).max()
    was = c.tk.clone()
    fa.paged_kv_append(c.obj, c.ints([-1, 0, 1 << 30]), x, x, new_lens=c.ints([1, 0, 1]))
    assert _status() == fa.FA_ERR_INDEX
    assert bool((c.tk == was).all())


# ------------------------------------------------------------------ decode
DECODE = [
    # dtype, B, Hq, Hkv, D, page, Sq, lens, pre, layout
    ("bf16", 1, 1, 1, 128, 16, 1, [1], None, "hnd"),
    ("bf16", 4, 8, 2, 128, 64, 1, [0, 1, 63, 64], None, "hnd"),
    ("fp16", 3, 4, 4, 64, 16, 1, [15, 17, 1000], None, "nhd"),
    ("bf16", 2, 32, 8, 128, 64, 1, [517, 3001], None, "halves"),
    ("bf16", 1, 12, 4, 64, 256, 1, [777], None, "hnd"),
    ("fp16", 2, 40, 8, 128, 32, 1, [129, 31], None, "nhd"),
    ("bf16", 2, 24, 2, 128, 128, 1, [700, 5], None, "hnd"),
    ("bf16", 3, 32, 1, 128, 64, 1, [900, 64, 1], None, "hnd"),
    ("fp16", 1, 71, 1, 64, 16, 1, [530], None, "halves"),
    ("bf16", 3, 8, 2, 128, 64, 5, [700, 3, 66], None, "hnd"),
    ("fp16", 2, 16, 2, 64, 16, 7, [6, 515], None, "nhd"),
    ("bf16", 2, 6, 6, 128, 32, 2, [65, 1], None, "hnd"),
    ("bf16", 3, 8, 2, 128, 64, 1, [700, 64, 3], 100, "hnd"),
    ("bf16", 3, 8, 2, 64, 16, 5, [700, 64, 3], 100, "hnd"),
    ("fp16", 2, 4, 1, 128, 128, 3, [1000, 130], 0, "nhd"),
    ("bf16", 1, 4, 1, 128, 64, 1, [20000], None, "hnd"),
    ("bf16", 2, 64, 1, 128, 64, 1, [300, 33], None, "hnd"),
    ("fp16", 1, 16, 2, 128, 32, 8, [260], None, "nhd"),
    ("fp16", 2, 56, 1, 64, 16, 1, [300, 17], None, "hnd"),
    ("bf16", 1, 8, 1, 64, 128, 17, [150], 40, "halves"),
    ("bf16", 1, 20, 1, 128, 16, 2, [99], None, "hnd"),
    ("bf16", 1, 128, 1, 128, 256, 1, [500], None, "hnd"),
    ("fp16", 2, 16, 16, 64, 16, 1, [5000, 4999], 4097, "hnd"),
    ("bf16", 3, 8, 2, 128, 64, 150, [400, 151, 100], None, "nhd"),       # a chunk of a prompt
    ("fp16", 1, 6, 2, 64, 32, 333, [333], 64, "hnd"),
]


def _check(got_o, got_l, ref, dtype, where=""):
    O, L, A, X, V = ref
    o, l = _host(got_o), _host(got_l)
    u = U[dtype]
    empty = np.isposinf(L)
    assert np.array_equal(np.isposinf(l), empty), f"{where}: rows without keys"
    assert (o[empty] == 0).all()
    es = 2.0 ** -16 * X
    lim = (2 * es + 2.0 ** -20 * X + 2.0 ** -15)[..., None] * A + (u + 2.0 ** -20) * np.abs(O) + SUB[dtype]
    lim += (2.0 ** -32 if dtype == "fp16" else 0.0) * V
    err = np.abs(o - O)
    assert (err <= lim).all(), f"{where}: O off by {(err / np.maximum(lim, 1e-30)).max():.3g} of its bound"
    le = np.abs(l[~empty] - L[~empty])
    ll = (es + 2.0 ** -21 * X)[~empty] + 2.0 ** -20 * (1 + np.abs(L[~empty]))
    assert (le <= ll).all(), f"{where}: LSE off by {(le / ll).max():.3g} of its bound"


@pytest.mark.parametrize("case", DECODE, ids=lambda c: "-".join(map(str, c[:7])) + ("" if c[8] is None else f"-w{c[8]}"))
def test_decode(case):
    import attention_forward_fa_gb300 as fa
    dtype, B, Hq, Hkv, D, page, Sq, lens, pre, layout = case
    c = Cache(5, dtype, B, Hkv, D, page, lens, layout)
    q = _round(c.rng.standard_normal((B, Hq, Sq, D)), dtype)
    o, l = fa.flash_attention_decode(_dev(q, dtype), c.obj, c.ints(lens), pre_tokens=pre)
    assert _status() == 0
    _check(o, l, P.decode(q, c.k, c.v, c.table, lens, 1 / math.sqrt(D), pre), dtype, str(case))


@pytest.mark.parametrize("scale", [0.0, -0.2, 1.0, 5.0])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_decode_scales_and_peaks(dtype, scale):
    """Scores from flat to one-hot, and a negative scale; a channel whose values
    are 0 at the keys that matter shows the small probabilities."""
    import attention_forward_fa_gb300 as fa
    lens = [300, 33]
    c = Cache(6, dtype, 2, 2, 128, 32, lens)
    q = _round(c.rng.standard_normal((2, 8, 1, 128)), dtype)
    s = np.einsum("hd,kd->hk", q[0, :4, 0], c.k[c.table[0], 0].reshape(-1, 128)[:300])
    v = c.v[c.table[0], 0].reshape(-1, 128)
    v[np.unique(np.argsort(-abs(scale) * s, axis=1)[:, :2]), 5] = 0
    c.v[c.table[0], 0] = v.reshape(-1, 32, 128)
    c.tv.copy_(_dev(c.v, dtype))
    o, l = fa.flash_attention_decode(_dev(q, dtype), c.obj, c.ints(lens), scale=scale)
    assert _status() == 0
    _check(o, l, P.decode(q, c.k, c.v, c.table, lens, scale), dtype, f"scale {scale}")


def test_decode_growing_scores():
    """Keys of ever larger scores: the reference of every row moves many times,
    in the middle of the pieces and between them, and never by too little."""
    import attention_forward_fa_gb300 as fa
    for dtype, step in (("bf16", 0.02), ("fp16", 0.02), ("fp16", 0.3), ("bf16", -0.05)):
        lens = [1500]
        c = Cache(29, dtype, 1, 1, 64, 64, lens)
        k = c.k[c.table[0], 0].reshape(-1, 64)
        k[:, 0] = _round(np.arange(k.shape[0]) * step, dtype)
        c.k[c.table[0], 0] = k.reshape(-1, 64, 64)
        c.tk.copy_(_dev(c.k, dtype))
        q = _round(0.1 * c.rng.standard_normal((1, 4, 1, 64)), dtype)
        q[..., 0] = np.array([1.0, 0.5, -1.0, 0.0])[None, :, None]
        o, l = fa.flash_attention_decode(_dev(q, dtype), c.obj, c.ints(lens), scale=1.0)
        assert _status() == 0
        _check(o, l, P.decode(q, c.k, c.v, c.table, lens, 1.0), dtype, f"{dtype} {step}")


@pytest.mark.parametrize("dtype,Sq,pre", [("bf16", 1, None), ("fp16", 1, 20), ("bf16", 4, 37), ("fp16", 3, None)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -65504.0])
def test_decode_never_uses_what_no_row_sees(dtype, Sq, pre, bad):
    """Slots behind the last token, tokens before the window and pages that
    belong to no sequence hold anything."""
    import attention_forward_fa_gb300 as fa
    lens, page = [70, 64, 16, 129], 32
    c = Cache(7, dtype, 4, 2, 64, page, lens)
    q = _round(c.rng.standard_normal((4, 4, Sq, 64)), dtype)
    ref = P.decode(q, c.k, c.v, c.table, lens, 0.125, pre)
    seen = np.zeros(c.k.shape[:1] + (page,), dtype=bool)
    for b, n in enumerate(lens):
        low = 0 if pre is None else max(0, n - Sq - pre)
        for t in range(low, n):
            seen[c.table[b, t // page], t % page] = True
    import torch
    hide = _dev(~seen)[:, None, :, None]
    c.tk.masked_fill_(hide, bad)
    c.tv.masked_fill_(hide, bad)
    o, l = fa.flash_attention_decode(_dev(q, dtype), c.obj, c.ints(lens), scale=0.125, pre_tokens=pre)
    assert _status() == 0
    _check(o, l, ref, dtype)
    torch.cuda.synchronize()


@pytest.mark.parametrize("dtype,B,Hq,Hkv,D,page,Sq,lens,sel", [
    ("bf16", 2, 8, 2, 128, 64, 1, [1000, 300], 3), ("fp16", 1, 4, 4, 64, 16, 1, [3000], 40),
    ("bf16", 3, 8, 1, 64, 256, 3, [1000, 1, 257], 2), ("bf16", 1, 16, 4, 128, 32, 1, [5000], 100),
    ("fp16", 2, 4, 2, 128, 128, 1, [129, 0], 5), ("bf16", 4, 8, 2, 64, 16, 2, [100, 17, 700, 3], 60),
])
def test_decode_listed_pages(dtype, B, Hq, Hkv, D, page, Sq, lens, sel):
    """Lists in any order, with invalid slots, repeats and an empty one, longer
    than their sequences too."""
    import attention_forward_fa_gb300 as fa
    c = Cache(8, dtype, B, Hkv, D, page, lens)
    wide = c.table.shape[1]
    idx = c.rng.integers(-1, wide + 2, (B, Hkv, sel)).astype(np.int32)
    idx[0, 0, -1] = idx[0, 0, 0]
    if Hkv > 1:
        idx[0, 1] = -1
    idx[0, 0, 0] = 2 ** 31 - 1
    q = _round(c.rng.standard_normal((B, Hq, Sq, D)), dtype)
    o, l = fa.flash_attention_decode(_dev(q, dtype), c.obj, c.ints(lens), page_idx=_dev(idx))
    assert _status() == 0
    _check(o, l, P.decode(q, c.k, c.v, c.table, lens, 1 / math.sqrt(D), None, idx), dtype)


@pytest.mark.parametrize("dtype,Hq,Hkv,D,page,Sq,pre,sel", [
    ("bf16", 8, 4, 128, 64, 1, None, 0), ("fp16", 6, 6, 64, 16, 1, None, 0), ("bf16", 12, 1, 128, 32, 1, None, 0),
    ("bf16", 20, 2, 128, 16, 2, None, 0), ("fp16", 8, 4, 128, 256, 5, 300, 0), ("bf16", 8, 4, 64, 64, 1, None, 7),
    ("fp16", 32, 2, 64, 128, 3, None, 0),
])
def test_decode_many_units_per_block(dtype, Hq, Hkv, D, page, Sq, pre, sel):
    """70 sequences of mixed lengths: every block of the grid takes several
    units, whole ones and pieces of shared ones, many tiles each."""
    import attention_forward_fa_gb300 as fa
    rng = np.random.default_rng(20)
    lens = [int(x) for x in rng.integers(0, 1500, 70)]
    lens[3], lens[40], lens[69] = 0, 1, 2900
    c = Cache(21, dtype, 70, Hkv, D, page, lens)
    q = _round(c.rng.standard_normal((70, Hq, Sq, D)), dtype)
    idx = None
    if sel:
        idx = np.sort(c.rng.integers(-3, c.table.shape[1], (70, Hkv, sel)).astype(np.int32), -1)
    o, l = fa.flash_attention_decode(_dev(q, dtype), c.obj, c.ints(lens), pre_tokens=pre,
                                     page_idx=None if idx is None else _dev(idx))
    assert _status() == 0
    _check(o, l, P.decode(q, c.k, c.v, c.table, lens, D ** -0.5, pre, idx), dtype)


@pytest.mark.parametrize("pre", [0, 50, 400])
def test_decode_listed_pages_in_a_window(pre):
    import attention_forward_fa_gb300 as fa
    lens, page = [700, 64, 3], 32
    c = Cache(22, "bf16", 3, 2, 128, page, lens)
    idx = c.rng.integers(-1, c.table.shape[1], (3, 2, 12)).astype(np.int32)
    idx[0, 0, :3] = [21, 20, 21]           # the newest page twice
    q = _round(c.rng.standard_normal((3, 8, 3, 128)), "bf16")
    o, l = fa.flash_attention_decode(_dev(q, "bf16"), c.obj, c.ints(lens), page_idx=_dev(idx), pre_tokens=pre)
    assert _status() == 0
    _check(o, l, P.decode(q, c.k, c.v, c.table, lens, 128 ** -0.5, pre, idx), "bf16")


def test_decode_more_sequences_than_one_look_up():
    """700 sequences, empty ones among them: the lengths come in several rounds."""
    import attention_forward_fa_gb300 as fa
    rng = np.random.default_rng(23)
    lens = [int(x) for x in rng.integers(0, 90, 700)]
    lens[300] = 2000
    c = Cache(24, "fp16", 700, 1, 64, 16, lens)
    q = _round(c.rng.standard_normal((700, 2, 1, 64)), "fp16")
    o, l = fa.flash_attention_decode(_dev(q, "fp16"), c.obj, c.ints(lens))
    assert _status() == 0
    _check(o, l, P.decode(q, c.k, c.v, c.table, lens, 0.125), "fp16")


@pytest.mark.parametrize("B,Hq", [(300, 1), (1300, 1), (513, 5)])
def test_decode_joins_among_many_sequences(B, Hq):
    """More sequences than one look-up holds, a few of them long: their pieces
    are joined by blocks whose rows belong to one sequence or to several."""
    import attention_forward_fa_gb300 as fa
    rng = np.random.default_rng(B)
    lens = [int(x) for x in rng.integers(0, 40, B)]
    for b in (0, 1, 255, 256, B - 1):
        lens[b] = 900 + b
    c = Cache(25, "bf16", B, 1, 64, 32, lens)
    q = _round(c.rng.standard_normal((B, Hq, 1, 64)), "bf16")
    o, l = fa.flash_attention_decode(_dev(q, "bf16"), c.obj, c.ints(lens))
    assert _status() == 0
    _check(o, l, P.decode(q, c.k, c.v, c.table, lens, 0.125), "bf16")


def test_two_streams_at_once():
    """Eager calls of all three operators on two streams, each with scratch of its own."""
    import torch
    import attention_forward_fa_gb300 as fa
    cs = [Cache(25 + i, "bf16", 2, 4, 128, 64, [4000, 900], bounds=True) for i in range(2)]
    qs = [_dev(_round(c.rng.standard_normal((2, 16, 1, 128)), "bf16"), "bf16") for c in cs]
    n = cs[0].ints([3999, 899])
    want = [(fa.flash_attention_decode(q, c.obj, n), fa.select_kv_pages(q, c.obj, n, 20)) for q, c in zip(qs, cs)]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(2)], [[], []]
    for _ in range(30):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i].append((fa.flash_attention_decode(qs[i], cs[i].obj, n), fa.select_kv_pages(qs[i], cs[i].obj, n, 20)))
    torch.cuda.synchronize()
    for i in range(2):
        for (o, l), idx in got[i]:
            assert torch.equal(o, want[i][0][0]) and torch.equal(l, want[i][0][1]) and torch.equal(idx, want[i][1])
    assert _status() == 0


def test_decode_leaves_out_bad_pages():
    """A page id outside the pool: its keys are masked, the status says so; the
    other sequences are as they would be."""
    import attention_forward_fa_gb300 as fa
    lens = [100, 100, 100]
    c = Cache(9, "bf16", 3, 2, 128, 16, lens)
    q = _round(c.rng.standard_normal((3, 4, 1, 128)), "bf16")
    c.table[0, 2], c.table[1, 6] = c.k.shape[0], -1
    c.obj.page_table.copy_(_dev(c.table))
    o, l = fa.flash_attention_decode(_dev(q, "bf16"), c.obj, c.ints(lens))
    assert _status() == fa.FA_ERR_INDEX and _status() == 0
    idx = np.tile(np.arange(7, dtype=np.int32), (3, 2, 1))
    idx[0, :, 2], idx[1, :, 6] = -1, -1
    _check(o, l, P.decode(q, c.k, c.v, c.table, lens, 128 ** -0.5, None, idx), "bf16")
    o, l = fa.flash_attention_decode(_dev(q, "bf16"), c.obj, c.ints([-3, 200000, 100]))
    assert _status() == fa.FA_ERR_INDEX
    assert bool((o[:2] == 0).all()) and bool((l[:2] == math.inf).all())


def test_decode_is_repeatable_and_fills_given_outputs():
    import torch
    import attention_forward_fa_gb300 as fa
    lens = [4000, 2500, 1, 0]
    c = Cache(10, "bf16", 4, 4, 128, 64, lens)
    q = _dev(_round(c.rng.standard_normal((4, 16, 1, 128)), "bf16"), "bf16")
    n = c.ints(lens)
    o, l = fa.flash_attention_decode(q, c.obj, n)
    o2, l2 = torch.empty_like(o), torch.empty_like(l)
    for _ in range(3):
        r = fa.flash_attention_decode(q, c.obj, n, out=o2, lse=l2)
        assert r[0] is o2 and r[1] is l2
        assert torch.equal(o, o2) and torch.equal(l, l2)
    # a sequence's answer does not depend on the others
    one = fa.PagedKV(c.tk, c.tv, c.obj.page_table[:1].contiguous())
    o3, l3 = fa.flash_attention_decode(q[:1].contiguous(), one, n[:1].contiguous())
    _check(o3, l3, P.decode(_host(q)[:1], c.k, c.v, c.table[:1], lens[:1], 128 ** -0.5), "bf16")
    assert _status() == 0


def test_decode_beyond_32_bit_offsets():
    """A pool of more than 2^31 elements; the sequence's pages lie at its end."""
    import torch
    import attention_forward_fa_gb300 as fa
    Hkv, page, D = 8, 64, 128
    num = 2 ** 31 // (Hkv * page * D) + 40
    rng = np.random.default_rng(11)
    k = torch.empty(num, Hkv, page, D, dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    table = np.arange(num - 1, num - 21, -1, dtype=np.int32)[None]
    lens = [1250]
    kk, vv = (_round(rng.standard_normal((20, Hkv, page, D)), "bf16") for _ in range(2))
    cache = fa.PagedKV(k, v, _dev(table))
    x = _dev(kk, "bf16").transpose(0, 1).reshape(1, Hkv, 20 * page, D).contiguous()
    y = _dev(vv, "bf16").transpose(0, 1).reshape(1, Hkv, 20 * page, D).contiguous()
    fa.paged_kv_append(cache, _dev(np.zeros(1, dtype=np.int32)), x, y)
    assert torch.equal(k[num - 20:].flip(0), _dev(kk, "bf16")) and torch.equal(v[num - 20:].flip(0), _dev(vv, "bf16"))
    q = _round(rng.standard_normal((1, 16, 1, D)), "bf16")
    o, l = fa.flash_attention_decode(_dev(q, "bf16"), cache, _dev(np.array(lens, dtype=np.int32)))
    assert _status() == 0
    flat = np.arange(20, dtype=np.int32)[None]
    _check(o, l, P.decode(q, kk, vv, flat, lens, D ** -0.5), "bf16")


# ------------------------------------------------------------------ choice of pages
SELECT = [
    # dtype, B, Hq, Hkv, D, page, Sq, lens, max_sel, first, last
    ("bf16", 2, 8, 2, 128, 64, 1, [5000, 130], 8, 1, 1),
    ("fp16", 3, 4, 4, 64, 16, 1, [0, 1, 3000], 17, 1, 1),
    ("bf16", 1, 5, 1, 128, 32, 1, [4097], 1, 0, 0),
    ("bf16", 2, 16, 2, 64, 128, 3, [9000, 8999], 20, 0, 4),
    ("fp16", 1, 40, 1, 128, 16, 2, [2000], 100, 3, 0),
    ("bf16", 1, 2, 2, 64, 256, 1, [1000], 64, 2, 3),
    ("bf16", 2, 2, 1, 64, 16, 1, [40000, 20001], 33, 1, 1),
    ("fp16", 1, 8, 8, 128, 16, 1, [1600], 99, 1, 1),
    ("bf16", 1, 2, 1, 128, 16, 1, [150000], 200, 1, 1),
]


@pytest.mark.parametrize("case", SELECT, ids=lambda c: "-".join(map(str, c[:7])))
def test_select(case):
    import attention_forward_fa_gb300 as fa
    dtype, B, Hq, Hkv, D, page, Sq, lens, M, first, last = case
    c = Cache(12, dtype, B, Hkv, D, page, lens, bounds=True)
    q = _round(c.rng.standard_normal((B, Hq, Sq, D)), dtype)
    got = fa.select_kv_pages(_dev(q, dtype), c.obj, c.ints(lens), M, first=first, last=last)
    assert _status() == 0
    assert np.array_equal(got.cpu().numpy(), P.select(q, c.lo, c.hi, c.table, lens, page, M, first, last))


def test_select_ties_and_near_ties():
    """Equal scores go to the lower page; scores that differ by far less than
    fp32 resolves are told apart."""
    import attention_forward_fa_gb300 as fa
    D, n, M = 128, 200, 50
    c = Cache(13, "bf16", 1, 1, D, 16, [n * 16], bounds=True)
    q = np.ones((1, 2, 1, D))
    q[0, 1] = -1.0
    lo, hi = np.zeros_like(c.lo), np.zeros_like(c.hi)
    hi[:, 0, 0] = 4096.0                              # all pages alike
    rank = c.rng.permutation(n)
    for case in ("equal", "near"):
        if case == "near":                            # 4096 + r 2^-30, r a permutation
            for p in range(n):
                hi[c.table[0, p], 0, 1] = rank[p] * 2.0 ** -30
        c.tlo.copy_(_dev(lo, "bf16"))
        c.thi.copy_(_dev(hi, "bf16"))
        got = fa.select_kv_pages(_dev(q, "bf16"), c.obj, c.ints([n * 16]), M)
        assert _status() == 0
        assert np.array_equal(got.cpu().numpy(), P.select(q, lo, hi, c.table, [n * 16], 16, M)), case


def test_select_many_near_the_threshold():
    """Pages that differ past fp32 only, more of them than are kept on chip, and
    more pages than scores are kept: all told apart in 64 bits."""
    import attention_forward_fa_gb300 as fa
    n, M = 9000, 700
    c = Cache(28, "bf16", 1, 1, 64, 16, [n * 16], bounds=True)
    q = np.ones((1, 1, 1, 64))
    lo, hi = np.zeros_like(c.lo), np.zeros_like(c.hi)
    hi[:, 0, 0] = 2.0 ** 20
    hi[:, 0, 1] = 2.0 ** -20 * c.rng.integers(0, 256, hi.shape[0])    # many ties as well
    hi[:, 0, 2] = 2.0 ** -28 * c.rng.integers(0, 256, hi.shape[0])
    c.tlo.copy_(_dev(lo, "bf16"))
    c.thi.copy_(_dev(hi, "bf16"))
    got = fa.select_kv_pages(_dev(q, "bf16"), c.obj, c.ints([n * 16]), M)
    assert _status() == 0
    assert np.array_equal(got.cpu().numpy(), P.select(q, lo, hi, c.table, [n * 16], 16, M))


@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("fp16", 64)])
def test_select_tables_with_room_to_spare(dtype, D):
    """Tables for 32768 pages, sequences of none to a few hundred (one as long as
    its table): the entries behind a sequence's last page may be anything."""
    import torch
    import attention_forward_fa_gb300 as fa
    room, Hkv, M = 32768, 3, 9
    c = Cache(31, dtype, 7, Hkv, D, 16, [0, 1, 16, 4000, 333, 5000, 64], bounds=True)
    table = torch.full((8, room), -7, device="cuda", dtype=torch.int32)
    table[:7, :c.table.shape[1]] = _dev(c.table)
    table[:7, c.table.shape[1]:] = 2 ** 31 - 1
    table[7] = torch.arange(room, device="cuda", dtype=torch.int32) % c.k.shape[0]
    cache = fa.PagedKV(c.tk, c.tv, table, c.tlo, c.thi)
    lens = [0, 1, 16, 4000, 333, 5000, 64, 16 * room]
    q = _round(c.rng.standard_normal((8, 2 * Hkv, 1, D)), dtype)
    got = fa.select_kv_pages(_dev(q, dtype), cache, c.ints(lens), M)
    assert _status() == 0
    assert np.array_equal(got.cpu().numpy(), P.select(q, c.lo, c.hi, table.cpu().numpy(), lens, 16, M))
    lens[2], lens[5] = -1, 16 * room + 1
    got = fa.select_kv_pages(_dev(q, dtype), cache, c.ints(lens), M)
    assert _status() == fa.FA_ERR_INDEX
    lens[2], lens[5] = 0, 0
    assert np.array_equal(got.cpu().numpy(), P.select(q, c.lo, c.hi, table.cpu().numpy(), lens, 16, M))


def test_select_pages_that_are_all_alike():
    """So many equal scores that a pairwise ranking would take seconds: the
    lowest page numbers among the equal, behind the few that are larger."""
    import torch
    import attention_forward_fa_gb300 as fa
    n, M = 131072, 300
    table = torch.randperm(64, device="cuda", dtype=torch.int32).repeat(n // 64).view(1, n)   # shared pages
    pool = torch.zeros(64, 1, 16, 64, device="cuda", dtype=torch.bfloat16)
    lo, hi = (torch.ones(64, 1, 64, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    cache = fa.PagedKV(pool, pool.clone(), table, lo, hi)
    q = torch.ones(1, 4, 1, 64, device="cuda", dtype=torch.bfloat16)
    lens = torch.tensor([16 * n], device="cuda", dtype=torch.int32)
    got = fa.select_kv_pages(q, cache, lens, M, first=2, last=3)
    assert _status() == 0
    assert got.flatten().tolist() == list(range(M - 3)) + [n - 3, n - 2, n - 1]
    best = int(table[0, 40])                          # one page of the pool, in 2048 places: less than
    hi[best, 0, 7] = 1.0 + 2.0 ** -7                  # fp32's error above the rest with 2^20 beside it
    lo[:, 0, 0] = hi[:, 0, 0] = 2.0 ** 20
    places = (table[0] == best).nonzero().flatten().tolist()
    got = fa.select_kv_pages(q, cache, lens, M, first=2, last=3)
    assert _status() == 0
    assert got.flatten().tolist() == [0, 1] + places[:M - 5] + [n - 3, n - 2, n - 1]


def test_select_lists_short_sequences_unscored():
    """At most max_sel pages: all of them, without a look at table or bounds."""
    import torch
    import attention_forward_fa_gb300 as fa
    c = Cache(32, "bf16", 2, 2, 64, 16, [320, 800], bounds=True)
    c.obj.page_table[0] = -7
    c.tlo[_dev(c.table[0, :20]).long()] = float("nan")
    q = _round(c.rng.standard_normal((2, 4, 1, 64)), "bf16")
    got = fa.select_kv_pages(_dev(q, "bf16"), c.obj, c.ints([320, 800]), 20).cpu().numpy()
    assert _status() == 0
    assert (got[0] == np.arange(20)).all()
    assert np.array_equal(got[1], P.select(q[1:], c.lo, c.hi, c.table[1:], [800], 16, 20)[0])
    torch.cuda.synchronize()


def test_select_extreme_bounds_and_bad_pages():
    """Sums past the fp32 range of a score, and page ids outside the pool: no
    page is listed twice or out of range."""
    import attention_forward_fa_gb300 as fa
    c = Cache(14, "bf16", 2, 1, 64, 16, [640, 640], bounds=True)
    c.tlo.fill_(-3e38)
    c.thi.fill_(3e38)
    q = _dev(np.full((2, 1, 1, 64), 3e38), "bf16")
    c.table[1, 5] = c.k.shape[0] + 7
    c.obj.page_table.copy_(_dev(c.table))
    got = fa.select_kv_pages(q, c.obj, c.ints([640, 640]), 10).cpu().numpy()
    assert _status() == fa.FA_ERR_INDEX
    assert list(got[0, 0]) == list(range(9)) + [39]
    assert len(set(got[1, 0])) == 10 and got.min() >= 0 and got.max() < 40


# ------------------------------------------------------------------ together
@pytest.mark.parametrize("dtype,D,page,inter", [("bf16", 128, 64, False), ("fp16", 64, 16, True)])
def test_serving_run(dtype, D, page, inter):
    """Prompts into the cache, then tokens one by one and three at once: each
    attends over what was appended; last over chosen pages."""
    import attention_forward_fa_gb300 as fa
    B, Hq, Hkv = 3, 8, 2
    prompt, total = [100, 1, 333], 345
    c = Cache(15, dtype, B, Hkv, D, page, [total] * B, bounds=True)
    cos, sin = _tables(total, D)
    tc, ts = _dev(cos), _dev(sin)
    lens = np.array(prompt) * 0

    def step(S, new):
        nonlocal lens
        x = _round(c.rng.standard_normal((B, Hq + 2 * Hkv, S, D)), dtype)
        t = _dev(x, dtype)
        q = fa.paged_kv_append(c.obj, c.ints(lens), t[:, Hq:Hq + Hkv], t[:, Hq + Hkv:], new_lens=c.ints(new),
                               q=t[:, :Hq], cos=tc, sin=ts, interleaved=inter)
        lens = lens + np.array(new)
        return q

    step(333, prompt)
    for S in (1, 1, 3, 1):
        q = step(S, [S] * B)
        o, l = fa.flash_attention_decode(q, c.obj, c.ints(lens))
        # the reference reads the pages as stored (the append is tested by itself)
        k, v = _host(c.tk), _host(c.tv)
        _check(o, l, P.decode(_host(q), k, v, c.table, lens, D ** -0.5), dtype)
    idx = fa.select_kv_pages(q, c.obj, c.ints(lens), 3)
    lo, hi = _host(c.tlo), _host(c.thi)
    ref = P.select(_host(q), lo, hi, c.table, lens, page, 3)
    assert np.array_equal(idx.cpu().numpy(), ref)
    o, l = fa.flash_attention_decode(q, c.obj, c.ints(lens), page_idx=idx)
    _check(o, l, P.decode(_host(q), k, v, c.table, lens, D ** -0.5, None, ref), dtype)
    assert _status() == 0


def test_other_streams_and_graphs():
    """A stream of its own, and two captured graphs replayed on two streams at
    once, while eager calls run on a third: every answer as alone."""
    import torch
    import attention_forward_fa_gb300 as fa
    lens = [3000, 700]
    c = Cache(16, "bf16", 2, 2, 128, 64, [n + 1 for n in lens], bounds=True)
    n = c.ints(lens)
    q = [_dev(_round(c.rng.standard_normal((2, 8, 1, 128)), "bf16"), "bf16") for _ in range(3)]
    want = [fa.flash_attention_decode(x, c.obj, n) for x in q]
    picks = [fa.select_kv_pages(x, c.obj, n, 8) for x in q]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    o, l = fa.flash_attention_decode(q[0], c.obj, n, stream=s)
    i = fa.select_kv_pages(q[0], c.obj, n, 8, stream=s.cuda_stream)
    s.synchronize()
    assert torch.equal(fa.select_kv_pages(q[0], c.obj, n, 8, stream=0), picks[0])     # the default stream by its handle
    assert torch.equal(o, want[0][0]) and torch.equal(l, want[0][1]) and torch.equal(i, picks[0])
    graphs, outs = [], []
    for x in q[:2]:
        out, lse, idx = torch.empty_like(x), torch.empty(2, 8, 1, device="cuda"), torch.empty_like(picks[0])
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            fa.flash_attention_decode(x, c.obj, n, out=out, lse=lse)
            fa.select_kv_pages(x, c.obj, n, 8, out=idx)
        side.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            fa.flash_attention_decode(x, c.obj, n, out=out, lse=lse)
            fa.select_kv_pages(x, c.obj, n, 8, out=idx)
        graphs.append(g)
        outs.append((out, lse, idx))
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(20):
        for t in (t for o3 in outs for t in o3):
            t.zero_()
        torch.cuda.synchronize()
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                for _ in range(5):
                    g.replay()
        o, l = fa.flash_attention_decode(q[2], c.obj, n)
        torch.cuda.synchronize()
        assert torch.equal(o, want[2][0])
        for (a, b, d), w, pk in zip(outs, want, picks):
            assert torch.equal(a, w[0]) and torch.equal(b, w[1]) and torch.equal(d, pk)
    # new lengths and a new token between two replays: the graph reads them anew
    tok = _dev(_round(c.rng.standard_normal((2, 2, 1, 128)), "bf16"), "bf16")
    fa.paged_kv_append(c.obj, n, tok, tok)
    n += 1
    graphs[0].replay()
    torch.cuda.synchronize()
    k, v = _host(c.tk), _host(c.tv)
    _check(outs[0][0], outs[0][1], P.decode(_host(q[0]), k, v, c.table, [3001, 701], 128 ** -0.5), "bf16")
    assert _status() == 0


def test_wrappers_refuse_what_does_not_fit():
    import torch
    import attention_forward_fa_gb300 as fa
    c = Cache(17, "bf16", 2, 2, 64, 16, [40, 40])
    n = c.ints([40, 40])
    q = torch.zeros(2, 4, 1, 64, dtype=torch.bfloat16, device="cuda")
    x = q[:, :2].contiguous()
    for bad in (q.half(), q.cpu(), q[:1], q[..., :32], q[:, :3], q[:, :, 0], torch.zeros_like(q).transpose(0, 1)):
        with pytest.raises(ValueError):
            fa.flash_attention_decode(bad, c.obj, n)
    for bad in (n.long(), n[:1], n.cpu(), torch.stack((n, n), 1)[:, 0]):
        with pytest.raises(ValueError):
            fa.flash_attention_decode(q, c.obj, bad)
        with pytest.raises(ValueError):
            fa.paged_kv_append(c.obj, bad, x, x)
    with pytest.raises(ValueError):
        fa.flash_attention_decode(q, c.obj, n, pre_tokens=-1)
    with pytest.raises(ValueError):
        fa.flash_attention_decode(q, c.obj, n, page_idx=torch.zeros(2, 1, 3, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):
        fa.flash_attention_decode(q, c.obj, n, out=torch.empty(2, 4, 2, 64, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(ValueError):
        fa.select_kv_pages(q, c.obj, n, 2)                      # no bounds
    with pytest.raises(fa.FaError):
        fa.flash_attention_decode(q, c.obj, n, scale=float("nan"))
    pool = torch.zeros(8 * 2 * 16 * 64 + 4, dtype=torch.bfloat16, device="cuda")[4:].view(8, 2, 16, 64)
    with pytest.raises(fa.FaError) as e:
        fa.flash_attention_decode(q, fa.PagedKV(pool, pool, c.obj.page_table), n)
    assert e.value.code == fa.FA_ERR_ALIGN
    with pytest.raises(ValueError):
        fa.paged_kv_append(c.obj, n, x, x[:, :, :0])
    with pytest.raises(ValueError):
        fa.paged_kv_append(c.obj, n, x, x, cos=torch.zeros(50, 8, device="cuda"))
    assert _status() == 0


def test_front_page_serving_example_runs():
    """The front page's generation step, as written there; over all pages and over
    the chosen ones it answers what the reference does."""
    import re
    from pathlib import Path
    import torch
    import attention_forward_fa_gb300 as fa
    text = (Path(__file__).resolve().parents[1] / "README.md").read_text()
    block = [b for b in re.findall(r"```python\n(.*?)```", text, re.S) if "paged_kv_append" in b][0]
    env = {"torch": torch, "fa": fa}
    torch.manual_seed(30)
    exec(compile(block, "serving-example", "exec"), env)
    k, v, t = _host(env["k_pages"]), _host(env["v_pages"]), env["table"].cpu().numpy()
    q, pages = _host(env["q"]), env["pages"].cpu().numpy()
    _check(env["o"], env["lse"], P.decode(q, k, v, t, [1001, 38], 128 ** -0.5), "bf16")
    lo, hi = (_host(b) for b in env["bounds"])
    assert np.array_equal(pages, P.select(q, lo, hi, t, [1001, 38], 64, 8))
    _check(env["o8"], env["lse8"], P.decode(q, k, v, t, [1001, 38], 128 ** -0.5, None, pages), "bf16")
