"""Rows of an 8-bit cache that are not finite, and rows of very different sizes, in decode and trees
by every kernel (up to 64 rows per KV head by warps, more by tcgen05), against the fp64 reference
of oracle/paged.py with the bounds of tests/test_gpu_paged8.py.

A row that is not finite is stored as codes 0 with the scale byte 255.  Of a value it is NaN in the
answer of each row that sees it; its weight and so the LSE are those of its key.  Of a key the
answer and the LSE of a row that sees it are NaN.  A row that does not see it is answered as
without: as if its codes stood for zeros."""
import numpy as np
import pytest

from oracle import paged as P
from tests.test_gpu_paged import _dev, _host, _round, _status
from tests.test_gpu_paged8 import Cache8, _check8, _spread, _trees

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from attention_forward_fa_gb300 import build
    build.build()


def _seen(lens, Sq, pre=None, tree=None):
    """bool [B, Sq, longest]: which keys a row sees."""
    pos = np.arange(max(lens))
    see = np.zeros((len(lens), Sq, pos.size), dtype=bool)
    for b, n in enumerate(lens):
        for i in range(Sq):
            t = n - Sq + i
            see[b, i] = pos <= t if tree is None else pos < n - tree[1][b]
            if pre is not None:
                see[b, i] &= pos >= t - pre
            if tree is not None and i < tree[1][b]:
                first = n - tree[1][b]
                see[b, i, first:n] = tree[0][b, i, : tree[1][b]]
    return see


def _spoil(c, kind, b, t):
    """Token t of sequence b, every head: a key ("k") or value ("v") row that is not finite, zero on the
    reference's side."""
    p, s = int(c.table[b, t // c.page]), t % c.page
    codes, scale = (c.bk, c.sk) if kind == "k" else (c.bv, c.sv)
    codes[p, :, s], scale[p, :, s] = 0, 255
    (c.k if kind == "k" else c.v)[p, :, s] = 0
    (c.kc if kind == "k" else c.vc)[p, :, s] = 0
    (c.ke if kind == "k" else c.ve)[p, :, s] = 0


def _compare(c, q, lens, got, bad_k, bad_v, pre=None, tree=None, where=""):
    """bad_k, bad_v: per sequence the tokens whose rows are not finite."""
    o, l = (_host(x) for x in got)
    B, Hq, Sq, D = q.shape
    a = (c.table, lens, D ** -0.5)
    ref = P.decode(q, c.k, c.v, *a, pre, None, tree)
    see = _seen(lens, Sq, pre, tree)
    nan_k, nan_v = (np.array([see[b][:, bad[b]].any(-1) for b in range(B)]) for bad in (bad_k, bad_v))     # [B, Sq]
    every = lambda x: np.broadcast_to(x[:, None], (B, Hq, Sq))
    assert np.isnan(o[every(nan_k | nan_v)]).all(), f"{where}: rows that see what is not finite"
    assert np.isnan(l[every(nan_k)]).all() and not np.isnan(l[~every(nan_k)]).any(), f"{where}: LSE"
    clean = np.where(every(nan_k | nan_v)[..., None], ref[0], o)
    lse = np.where(every(nan_k), ref[1], l)
    _check8(_dev(clean.astype(np.float32)), _dev(lse.astype(np.float32)), ref, *_spread(c, q, *a, tree, pre), c.dtype, where)


ROWS = [
    # dtype, fmt, Hq, Hkv, D, page, Sq
    ("bf16", "e4m3fn", 4, 1, 128, 64, 1), ("fp16", "e5m2", 4, 2, 64, 16, 5), ("bf16", "e5m2", 12, 2, 128, 32, 4),
    ("fp16", "e4m3fn", 8, 2, 128, 64, 10), ("bf16", "e4m3fn", 4, 2, 64, 128, 27),          # by warps: 1 to 54 rows
    ("bf16", "e4m3fn", 8, 2, 128, 64, 25), ("fp16", "e5m2", 8, 2, 64, 16, 20),             # by tcgen05, up to 128
    ("fp16", "e4m3fn", 4, 1, 128, 32, 40), ("bf16", "e5m2", 7, 1, 64, 256, 40),            # and more
]


@pytest.mark.parametrize("case", ROWS, ids=lambda c: "-".join(map(str, c)))
@pytest.mark.parametrize("kinds", ["v", "k", "kv"])
def test_rows_that_are_not_finite(case, kinds):
    """Among the newest tokens, in the text before them (one sequence in one piece, one cut into many),
    and where a window ends."""
    import attention_forward_fa_gb300 as fa
    dtype, fmt, Hq, Hkv, D, page, Sq = case
    lens = [200, 3000, 130]
    for form in ("decode", "window", "tree"):
        c = Cache8(41, dtype, fmt, 3, Hkv, D, page, lens)
        late = [[n - 1 - Sq // 2] for n in lens]
        text = [[], [17, 2000], []]
        bad = [x + y for x, y in zip(late, text if form != "window" else [[], [lens[1] - Sq - 9], []])]
        for kind in kinds:
            for b in range(3):
                for t in bad[b]:
                    _spoil(c, kind, b, t)
        q = _round(c.rng.standard_normal((3, Hq, Sq, D)), dtype)
        tq, n = _dev(q, dtype), c.ints(lens)
        pre, tree = (10 if form == "window" else None), None
        if form == "tree":
            drafts = [Sq, Sq, max(Sq - 2, 0)]
            tree = (_trees(c.rng, 3, Sq)[0], drafts)
            got = fa.flash_attention_decode_tree(tq, c.obj, n, _dev(tree[0]), new_lens=c.ints(drafts))
        else:
            got = fa.flash_attention_decode(tq, c.obj, n, pre_tokens=pre)
        assert _status() == 0
        none = [[], [], []]
        _compare(c, q, lens, got, bad if "k" in kinds else none, bad if "v" in kinds else none, pre, tree, f"{kinds} {form}")


@pytest.mark.parametrize("case", ROWS, ids=lambda c: "-".join(map(str, c)))
@pytest.mark.parametrize("kinds", ["v", "k", "kv"])
def test_rows_that_see_nothing_finite(case, kinds):
    """A sequence of such tokens alone, and one whose first row sees one of them and no other."""
    import attention_forward_fa_gb300 as fa
    dtype, fmt, Hq, Hkv, D, page, Sq = case
    lens = [Sq, Sq + 200, Sq]
    c = Cache8(46, dtype, fmt, 3, Hkv, D, page, lens)
    bad = [list(range(Sq)), [], [0]]
    for b in range(3):
        for t in bad[b]:
            for kind in kinds:
                _spoil(c, kind, b, t)
    q = _round(c.rng.standard_normal((3, Hq, Sq, D)), dtype)
    none = [[], [], []]
    for tree in (None, (np.broadcast_to(np.tril(np.ones((Sq, Sq), dtype=bool)), (3, Sq, Sq)).copy(), [Sq, Sq, Sq])):
        got = (fa.flash_attention_decode(_dev(q, dtype), c.obj, c.ints(lens)) if tree is None else
               fa.flash_attention_decode_tree(_dev(q, dtype), c.obj, c.ints(lens), _dev(tree[0])))
        assert _status() == 0
        _compare(c, q, lens, got, bad if "k" in kinds else none, bad if "v" in kinds else none, None, tree, f"{kinds} tree {tree is not None}")


def _set_keys(c, k):
    """The cache's keys become k [num_pages, Hkv, page, D], quantised."""
    c.kc, c.ke = P.quantise(k, c.fmt)
    c.k = np.ldexp(c.kc, c.ke[..., None])
    from tests.test_gpu_paged8 import _codes
    c.bk.copy_(_codes(c.kc, c.fmt).view(c.bk.dtype))
    c.sk.copy_(_dev((c.ke + 127).astype(np.uint8)))


@pytest.mark.parametrize("case", ROWS, ids=lambda c: "-".join(map(str, c)))
def test_small_keys_beside_large_ones(case):
    """Keys up to 2^60 times the others, orthogonal to every query, so that the answers are the small
    keys' own; zero rows among them."""
    import attention_forward_fa_gb300 as fa
    dtype, fmt, Hq, Hkv, D, page, Sq = case
    lens = [200, 3000, 130]
    c = Cache8(42, dtype, fmt, 3, Hkv, D, page, lens)
    q = _round(c.rng.standard_normal((3, Hq, Sq, D)), dtype)
    q[..., 0] = 0
    for share in (0.02, 0.5):
        k = c.rng.standard_normal(c.k.shape)
        large = c.rng.random(c.k.shape[:3]) < share
        k[large] = 0
        k[large, 0] = 2.0 ** c.rng.integers(5, 60, int(large.sum()))
        k[c.rng.random(c.k.shape[:3]) < 0.02] = 0
        _set_keys(c, k)
        for tree in (None, (_trees(c.rng, 3, Sq)[0], [Sq, Sq, max(Sq - 2, 0)])):
            tq, n = _dev(q, dtype), c.ints(lens)
            got = (fa.flash_attention_decode(tq, c.obj, n) if tree is None else
                   fa.flash_attention_decode_tree(tq, c.obj, n, _dev(tree[0]), new_lens=c.ints(tree[1])))
            assert _status() == 0
            none = [[], [], []]
            _compare(c, q, lens, got, none, none, None, tree, f"share {share} tree {tree is not None}")


def _set_values(c, v):
    """The cache's values become v [num_pages, Hkv, page, D], quantised."""
    from tests.test_gpu_paged8 import _codes
    c.vc, c.ve = P.quantise(v, c.fmt)
    c.v = np.ldexp(c.vc, c.ve[..., None])
    c.bv.copy_(_codes(c.vc, c.fmt).view(c.bv.dtype))
    c.sv.copy_(_dev((c.ve + 127).astype(np.uint8)))


@pytest.mark.parametrize("order", ["mixed", "small first", "large first", "one large"])
@pytest.mark.parametrize("case", [c for c in ROWS if c[0] == "bf16"], ids=lambda c: "-".join(map(str, c)))
def test_values_over_the_whole_range(case, order):
    """Rows of zeros (e = -80) and values of 2^-70 beside values of 2^110: a key's share of the sum does
    not go by its value's size, within a tile, from tile to tile and from piece to piece."""
    import attention_forward_fa_gb300 as fa
    dtype, fmt, Hq, Hkv, D, page, Sq = case
    lens = [200, 3000, 130]
    c = Cache8(44, dtype, fmt, 3, Hkv, D, page, lens)
    q = _round(c.rng.standard_normal((3, Hq, Sq, D)), dtype)
    size = np.full(c.v.shape[:3], -200.0)
    for b, n in enumerate(lens):
        for t in range(n):
            late = t >= n // 2
            e = {"mixed": c.rng.choice([-200, -70, 0, 60, 110]), "small first": 110 if late else -200,
                 "large first": -200 if late else 110, "one large": 110 if t == n // 3 else -70}[order]
            size[c.table[b, t // page], :, t % page] = e
    _set_values(c, np.where(size[..., None] < -190, 0.0, c.rng.standard_normal(c.v.shape) * np.exp2(size)[..., None]))
    for scale in (0.0, D ** -0.5, 2.0):
        for tree in (None, (_trees(c.rng, 3, Sq)[0], [Sq, Sq, max(Sq - 2, 0)])):
            tq, n = _dev(q, dtype), c.ints(lens)
            o, l = (fa.flash_attention_decode(tq, c.obj, n, scale=scale) if tree is None else
                    fa.flash_attention_decode_tree(tq, c.obj, n, _dev(tree[0]), new_lens=c.ints(tree[1]), scale=scale))
            assert _status() == 0
            a = (c.table, lens, scale)
            ref = P.decode(q, c.k, c.v, *a, tree=tree)
            _check8(o, l, ref, *_spread(c, q, *a, tree), dtype, f"scale {scale} tree {tree is not None}")


@pytest.mark.parametrize("case", [c for c in ROWS if c[-1] >= 4], ids=lambda c: "-".join(map(str, c)))
def test_a_large_draft_reaches_no_other_branch(case):
    """One draft's key of 2^70: rows that do not see it are answered to the usual bounds."""
    import attention_forward_fa_gb300 as fa
    dtype, fmt, Hq, Hkv, D, page, Sq = case
    lens, drafts = [200, 3000, 130], [Sq, Sq, Sq - 1]
    c = Cache8(43, dtype, fmt, 3, Hkv, D, page, lens)
    k = c.k.copy()
    for b in range(3):
        t = lens[b] - drafts[b] + 1
        k[c.table[b, t // page], :, t % page] *= 2.0 ** 70
    _set_keys(c, k)
    anc = _trees(c.rng, 3, Sq)[0]
    anc[:, 2:, 1] = c.rng.random((3, Sq - 2)) < 0.3
    q = _round(c.rng.standard_normal((3, Hq, Sq, D)), dtype)
    o, l = fa.flash_attention_decode_tree(_dev(q, dtype), c.obj, c.ints(lens), _dev(anc), new_lens=c.ints(drafts))
    assert _status() == 0
    a = (c.table, lens, D ** -0.5)
    ref = P.decode(q, c.k, c.v, *a, tree=(anc, drafts))
    W, E = _spread(c, q, *a, (anc, drafts))
    clear = np.array([[i >= drafts[b] or not anc[b, i, 1] for i in range(Sq)] for b in range(3)])
    assert clear.any() and not clear.all()
    rows = np.broadcast_to(clear[:, None], (3, Hq, Sq))
    pick = lambda x: x[rows][None, None]
    got = [_dev(np.ascontiguousarray(pick(_host(x))).astype(np.float32)) for x in (o, l)]
    _check8(*got, [pick(x) for x in ref], pick(W), E, dtype, "clear rows")


@pytest.mark.parametrize("dtype,fmt,Hq,Hkv,D,page,S", [
    ("bf16", None, 4, 1, 128, 64, 8), ("fp16", None, 2, 1, 64, 16, 16), ("bf16", None, 1, 1, 128, 32, 32),          # by warps
    ("bf16", None, 8, 1, 128, 64, 12), ("fp16", None, 8, 2, 64, 32, 60), ("bf16", None, 2, 1, 128, 16, 150),         # by tcgen05
    ("bf16", "e4m3fn", 4, 1, 128, 64, 8), ("fp16", "e5m2", 2, 2, 64, 32, 30), ("bf16", "e5m2", 1, 1, 128, 16, 60),
    ("bf16", "e4m3fn", 8, 1, 128, 64, 12), ("fp16", "e4m3fn", 8, 2, 64, 32, 60), ("bf16", "e4m3fn", 2, 1, 128, 16, 150),
])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_drafts_that_no_row_sees_may_be_anything(dtype, fmt, Hq, Hkv, D, page, S, bad):
    """Keys and values of drafts whose column of ancestors is empty, the first and the last among them, and
    of those that only rows past a sequence's drafts name: anything in a 16-bit cache, rows that are not
    finite in an 8-bit one."""
    import attention_forward_fa_gb300 as fa
    from tests.test_gpu_paged import Cache, _check
    lens, drafts = [S + 300, S, 2 * S + 77], [S, S, S - 3]
    c = Cache(45, dtype, 3, Hkv, D, page, lens) if fmt is None else Cache8(45, dtype, fmt, 3, Hkv, D, page, lens)
    anc, _ = _trees(c.rng, 3, S)
    blind = c.rng.random((3, S)) < 0.3
    blind[0, 0] = blind[1, S - 1] = blind[2, S - 4] = True
    for b in range(3):
        anc[b][:, blind[b]] = False
        anc[b, drafts[b]:] = True
        for j in range(drafts[b]):
            if blind[b, j]:
                t = lens[b] - drafts[b] + j
                p, s = int(c.table[b, t // page]), t % page
                if fmt is None:
                    c.tk[p, :, s], c.tv[p, :, s] = bad, -bad
                else:
                    c.bk[p, :, s], c.bv[p, :, s] = 0, 0
                    c.sk[p, :, s], c.sv[p, :, s] = 255, 255
    q = _round(c.rng.standard_normal((3, Hq, S, D)), dtype)
    o, l = fa.flash_attention_decode_tree(_dev(q, dtype), c.obj, c.ints(lens), _dev(anc), new_lens=c.ints(drafts))
    assert _status() == 0
    a = (c.table, lens, D ** -0.5)
    ref = P.decode(q, c.k, c.v, *a, tree=(anc, drafts))
    if fmt is None:
        _check(o, l, ref, dtype, "blind drafts")
    else:
        _check8(o, l, ref, *_spread(c, q, *a, (anc, drafts)), dtype, "blind drafts")
