"""fp64 reference of the operators over a paged key-value cache: the position
rotation and append, the attention of a sequence's newest tokens over its
pages, and the choice of pages by their key bounds.

Plain NumPy in 64 bits on the exact input values, every matrix materialised;
shares no code with the GPU path.  The cache is a pair of pools
[num_pages, Hkv, page_size, D] and a table [B, max_pages]; a length is the
number of tokens of a sequence.  Where a function is given the rounding
`store`, it is that of the cache's type (value -> nearest representable value).
"""
from __future__ import annotations

import numpy as np

from oracle import fp8 as F

LEAST = -80      # of a scale's exponent
TOP = {"e4m3fn": (8, 119), "e5m2": (15, 112)}      # the largest code is 1.75 * 2^(first); the largest exponent


def exponent(x, fmt):
    """e of the scale 2^e of rows x [..., D] (finite): the least >= LEAST with
    max |x| <= (largest code) 2^e."""
    a = np.abs(np.asarray(x, dtype=np.float64)).max(-1)
    m, k = np.frexp(np.where(a > 0, a, 1.0))             # a = 2 m * 2^(k - 1), 1 <= 2 m < 2
    e = k - 1 - TOP[fmt][0] + (m > 0.875)
    return np.where(a > 0, np.clip(e, LEAST, TOP[fmt][1]), LEAST).astype(np.int64)


def quantise(x, fmt):
    """(codes [..., D], exponents [...]) of rows: x is stored as codes * 2^e."""
    e = exponent(x, fmt)
    z = np.ldexp(np.asarray(x, dtype=np.float64), -e[..., None])
    top = F.FORMATS[fmt][2]
    return F.round_fp8(np.clip(z, -top, top), fmt), e


def rotate(x, pos, cos, sin, interleaved: bool):
    """x [..., S, D] with the first r = 2 * cos.shape[1] channels turned by the
    angles of positions pos [S]: (a, b) -> (a cos - b sin, a sin + b cos) for
    the pairs (j, j + r/2), or (2j, 2j + 1) when interleaved."""
    r = 2 * cos.shape[1]
    y = np.array(x, dtype=np.float64)
    c, s = cos[pos].astype(np.float64), sin[pos].astype(np.float64)
    ia = np.arange(0, r, 2) if interleaved else np.arange(r // 2)
    ib = ia + (1 if interleaved else r // 2)
    a, b = x[..., ia].astype(np.float64), x[..., ib].astype(np.float64)
    y[..., ia] = a * c - b * s
    y[..., ib] = a * s + b * c
    return y


def append(k_pages, v_pages, table, lens, k, v, new_lens, cos=None, sin=None,
           interleaved=False, store=lambda x: x, k_min=None, k_max=None, positions=None,
           store_v=lambda x: x):
    """The pools (and bounds, where given) after the append; the arguments are
    left alone.  k, v [B, Hkv, S, D].  positions [B, S]: the tokens turn by them
    instead of by where they stand."""
    kp, vp = k_pages.copy(), v_pages.copy()
    lo = None if k_min is None else k_min.copy()
    hi = None if k_max is None else k_max.copy()
    page = kp.shape[2]
    for b in range(table.shape[0]):
        for i in range(int(new_lens[b])):
            t = int(lens[b]) + i
            x = k[b, :, i]
            if cos is not None:
                at = t if positions is None else int(positions[b, i])
                x = rotate(x[:, None], np.array([at]), cos, sin, interleaved)[:, 0]
            x = store(x)
            p, slot = table[b, t // page], t % page
            kp[p, :, slot] = x
            vp[p, :, slot] = store_v(v[b, :, i])
            if lo is not None:
                lo[p] = x if slot == 0 else np.minimum(lo[p], x)
                hi[p] = x if slot == 0 else np.maximum(hi[p], x)
    return kp, vp, lo, hi


def decode(q, k_pages, v_pages, table, lens, scale, pre_tokens=None, page_idx=None, tree=None):
    """(O, LSE, A, X, V): the attention of q [B, Hq, Sq, D] over the pages, its
    log-sum-exp (+inf for a row that sees no key, O = 0 there), and for error
    bounds A = sum_j p_j |v_j| and V = sum_j |v_j| per output and X = max over
    the row's keys of scale * sum_d |q_d k_jd|.  tree: (ancestors [B, Sq, Sq],
    drafts [B]): the last drafts[b] tokens are a tree, row i its draft i, which
    sees the tokens before and the drafts of its row of ancestors; rows past
    drafts[b] see the tokens before."""
    B, Hq, Sq, D = q.shape
    Hkv, page = k_pages.shape[1], k_pages.shape[2]
    G = Hq // Hkv
    O = np.zeros((B, Hq, Sq, D))
    A = np.zeros((B, Hq, Sq, D))
    V = np.zeros((B, Hq, Sq, D))
    L = np.full((B, Hq, Sq), np.inf)
    X = np.zeros((B, Hq, Sq))
    for b in range(B):
        n = int(lens[b])
        n_pages = -(-n // page)
        for h in range(Hkv):
            pages = np.arange(n_pages)
            if page_idx is not None:
                pages = page_idx[b, h, :n_pages]     # as many entries count as there are pages
                pages = pages[(pages >= 0) & (pages < n_pages)]
            pos = (pages[:, None] * page + np.arange(page)).reshape(-1)
            ids = table[b, pages]
            k = k_pages[ids, h].reshape(-1, D)
            v = v_pages[ids, h].reshape(-1, D)
            for i in range(Sq):
                t = n - Sq + i
                see = pos <= t
                if tree is not None:
                    first = n - int(tree[1][b])
                    see = pos < first
                    if i < tree[1][b]:
                        see = see | ((pos < n) & tree[0][b][i][np.clip(pos - first, 0, Sq - 1)].astype(bool))
                if pre_tokens is not None:
                    see &= pos >= t - pre_tokens
                if not see.any():
                    continue
                ks, vs = k[see], v[see]
                for g in range(G):
                    x = q[b, h * G + g, i]
                    s = scale * (ks @ x)
                    m = s.max()
                    e = np.exp(s - m)
                    l = e.sum()
                    O[b, h * G + g, i] = (e / l) @ vs
                    A[b, h * G + g, i] = (e / l) @ np.abs(vs)
                    V[b, h * G + g, i] = np.abs(vs).sum(0)
                    L[b, h * G + g, i] = m + np.log(l)
                    X[b, h * G + g, i] = abs(scale) * (np.abs(ks) @ np.abs(x)).max()
    return O, L, A, X, V


def select(q, k_min, k_max, table, lens, page, max_sel, first=1, last=1):
    """page_idx [B, Hkv, max_sel]: the `first` and `last` pages, then those of
    the largest scores (equal scores by page number), ascending, -1 behind."""
    B, Hq, Sq, D = q.shape
    Hkv = k_min.shape[1]
    G = Hq // Hkv
    out = np.full((B, Hkv, max_sel), -1, dtype=np.int32)
    for b in range(B):
        n = -(-int(lens[b]) // page)
        for h in range(Hkv):
            lo, hi = k_min[table[b, :n], h], k_max[table[b, :n], h]
            score = np.full(n, -np.inf)
            for g in range(G):
                for i in range(Sq):
                    x = q[b, h * G + g, i]
                    score = np.maximum(score, np.maximum(x * lo, x * hi).sum(-1))
            forced = [p for p in range(n) if p < first or p >= n - last]
            others = sorted((p for p in range(n) if first <= p < n - last),
                            key=lambda p: (-score[p], p))
            take = sorted(forced + others[:max_sel - len(forced)])
            out[b, h, :len(take)] = take
    return out


def read(k_pages, v_pages, table, starts, lens, k_out, v_out):
    """(k, v) [B, Hkv, S, D]: row i < lens[b] is token starts[b] + i, the others
    as in k_out, v_out."""
    k, v, page = k_out.copy(), v_out.copy(), k_pages.shape[2]
    for b in range(table.shape[0]):
        for i in range(int(lens[b])):
            t = int(starts[b]) + i
            k[b, :, i] = k_pages[table[b, t // page], :, t % page]
            v[b, :, i] = v_pages[table[b, t // page], :, t % page]
    return k, v


def keep(pools, table, lens, idx, keep_lens, page, keys=None, k_min=None, k_max=None):
    """The pools [num_pages, Hkv, page, ...] after each sequence's accepted drafts
    idx[b, :keep_lens[b]] moved behind its lens[b] tokens; with keys (what the
    first pool's rows stand for, [num_pages, Hkv, page, D]) the bounds too."""
    pools = [x.copy() for x in pools]
    lo, hi = (None, None) if k_min is None else (k_min.copy(), k_max.copy())
    for b in range(table.shape[0]):
        n = int(lens[b])
        path = [int(j) for j in idx[b, :int(keep_lens[b])]]
        rows = [[x[table[b, (n + j) // page], :, (n + j) % page].copy() for x in pools + ([] if lo is None else [keys])]
                for j in path]
        for i, (j, row) in enumerate(zip(path, rows)):
            if i == j:
                continue
            p, slot = table[b, (n + i) // page], (n + i) % page
            for x, r in zip(pools, row):
                x[p, :, slot] = r
            if lo is not None:
                lo[p] = row[-1] if slot == 0 else np.minimum(lo[p], row[-1])
                hi[p] = row[-1] if slot == 0 else np.maximum(hi[p], row[-1])
    return pools, lo, hi
