"""GPU tests of the paged operators at sizes and in orders of calls beyond
those of tests/test_gpu_paged.py."""
import math

import numpy as np
import pytest

from oracle import paged as P
from tests.test_gpu_paged import Cache, _check, _dev, _host, _round, _status, _tables

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from attention_forward_fa_gb300 import build
    build.build()


@pytest.mark.parametrize("dtype,B,Hq,Hkv,D,page,S,rot,inter,lengths", [
    ("bf16", 3, 40, 5, 128, 16, 8192, 128, False, False),
    ("bf16", 3, 40, 5, 128, 16, 8192, 64, True, True),
    ("fp16", 2, 9, 9, 64, 16, 16000, 64, False, True),
    ("fp16", 1, 24, 3, 64, 32, 70000, 32, True, False),
    ("bf16", 1, 1, 1, 128, 16, 60000, 0, False, False),
])
def test_append_of_more_pieces_than_blocks(dtype, B, Hq, Hkv, D, page, S, rot, inter, lengths):
    """Large prompts, every page full: the keys and queries within their
    rounding of the 64-bit rotation, the values and untouched rows as they are,
    the bounds those of the stored keys."""
    import torch
    import attention_forward_fa_gb300 as fa
    dt = torch.bfloat16 if dtype == "bf16" else torch.float16
    g = torch.Generator(device="cuda").manual_seed(40)
    old = 5
    wide = -(-(S + old) // page)
    num = B * wide + 3
    k, v = (torch.randn(num, Hkv, page, D, generator=g, device="cuda", dtype=dt) for _ in range(2))
    was_k, was_v = k.clone(), v.clone()
    lo, hi = torch.full((num, Hkv, D), 9.0, device="cuda", dtype=dt), torch.full((num, Hkv, D), -9.0, device="cuda", dtype=dt)
    table = torch.randperm(num, generator=g, device="cuda").to(torch.int32)[:B * wide].view(B, wide).contiguous()
    cache = fa.PagedKV(k, v, table, lo, hi)
    x = torch.randn(B, S, Hq + 2 * Hkv, D, generator=g, device="cuda", dtype=dt).transpose(1, 2)
    q, kn, vn = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
    cos, sin = _tables(S + old, rot) if rot else (None, None)
    tc, ts = (_dev(cos), _dev(sin)) if rot else (None, None)
    lens = torch.full((B,), old, device="cuda", dtype=torch.int32)
    new = [S] * B
    if lengths:
        new[-1] = S - 37
    n = torch.tensor(new, device="cuda", dtype=torch.int32)
    qo = torch.zeros(B, Hq, S, D, device="cuda", dtype=dt)
    fa.paged_kv_append(cache, lens, kn, vn, new_lens=n if lengths else None, q=q, q_out=qo, cos=tc, sin=ts, interleaved=inter)
    assert _status() == 0
    u, sub = (2.0 ** -8, 0.0) if dtype == "bf16" else (2.0 ** -11, 2.0 ** -25)

    def turned(y, b):
        """(rotation, bound) of y [heads, n, D] in 64 bits: the products and sums in fp32 are three roundings."""
        y = y.double()
        r, lim = y.clone(), torch.zeros_like(y)
        if rot:
            c, s = tc[old:old + y.shape[1]].double(), ts[old:old + y.shape[1]].double()
            i = torch.arange(rot // 2, device="cuda")
            ia, ib = (2 * i, 2 * i + 1) if inter else (i, i + rot // 2)
            a, d = y[..., ia], y[..., ib]
            r[..., ia], r[..., ib] = a * c - d * s, a * s + d * c
            e = (1 + u) * 3 * 2.0 ** -24
            lim[..., ia] = u * r[..., ia].abs() + e * ((a * c).abs() + (d * s).abs()) + sub
            lim[..., ib] = u * r[..., ib].abs() + e * ((a * s).abs() + (d * c).abs()) + sub
        return r, lim

    wrote = torch.zeros(num, page, dtype=torch.bool, device="cuda")
    for b in range(B):
        pos = torch.arange(old, old + new[b], device="cuda")
        at, slot = table[b].long()[pos // page], pos % page
        wrote[at, slot] = True
        ref, lim = turned(kn[b, :, :new[b]], b)
        assert bool(((k[at, :, slot].transpose(0, 1).double() - ref).abs() <= lim).all())
        assert torch.equal(v[at, :, slot].transpose(0, 1), vn[b, :, :new[b]])
        ref, lim = turned(q[b, :, :new[b]], b)
        assert bool(((qo[b, :, :new[b]].double() - ref).abs() <= lim).all())
        assert bool((qo[b, :, new[b]:] == 0).all())
        full = table[b, 1:(old + new[b]) // page].long()   # (the first page held keys before, the last may be short)
        assert torch.equal(lo[full], k[full].amin(2)) and torch.equal(hi[full], k[full].amax(2))
        first = int(table[b, 0])
        assert torch.equal(lo[first], k[first, :, old:].amin(1).clamp(max=9.0))
        assert torch.equal(hi[first], k[first, :, old:].amax(1).clamp(min=-9.0))
    keep = ~wrote[:, None, :, None].expand_as(k)
    assert torch.equal(k[keep], was_k[keep]) and torch.equal(v[keep], was_v[keep])


@pytest.mark.parametrize("dtype,Hq,Hkv,D,page,S,old,new,pre", [
    ("bf16", 8, 2, 128, 16, 5, [40, 7, 0, 100], [5, 2, 3, 0], None),
    ("fp16", 6, 6, 64, 32, 4, [0, 31, 700], [4, 1, 3], 20),
    ("bf16", 16, 1, 128, 64, 9, [1000, 64], [1, 9], None),
    ("bf16", 8, 4, 64, 16, 60, [0, 3], [60, 21], None),
])
def test_steps_of_different_lengths(dtype, Hq, Hkv, D, page, S, old, new, pre):
    """A padded step: the append's rows lie at the front, the attention takes
    them at the end of its rows; moved there and back by one gather each, every
    sequence is answered as by a call of its own.  The rows in front belong to
    no token and may hold anything: they reach no other row."""
    import torch
    import attention_forward_fa_gb300 as fa
    B = len(old)
    c = Cache(41, dtype, B, Hkv, D, page, [o + n for o, n in zip(old, new)])
    x = _dev(_round(c.rng.standard_normal((B, Hq + 2 * Hkv, S, D)), dtype), dtype)
    cos, sin = _tables(max(old) + S, D)
    lens, n = c.ints(old), c.ints(new)
    q = torch.full((B, Hq, S, D), float("nan"), dtype=x.dtype, device="cuda")
    fa.paged_kv_append(c.obj, lens, x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], new_lens=n, q=x[:, :Hq], q_out=q, cos=_dev(cos), sin=_dev(sin))
    lens = lens + n
    i, gap = torch.arange(S, device="cuda"), (S - n)[:, None]
    to_end = ((i - gap) % S)[:, None, :, None].expand_as(q)
    o, l = fa.flash_attention_decode(q.gather(2, to_end), c.obj, lens, pre_tokens=pre)
    to_front = (i + gap) % S
    o = o.gather(2, to_front[:, None, :, None].expand_as(o))
    l = l.gather(2, to_front[:, None].expand_as(l))
    assert _status() == 0
    k, v, qh = _host(c.tk), _host(c.tv), _host(q)
    for b in range(B):
        m = new[b]
        if m:
            ref = P.decode(qh[b:b + 1, :, :m], k, v, c.table[b:b + 1], [old[b] + m], D ** -0.5, pre)
            _check(o[b:b + 1, :, :m], l[b:b + 1, :, :m], ref, dtype, f"sequence {b}")


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_bounds_after_tokens_are_taken_back(dtype):
    """Draft tokens that are refused: kv_lens goes back inside a page and the
    next tokens overwrite them.  The bounds stay those of all keys stored in the
    page since its slot 0 was written, so that no score falls below a key's;
    a page whose slot 0 is written again starts anew."""
    import torch
    import attention_forward_fa_gb300 as fa
    page, D = 16, 64
    c = Cache(42, dtype, 1, 2, D, page, [3 * page], bounds=True)
    x = [_dev(_round(c.rng.standard_normal((1, 2, 12, D)), dtype), dtype) for _ in range(3)]
    fa.paged_kv_append(c.obj, c.ints([0]), x[0], x[0])                   # tokens 0 .. 11
    fa.paged_kv_append(c.obj, c.ints([12]), x[1], x[1])                  # 12 .. 23: 4 into page 0, 8 into page 1
    fa.paged_kv_append(c.obj, c.ints([14]), x[2], x[2])                  # back to 14: 14 .. 25
    assert _status() == 0
    p0, p1 = int(c.table[0, 0]), int(c.table[0, 1])
    every = torch.cat((x[0][0], x[1][0, :, :4], x[2][0, :, :2]), 1)      # whatever page 0 has held
    assert torch.equal(c.tlo[p0], every.amin(1)) and torch.equal(c.thi[p0], every.amax(1))
    assert torch.equal(c.tlo[p1], x[2][0, :, 2:].amin(1)) and torch.equal(c.thi[p1], x[2][0, :, 2:].amax(1))
    for p in (p0, p1):
        held = c.tk[p] if p == p0 else c.tk[p][:, :10]
        assert bool((c.tlo[p][:, None] <= held).all()) and bool((c.thi[p][:, None] >= held).all())


def test_a_window_past_32_bits_is_none():
    import torch
    import attention_forward_fa_gb300 as fa
    c = Cache(43, "bf16", 2, 2, 64, 32, [300, 33])
    q = _dev(_round(c.rng.standard_normal((2, 4, 3, 64)), "bf16"), "bf16")
    n = c.ints([300, 33])
    o, l = fa.flash_attention_decode(q, c.obj, n)
    for pre in (300, 2 ** 31 - 1, 2 ** 31, 2 ** 32, 2 ** 32 + 1, 2 ** 63):
        x, y = fa.flash_attention_decode(q, c.obj, n, pre_tokens=pre)
        assert torch.equal(o, x) and torch.equal(l, y), pre
    assert _status() == 0


@pytest.mark.parametrize("dtype,B,Hq,Hkv,D,page", [("bf16", 5, 8, 2, 128, 16), ("fp16", 40, 4, 4, 64, 32)])
def test_steps_in_flight(dtype, B, Hq, Hkv, D, page):
    """Many steps with nothing between their calls: each kernel may start while
    the one before it drains, and reads what that one wrote (pages, bounds, the
    list of pages, its rotated queries).  The same bits as with a wait after
    every call."""
    import torch
    import attention_forward_fa_gb300 as fa
    steps, S = 60, 2
    cos, sin = (_dev(x) for x in _tables(3 * steps + 200, D))
    rng = np.random.default_rng(44)
    start = [int(x) for x in rng.integers(0, 200, B)]
    cap = [n + S * steps for n in start]
    xs = [_dev(_round(rng.standard_normal((B, Hq + 2 * Hkv, S, D)), dtype), dtype) for _ in range(steps)]
    first = _dev(_round(rng.standard_normal((B, Hkv, 200, D)), dtype), dtype)
    lens = [_dev(np.asarray([n + S * i for n in start], dtype=np.int32)) for i in range(steps + 1)]
    zero = torch.zeros_like(lens[0])

    def run(wait):
        c = Cache(45, dtype, B, Hkv, D, page, cap, bounds=True)
        fa.paged_kv_append(c.obj, zero, first, first, new_lens=lens[0], cos=cos, sin=sin)
        torch.cuda.synchronize()
        out = []
        outs = [(torch.empty(B, Hq, S, D, dtype=first.dtype, device="cuda"), torch.empty(B, Hkv, 7, dtype=torch.int32, device="cuda"),
                 *(torch.empty(B, Hq, S, D, dtype=first.dtype, device="cuda") for _ in range(2)),
                 *(torch.empty(B, Hq, S, device="cuda") for _ in range(2))) for _ in range(steps)]
        torch.cuda.synchronize()
        for i, (q, idx, o, o7, l, l7) in enumerate(outs):
            x = xs[i]
            for call in (lambda: fa.paged_kv_append(c.obj, lens[i], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], q=x[:, :Hq], q_out=q, cos=cos, sin=sin),
                         lambda: fa.flash_attention_decode(q, c.obj, lens[i + 1], out=o, lse=l),
                         lambda: fa.select_kv_pages(q, c.obj, lens[i + 1], 7, out=idx),
                         lambda: fa.flash_attention_decode(q, c.obj, lens[i + 1], page_idx=idx, out=o7, lse=l7)):
                call()
                if wait:
                    torch.cuda.synchronize()
            out += [q, idx, o, o7, l, l7]
        torch.cuda.synchronize()
        return out + [c.tk, c.tv, c.tlo, c.thi]

    want = run(True)
    for _ in range(5):
        for i, (a, b) in enumerate(zip(run(False), want)):
            assert torch.equal(a, b), f"output {i}"
    assert _status() == 0
    # appends alone, one behind the other: the bounds are read and written by each
    for wait in (True, False, False, False):
        c = Cache(46, dtype, B, Hkv, D, page, cap, bounds=True)
        torch.cuda.synchronize()
        for i in range(steps):
            fa.paged_kv_append(c.obj, lens[i], xs[i][:, :Hkv], xs[i][:, :Hkv])
            if wait:
                torch.cuda.synchronize()
        torch.cuda.synchronize()
        got = [t.clone() for t in (c.tk, c.tv, c.tlo, c.thi)]
        if wait:
            want = got
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("dtype,D,B,G,n", [("fp16", 128, 304, 1, 131072), ("fp16", 64, 304, 8, 131072),
                                           ("bf16", 128, 304, 1, 131072), ("fp16", 64, 160, 48, 65536),
                                           ("fp16", 128, 160, 20, 65536)])
def test_decode_long_sums_lose_nothing(dtype, D, B, G, n):
    """So many long sequences that a block sums whole ones by itself, thousands of
    tiles; values of one sign, so that whatever the sums cut off adds up.  The
    bounds are those of the other decode tests: they know no length.  (Pages are
    shared: the reference weighs each by how often it is listed.)"""
    import torch
    import attention_forward_fa_gb300 as fa
    dt = torch.bfloat16 if dtype == "bf16" else torch.float16
    page, P_ = 256, 96
    g = torch.Generator(device="cuda").manual_seed(47)
    k = torch.randn(P_, 1, page, D, generator=g, device="cuda", dtype=dt)
    v = (1 + torch.rand(P_, 1, page, D, generator=g, device="cuda")).to(dt)
    t = torch.randint(P_, (B, n // page), generator=g, device="cuda").to(torch.int32)
    q = (0.1 * torch.randn(B, G, 1, D, generator=g, device="cuda")).to(dt)
    lens = torch.full((B,), n, device="cuda", dtype=torch.int32)
    o, l = fa.flash_attention_decode(q, fa.PagedKV(k, v, t), lens)
    assert _status() == 0
    u, sub, small = (2.0 ** -8, 0.0, 0.0) if dtype == "bf16" else (2.0 ** -11, 2.0 ** -25, 2.0 ** -32)
    for b in range(0, B, 9):
        w = torch.bincount(t[b].long(), minlength=P_).double()
        x = torch.einsum("gd,psd->gps", q[b, :, 0].double(), k[:, 0].double()) * D ** -0.5
        X = (torch.einsum("gd,psd->gps", q[b, :, 0].double().abs(), k[:, 0].double().abs()) * D ** -0.5).amax((1, 2))
        m = x.amax((1, 2))
        e = torch.exp(x - m[:, None, None]) * w[:, None]
        z = e.sum((1, 2))
        ref = torch.einsum("gps,psd->gd", e, v[:, 0].double()) / z[:, None]
        lim = (2 * 2.0 ** -16 * X + 2.0 ** -20 * X + 2.0 ** -15)[:, None] * ref + (u + 2.0 ** -20) * ref + sub
        lim += small * torch.einsum("p,psd->d", w, v[:, 0].double())
        err = (o[b, :, 0].double() - ref).abs()
        assert bool((err <= lim).all()), f"sequence {b}: O off by {(err / lim).max().item():.3g} of its bound"
        ll = (2.0 ** -16 + 2.0 ** -21) * X + 2.0 ** -20 * (1 + (m + torch.log(z)).abs())
        assert bool(((l[b, :, 0].double() - m - torch.log(z)).abs() <= ll).all())


def test_front_page_drafts_run():
    """The front page's padded step, behind its generation step, as written there."""
    import re
    from pathlib import Path
    import torch
    import attention_forward_fa_gb300 as fa
    text = (Path(__file__).resolve().parents[1] / "README.md").read_text()
    blocks = [b for b in re.findall(r"```python\n(.*?)```", text, re.S) if "paged_kv_append" in b]
    env = {"torch": torch, "fa": fa}
    torch.manual_seed(48)
    for i, b in enumerate(blocks):
        exec(compile(b, f"serving-example-{i}", "exec"), env)
    k, v, t = _host(env["k_pages"]), _host(env["v_pages"]), env["table"].cpu().numpy()
    for b, (m, n) in enumerate(((4, 1005), (2, 40))):
        q = _host(env["q"])[b:b + 1, :, :m]
        O, _, A, X, V = P.decode(q, k, v, t[b:b + 1], [n], 128 ** -0.5)
        lim = (2 * 2.0 ** -16 * X + 2.0 ** -20 * X + 2.0 ** -15)[..., None] * A + (2.0 ** -8 + 2.0 ** -20) * np.abs(O)
        assert (np.abs(_host(env["drafts"])[b:b + 1, :, :m] - O) <= lim).all()
