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
