"""Argument checks of fa_kv_append_ext, fa_decode_ext, fa_kv_read and fa_kv_keep: every
refusal is synchronous, with the documented code, and needs no GPU."""
import ctypes

import pytest

from attention_forward_fa_gb300 import _binding as B
from attention_forward_fa_gb300 import build as BUILD
from tests.test_abi_paged import CACHE, POOLS, SHAPE, cache

P = 0x10000


@pytest.fixture(scope="module", autouse=True)
def built():
    BUILD.build()
    return B.library()


@pytest.fixture(autouse=True)
def no_device_for_stand_in_addresses():
    import torch
    if torch.cuda.is_available():
        pytest.skip("stand-in device addresses: host-only check, no GPU may be visible")


def fp8(**kw):
    return B.fa_kv_fp8_t(**{**dict(k_scale=P, v_scale=P, format=0), **kw})


def tree(**kw):
    return B.fa_tree_t(**{**dict(ancestors=P, stride_b=9, new_lens=None), **kw})


def decode(kv=None, f=None, t=None, **kw):
    a = dict(q=P, o=P, lse=P, B=1, Hq=8, Hkv=2, S=3, D=128, scale=0.1, mask_mode=0, kv_lens=P, pre_tokens=-1,
             page_idx=None, max_sel=0)
    a.update(kw)
    return B.fa_decode_ext(a["q"], kv if kv is not None else cache(), f, a["o"], a["lse"], a["B"], a["Hq"], a["Hkv"], a["S"],
                           a["D"], a["scale"], a["mask_mode"], a["kv_lens"], a["pre_tokens"], a["page_idx"], a["max_sel"], t, 0)


def append(kv=None, f=None, new=None, **kw):
    a = dict(B=2, Hq=8, Hkv=2, S=3, D=128, mask_mode=0, kv_lens=P, new_lens=None, positions=P)
    a.update(kw)
    n = dict(k=P, v=P, q=P, q_out=P, cos=P, sin=P, rot_dim=64, interleaved=0, max_pos=100)
    n.update({f"{t}_stride_{d}": 1024 for t in ("k", "v", "q", "qo") for d in "bhs"})
    n.update(new or {})
    return B.fa_kv_append_ext(kv if kv is not None else cache(), f, B.fa_kv_new_t(**n), a["B"], a["Hq"], a["Hkv"], a["S"],
                              a["D"], a["mask_mode"], a["kv_lens"], a["new_lens"], a["positions"], 0)


def read(kv=None, f=None, out=None, **kw):
    a = dict(B=2, Hkv=2, S=3, D=128, mask_mode=0, starts=P, lens=P)
    a.update(kw)
    o = dict(k=P, v=P, **{f"{t}_stride_{d}": 1024 for t in "kv" for d in "bhs"})
    o.update(out or {})
    return B.fa_kv_read(kv if kv is not None else cache(), f, B.fa_kv_rows_t(**o), a["B"], a["Hkv"], a["S"], a["D"],
                        a["mask_mode"], a["starts"], a["lens"], 0)


def keep(kv=None, f=None, **kw):
    a = dict(B=2, Hkv=2, D=128, mask_mode=0, kv_lens=P, keep_idx=P, M=4, keep_lens=P)
    a.update(kw)
    return B.fa_kv_keep(kv if kv is not None else cache(), f, a["B"], a["Hkv"], a["D"], a["mask_mode"], a["kv_lens"],
                        a["keep_idx"], a["M"], a["keep_lens"], 0)


ALL = [decode, append, read, keep]


@pytest.mark.parametrize("kw,code", CACHE + POOLS)
@pytest.mark.parametrize("call", ALL)
def test_cache_struct(call, kw, code):
    assert call(kv=cache(**kw)) == code
    assert call(kv=cache(**kw), f=fp8()) == code


@pytest.mark.parametrize("kw,code", SHAPE)
@pytest.mark.parametrize("call", ALL)
def test_shapes(call, kw, code):
    if call in (read, keep) and "Hq" in kw or call is keep and "S" in kw:
        pytest.skip("no such argument")
    assert call(**kw) == code
    assert call(f=fp8(), **kw) == code


@pytest.mark.parametrize("kv,f,code", [
    ({}, dict(k_scale=None), -1), ({}, dict(v_scale=None), -1), ({}, dict(format=2), -2), ({}, dict(format=-1), -2),
    ({}, dict(k_scale=P + 8), -4), ({}, dict(v_scale=P + 1), -4),
    (dict(k_stride_slot=136), {}, -4), (dict(v_stride_page=8200), {}, -4), (dict(k_stride_head=2056), {}, -4),   # multiples of 8 only
])
@pytest.mark.parametrize("call", ALL)
def test_8_bit_cache(call, kv, f, code):
    assert call(kv=cache(**kv), f=fp8(**f)) == code


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), -1), (dict(o=None), -1), (dict(lse=None), -1), (dict(kv_lens=None), -1),
    (dict(scale=float("nan")), -2), (dict(pre_tokens=-2), -2), (dict(page_idx=P), -2),
    (dict(B=1 << 16, Hq=1 << 16, Hkv=1), -2), (dict(q=P + 8), -4), (dict(o=P + 4), -4), (dict(lse=P + 2), -4),
    (dict(kv_lens=P + 2), -4), (dict(page_idx=P + 2, max_sel=4), -4),
    (dict(t=tree(ancestors=None)), -1), (dict(t=tree(stride_b=-1)), -2), (dict(t=tree(new_lens=P + 2)), -4),
    (dict(t=tree(), pre_tokens=0), -3), (dict(t=tree(), page_idx=P, max_sel=4), -3),
])
@pytest.mark.parametrize("f", [None, fp8()])
def test_decode_arguments(f, kw, code):
    assert decode(f=f, **kw) == code


@pytest.mark.parametrize("new,kw,code", [
    (dict(k=None), {}, -1), (dict(q_out=None), {}, -1), (dict(cos=None), {}, -1), ({}, dict(kv_lens=None), -1),
    (dict(rot_dim=24), {}, -2), (dict(interleaved=2), {}, -2), (dict(max_pos=0), {}, -2), (dict(k_stride_s=1020), {}, -4),
    (dict(k=P + 8), {}, -4), ({}, dict(new_lens=P + 1), -4), ({}, dict(positions=P + 2), -4), ({}, dict(B=1 << 30, S=1 << 10), -2),
])
@pytest.mark.parametrize("f", [None, fp8()])
def test_append_arguments(f, new, kw, code):
    assert append(f=f, new=new, **kw) == code


@pytest.mark.parametrize("out,kw,code", [
    (dict(k=None), {}, -1), (dict(v=None), {}, -1), ({}, dict(lens=None), -1), (dict(k_stride_b=-8), {}, -2),
    (dict(v_stride_s=0), {}, -2), (dict(k_stride_h=0), {}, -2), (dict(v_stride_h=1028), {}, -4), (dict(k=P + 8), {}, -4),
    (dict(v=P + 2), {}, -4), ({}, dict(starts=P + 2), -4), ({}, dict(lens=P + 1), -4), (dict(k_stride_s=1 << 38), {}, -2),
    ({}, dict(B=1 << 30, S=1 << 10), -2), ({}, dict(S=(1 << 31) - 1), -2),
])
@pytest.mark.parametrize("f", [None, fp8()])
def test_read_arguments(f, out, kw, code):
    assert read(f=f, out=out, **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(kv_lens=None), -1), (dict(keep_idx=None), -1), (dict(keep_lens=None), -1), (dict(M=0), -2), (dict(M=-4), -2),
    (dict(kv_lens=P + 2), -4), (dict(keep_idx=P + 2), -4), (dict(keep_lens=P + 1), -4), (dict(B=(1 << 31) - 1, Hkv=64), -2),
])
@pytest.mark.parametrize("f", [None, fp8()])
def test_keep_arguments(f, kw, code):
    assert keep(f=f, **kw) == code


def test_structs_are_required():
    lib = B.library()
    no_kv, no_new, no_rows = (ctypes.POINTER(t)() for t in (B.fa_paged_kv_t, B.fa_kv_new_t, B.fa_kv_rows_t))
    assert lib.fa_kv_append_ext(cache(), None, no_new, 1, 8, 2, 1, 128, 0, P, None, None, None) == -1
    assert lib.fa_decode_ext(P, no_kv, None, P, P, 1, 8, 2, 1, 128, 0.1, 0, P, -1, None, 0, None, None) == -1
    assert lib.fa_kv_read(cache(), None, no_rows, 1, 2, 1, 128, 0, P, P, None) == -1
    assert lib.fa_kv_keep(no_kv, None, 1, 2, 128, 0, P, P, 1, P, None) == -1


def test_cache_object_refuses_what_is_no_8_bit_cache():
    import torch
    k = torch.zeros(4, 2, 16, 64, dtype=torch.uint8)
    s, t = torch.zeros(4, 2, 16, dtype=torch.uint8), torch.zeros(1, 4, dtype=torch.int32)
    with pytest.raises(TypeError):
        B.PagedKV(k, k, t, k_scale=s, v_scale=s)              # plain bytes name no format
    f = k.view(torch.float8_e4m3fn)
    with pytest.raises(TypeError):
        B.PagedKV(f, f, t, k_scale=s, v_scale=s, dtype=torch.float32)
    b = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        B.PagedKV(b, b, t, dtype=torch.float16)
    for a, kw in (((f, f, t), {}), ((b, b, t), dict(k_scale=s, v_scale=s)), ((f, f, t), dict(k_scale=s, v_scale=s))):   # the last: CPU tensors
        with pytest.raises(ValueError):
            B.PagedKV(*a, **kw)
