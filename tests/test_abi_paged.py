"""Argument checks of the paged entry points (fa_kv_append, fa_decode,
fa_select_pages): every refusal is synchronous, with the documented code, and
needs no GPU.  The wrappers' own checks run on CPU tensors."""
import ctypes

import pytest

from attention_forward_fa_gb300 import _binding as B
from attention_forward_fa_gb300 import build as BUILD

P = 0x10000   # a 16-byte aligned stand-in address; validation fails before any use


@pytest.fixture(scope="module", autouse=True)
def built():
    BUILD.build()
    return B.library()


@pytest.fixture(autouse=True)
def no_device_for_stand_in_addresses():
    """Stand-in addresses rely on the checks failing before any CUDA call, so
    that these run only where no GPU is visible."""
    import torch
    if torch.cuda.is_available():
        pytest.skip("stand-in device addresses: host-only check, no GPU may be visible")


def cache(**kw):
    a = dict(k=P, v=P, k_stride_page=8192, k_stride_head=2048, k_stride_slot=128,
             v_stride_page=8192, v_stride_head=2048, v_stride_slot=128, k_min=P, k_max=P,
             page_table=P, table_stride=8, max_pages=8, num_pages=64, page_size=16)
    a.update(kw)
    return B.fa_paged_kv_t(**a)


CACHE = [
    (dict(page_table=None), -1), (dict(k_min=None), -1), (dict(k_max=None), -1),
    (dict(page_size=0), -2), (dict(page_size=8), -2), (dict(page_size=48), -2),
    (dict(page_size=512), -2), (dict(num_pages=0), -2), (dict(max_pages=0), -2),
    (dict(table_stride=-1), -2), (dict(max_pages=(1 << 27) - 1), -2),
    (dict(page_table=P + 2), -4), (dict(k_min=P + 8), -4), (dict(k_max=P + 2), -4),
]
POOLS = [
    (dict(k=None), -1), (dict(v=None), -1), (dict(k_stride_page=-8), -2),
    (dict(v_stride_slot=0), -2), (dict(k_stride_head=0), -2), (dict(v_stride_page=0), -2),
    (dict(k_stride_page=1 << 38), -2), (dict(k_stride_slot=124), -4), (dict(v_stride_head=2052), -4),
    (dict(k=P + 8), -4), (dict(v=P + 2), -4),
]
SHAPE = [
    (dict(B=0), -2), (dict(Hq=3), -2), (dict(Hkv=0), -2), (dict(S=0), -2), (dict(D=0), -2),
    (dict(D=96), -3), (dict(D=256), -3), (dict(mask_mode=1), -2), (dict(mask_mode=0x200), -2),
]


def decode(kv=None, **kw):
    a = dict(q=P, o=P, lse=P, B=1, Hq=8, Hkv=2, S=1, D=128, scale=0.1, mask_mode=0, kv_lens=P,
             pre_tokens=-1, page_idx=None, max_sel=0)
    a.update(kw)
    return B.fa_decode(a["q"], kv if kv is not None else cache(), a["o"], a["lse"], a["B"], a["Hq"],
                       a["Hkv"], a["S"], a["D"], a["scale"], a["mask_mode"], a["kv_lens"],
                       a["pre_tokens"], a["page_idx"], a["max_sel"], 0)


def select(kv=None, **kw):
    a = dict(q=P, page_idx=P, B=1, Hq=8, Hkv=2, S=1, D=128, mask_mode=0, kv_lens=P, max_sel=4,
             first=1, last=1)
    a.update(kw)
    return B.fa_select_pages(a["q"], kv if kv is not None else cache(), a["page_idx"], a["B"], a["Hq"],
                             a["Hkv"], a["S"], a["D"], a["mask_mode"], a["kv_lens"], a["max_sel"],
                             a["first"], a["last"], 0)


def append(kv=None, new=None, **kw):
    a = dict(B=2, Hq=8, Hkv=2, S=3, D=128, mask_mode=0, kv_lens=P, new_lens=None)
    a.update(kw)
    n = dict(k=P, v=P, q=P, q_out=P, cos=P, sin=P, rot_dim=64, interleaved=0, max_pos=100)
    n.update({f"{t}_stride_{d}": 1024 for t in ("k", "v", "q", "qo") for d in "bhs"})
    n.update(new or {})
    return B.fa_kv_append(kv if kv is not None else cache(), B.fa_kv_new_t(**n), a["B"], a["Hq"],
                          a["Hkv"], a["S"], a["D"], a["mask_mode"], a["kv_lens"], a["new_lens"], 0)


@pytest.mark.parametrize("kw,code", CACHE)
@pytest.mark.parametrize("call", [decode, select, append])
def test_cache_struct(call, kw, code):
    assert call(kv=cache(**kw)) == code


@pytest.mark.parametrize("kw,code", POOLS)
@pytest.mark.parametrize("call", [decode, append])
def test_pools(call, kw, code):
    assert call(kv=cache(**kw)) == code


@pytest.mark.parametrize("kw,code", SHAPE)
@pytest.mark.parametrize("call", [decode, select, append])
def test_shapes(call, kw, code):
    assert call(**kw) == code


@pytest.mark.parametrize("kw", [
    dict(B=(1 << 31) - 1, Hq=(1 << 31) - 2, S=(1 << 31) - 1),        # past 64 bits as a product
    dict(B=1 << 30, Hq=1 << 30, S=16), dict(B=1 << 16, S=1 << 12), dict(S=(1 << 28) - 8192 + 1),
])
@pytest.mark.parametrize("call", [decode, select, append])
def test_more_rows_than_32_bits_count(call, kw):
    assert call(**kw) == -2


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), -1), (dict(o=None), -1), (dict(lse=None), -1), (dict(kv_lens=None), -1),
    (dict(scale=float("nan")), -2), (dict(scale=float("inf")), -2), (dict(pre_tokens=-2), -2),
    (dict(page_idx=P), -2), (dict(page_idx=P, max_sel=(1 << 20) + 1), -2),
    (dict(B=1 << 16, Hq=1 << 16, Hkv=1), -2),
    (dict(q=P + 8), -4), (dict(o=P + 4), -4), (dict(lse=P + 2), -4), (dict(kv_lens=P + 2), -4),
    (dict(page_idx=P + 2, max_sel=4), -4),
])
def test_decode_arguments(kw, code):
    assert decode(**kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), -1), (dict(page_idx=None), -1), (dict(kv_lens=None), -1), (dict(max_sel=0), -2),
    (dict(max_sel=1), -2), (dict(first=-1), -2), (dict(last=-1), -2), (dict(first=3, last=2), -2),
    (dict(max_sel=(1 << 20) + 1), -2), (dict(q=P + 8), -4), (dict(page_idx=P + 1), -4),
])
def test_select_arguments(kw, code):
    assert select(**kw) == code


def test_select_needs_bounds():
    assert select(kv=cache(k_min=None, k_max=None)) == -1


@pytest.mark.parametrize("new,kw,code", [
    (dict(k=None), {}, -1), (dict(v=None), {}, -1), (dict(q=None), {}, -1), (dict(q_out=None), {}, -1),
    (dict(cos=None), {}, -1), (dict(sin=None), {}, -1), ({}, dict(kv_lens=None), -1),
    (dict(rot_dim=24), {}, -2), (dict(rot_dim=144), {}, -2), (dict(rot_dim=-16), {}, -2),
    (dict(interleaved=2), {}, -2), (dict(max_pos=0), {}, -2), (dict(k_stride_b=-8), {}, -2),
    (dict(q_stride_s=-8), {}, -2), (dict(qo_stride_s=2048), {}, -2),
    (dict(k_stride_s=1020), {}, -4), (dict(v_stride_h=4), {}, -4), (dict(q_stride_b=4, qo_stride_b=4), {}, -4),
    (dict(q_out=P + 16, qo_stride_s=0), {}, -2), (dict(v_stride_b=1 << 38), {}, -2),
    (dict(k=P + 8), {}, -4), (dict(q=P + 8), {}, -4), (dict(cos=P + 4), {}, -4),
    ({}, dict(new_lens=P + 1), -4), ({}, dict(B=1 << 30, S=1 << 10), -2),
])
def test_append_arguments(new, kw, code):
    assert append(new=new, **kw) == code


def test_append_struct_is_required():
    lib = B.library()
    null = ctypes.POINTER(B.fa_kv_new_t)()
    assert lib.fa_kv_append(cache(), null, 1, 8, 2, 1, 128, 0, P, None, None) == -1
    assert lib.fa_decode(P, ctypes.POINTER(B.fa_paged_kv_t)(), P, P, 1, 8, 2, 1, 128, 0.1, 0, P, -1,
                         None, 0, None) == -1


def test_cache_object_refuses_what_is_no_cache():
    import torch
    k = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16)
    t = torch.zeros(1, 4, dtype=torch.int32)
    with pytest.raises(TypeError):
        B.PagedKV(k.float(), k.float(), t)
    for a in ((k, k[..., :32], t), (k, k, t.long()), (k, k, t[0]), (k, k, t, k[:, :, 0]),
              (k[0], k[0], t), (k, k, t)):        # the last: CPU tensors
        with pytest.raises(ValueError):
            B.PagedKV(*a)


def test_error_string_of_paged_calls():
    assert "page" in B.fa_strerror(B.FA_ERR_INDEX)


def test_wrappers_refuse_a_stream_of_another_device():
    import torch

    class Other:
        device = torch.device("cuda", 1)
        cuda_stream = 0

    with pytest.raises(ValueError):
        B._elsewhere(torch.device("cuda", 0), Other(), lambda raw: pytest.fail("called"))
