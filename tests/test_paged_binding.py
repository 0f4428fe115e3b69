"""What the paged wrappers hand to the library, recorded by a stand-in for it:
numbers past 32 bits keep their meaning instead of losing their upper bits."""
import ctypes

import pytest
import torch

from attention_forward_fa_gb300 import _binding as B

BIG = 2 ** 31 - 1


class Recorder:
    """Takes the calls with the C entry points' own argument types."""

    def __init__(self, real):
        self.calls = []
        for name in ("fa_kv_append", "fa_decode", "fa_select_pages"):
            types = getattr(real, name).argtypes
            setattr(self, name, lambda *a, types=types, name=name: self.take(name, a, types))

    def take(self, name, args, types):
        assert len(args) == len(types)
        got = [t(a).value if t is ctypes.c_int else a for a, t in zip(args, types)]
        self.calls.append((name, got))
        return 0


@pytest.fixture
def lib(monkeypatch):
    from attention_forward_fa_gb300 import build
    build.build()
    rec = Recorder(B.library())
    monkeypatch.setattr(B, "library", lambda: rec)
    monkeypatch.setattr(B, "_elsewhere", lambda device, stream, call: call(0))
    return rec


def cpu_cache(**kw):
    """A cache object around CPU tensors (its constructor wants CUDA ones)."""
    c = object.__new__(B.PagedKV)
    k = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16)
    a = dict(k_pages=k, v_pages=k, page_table=torch.zeros(1, 4, dtype=torch.int32), k_min=k[:, :, 0], k_max=k[:, :, 0],
             dtype=k.dtype, device=k.device, B=1, Hkv=2, D=64, page_size=16, num_pages=4, max_pages=4, _flags=0,
             _c=B.fa_paged_kv_t())
    a.update(kw)
    for name, x in a.items():
        setattr(c, name, x)
    return c


Q = torch.zeros(1, 4, 1, 64, dtype=torch.bfloat16)
N = torch.ones(1, dtype=torch.int32)


@pytest.mark.parametrize("pre,want", [(None, -1), (0, 0), (5, 5), (BIG, BIG), (2 ** 31, BIG), (2 ** 32, BIG),
                                      (2 ** 32 + 7, BIG), (2 ** 63 - 1, BIG)])
def test_a_window_of_any_length(lib, pre, want):
    B.flash_attention_decode(Q, cpu_cache(), N, pre_tokens=pre, stream=1)
    (name, got), = lib.calls
    assert name == "fa_decode" and got[12] == want


@pytest.mark.parametrize("first,last", [(2 ** 32, 0), (0, 2 ** 32 + 1), (2 ** 33, 2 ** 32), (-2 ** 32, 1)])
def test_forced_pages_past_32_bits(lib, first, last):
    B.select_kv_pages(Q, cpu_cache(), N, 4, first=first, last=last, stream=1)
    (name, got), = lib.calls
    assert name == "fa_select_pages"
    for x, y in ((first, got[11]), (last, got[12])):
        assert y == max(-2 ** 31, min(x, BIG))


@pytest.mark.parametrize("bad", [3.5, "7", 2.0 ** 40])
def test_what_is_no_whole_number_is_refused(lib, bad):
    with pytest.raises((TypeError, ctypes.ArgumentError)):
        B.flash_attention_decode(Q, cpu_cache(), N, pre_tokens=bad, stream=1)
    with pytest.raises((TypeError, ctypes.ArgumentError)):
        B.select_kv_pages(Q, cpu_cache(), N, 4, first=bad, stream=1)
    assert not lib.calls


def test_direct_calls(lib):
    kv, new = B.fa_paged_kv_t(), B.fa_kv_new_t()
    assert B.fa_decode(0, kv, 0, 0, 2 ** 32 + 1, 8, 2, 1, 128, 1.0, 0, 0, 2 ** 32, None, 2 ** 32 + 4, 0) == 0
    assert lib.calls[-1][1][4] == BIG and lib.calls[-1][1][12] == BIG and lib.calls[-1][1][14] == BIG
    assert B.fa_select_pages(0, kv, 0, 1, 8, 2, 2 ** 32, 128, 0, 0, 2 ** 32 + 4, 2 ** 32, -2 ** 40, 0) == 0
    assert lib.calls[-1][1][6] == BIG and lib.calls[-1][1][10:13] == [BIG, BIG, -2 ** 31]
    assert B.fa_kv_append(kv, new, 1, 8, 2, 2 ** 32 + 3, 128, 2 ** 32, 0, None, 0) == 0
    assert lib.calls[-1][1][5] == BIG and lib.calls[-1][1][7] == BIG


def test_tables_of_more_positions_than_32_bits_count(lib):
    """cos and sin of 2**32 + 5 rows (views of one row): every position has one."""
    rows = torch.zeros(1, 8).expand(2 ** 32 + 5, 8)

    class Rows:                      # contiguous as far as the wrapper can tell
        shape, dtype, device = rows.shape, rows.dtype, rows.device
        dim, is_contiguous, data_ptr = rows.dim, staticmethod(lambda: True), rows.data_ptr

    seen = {}
    lib.fa_kv_append = lambda kv, x, *a: seen.update(max_pos=x.max_pos, rot=x.rot_dim) or 0
    x = torch.zeros(1, 2, 1, 64, dtype=torch.bfloat16)
    B.paged_kv_append(cpu_cache(), N, x, x, cos=Rows, sin=Rows, stream=1)
    assert seen == {"max_pos": BIG, "rot": 16}


@pytest.mark.parametrize("scale", [2.4e38, -3e38, 1e39, float("nan")])
def test_a_scale_past_fp32_in_log2_units_is_refused(scale):
    """Scores are taken in log2 units: 2.4e38 * log2(e) is no fp32 number, and
    every score would be infinite or NaN."""
    if torch.cuda.is_available():
        pytest.skip("stand-in device addresses: no GPU may be visible")
    from attention_forward_fa_gb300 import build
    build.build()
    P = 0x10000
    kv = B.fa_paged_kv_t(k=P, v=P, k_stride_page=8192, k_stride_head=2048, k_stride_slot=128, v_stride_page=8192,
                         v_stride_head=2048, v_stride_slot=128, page_table=P, table_stride=8, max_pages=8,
                         num_pages=64, page_size=16)
    assert B.fa_decode(P, kv, P, P, 1, 8, 2, 1, 128, scale, 0, P, -1, None, 0, 0) == B.FA_ERR_SHAPE
