"""What the wrappers of the appending and reading calls hand to the library (recorded by a stand-in for
it): numbers of tokens past 32 bits keep their meaning, so that the library refuses them."""
import ctypes

import pytest
import torch

from attention_forward_fa_gb300 import _binding as B
from tests.test_paged_binding import BIG, N, cpu_cache


@pytest.fixture
def lib(monkeypatch):
    from attention_forward_fa_gb300 import build
    build.build()
    real, calls = B.library(), []

    class Recorder:
        pass

    rec = Recorder()
    rec.calls = calls
    for name in ("fa_kv_append", "fa_kv_append_ext", "fa_kv_read"):
        types = getattr(real, name).argtypes

        def take(*a, name=name, types=types):
            assert len(a) == len(types)
            calls.append((name, [t(x).value if t is ctypes.c_int else x for x, t in zip(a, types)]))
            return 0
        setattr(rec, name, take)
    monkeypatch.setattr(B, "library", lambda: rec)
    monkeypatch.setattr(B, "_elsewhere", lambda device, stream, call: call(0))
    return rec


def rows(S):
    """[1, 2, S, 64] of one row."""
    return torch.zeros(1, 2, 1, 64, dtype=torch.bfloat16).expand(1, 2, S, 64)


@pytest.mark.parametrize("S,want", [(1, 1), (7, 7), (BIG, BIG), (2 ** 32 + 1, BIG), (2 ** 33, BIG)])
def test_numbers_of_tokens(lib, S, want):
    B.paged_kv_read(cpu_cache(), N, k_out=rows(S), v_out=rows(S), stream=1)
    name, got = lib.calls.pop()
    assert name == "fa_kv_read" and got[5] == want
    B.paged_kv_append(cpu_cache(), N, rows(S), rows(S), stream=1)
    name, got = lib.calls.pop()
    assert name == "fa_kv_append" and got[5] == want
    cache = cpu_cache()
    cache._fp8 = B.fa_kv_fp8_t()
    B.paged_kv_append(cache, N, rows(S), rows(S), stream=1)
    name, got = lib.calls.pop()
    assert name == "fa_kv_append_ext" and got[6] == want
