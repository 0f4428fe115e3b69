"""Scratch of the paged calls where the device cannot be asked for its SMs: a
call that fails before its launch must not have taken any.  The library's own
helpers are replaced by fakes (a preloaded library) in a process of its own;
nothing runs on a GPU."""
import os
import subprocess
import sys
from pathlib import Path

import pytest

from attention_forward_fa_gb300 import build as BUILD

ROOT = Path(__file__).resolve().parents[1]

FAKE = """
#include <cstdlib>
#include <cstddef>
struct CUstream_st;
static int taken = 0;
static int word[4];
namespace fa_host {
int* status_ptr() { return word; }
void* scratch_alloc(size_t bytes, CUstream_st*) { ++taken; return std::malloc(bytes); }
int sm_count() { return 0; }
}
extern "C" int scratch_taken() { return taken; }
"""

CALL = """
import ctypes, sys
sys.path.insert(0, sys.argv[1])
from attention_forward_fa_gb300 import _binding as B
P = 0x10000
kv = B.fa_paged_kv_t(k=P, v=P, k_stride_page=8192, k_stride_head=2048, k_stride_slot=128, v_stride_page=8192,
                     v_stride_head=2048, v_stride_slot=128, k_min=P, k_max=P, page_table=P, table_stride=8,
                     max_pages=8, num_pages=64, page_size=16)
code = B.fa_select_pages(P, kv, P, 1, 8, 2, 1, 128, 0, P, 4, 1, 1, 0)
fake = ctypes.CDLL(sys.argv[2])
print("code", code, "taken", fake.scratch_taken())
"""


def test_a_choice_that_cannot_launch_takes_no_scratch(tmp_path):
    import torch
    if torch.cuda.is_available():
        pytest.skip("stand-in device addresses: no GPU may be visible")
    BUILD.build()
    (tmp_path / "fake.cpp").write_text(FAKE)
    lib = tmp_path / "libfake.so"
    subprocess.run(["g++", "-shared", "-fPIC", "-o", str(lib), str(tmp_path / "fake.cpp")], check=True)
    r = subprocess.run([sys.executable, "-c", CALL, str(ROOT), str(lib)], capture_output=True, text=True,
                       env=dict(os.environ, LD_PRELOAD=str(lib)))
    assert r.returncode == 0, r.stderr[-2000:]
    assert r.stdout.split() == ["code", "-6", "taken", "0"], r.stdout
