"""Registers of the append kernel's forms beside the plain one (tests/test_append_pieces.py): with positions
given, into a 16-bit cache, none spills; into an 8-bit cache each does, by no more than the few bytes that
its comment names."""
import re
import subprocess
from pathlib import Path

import pytest

from attention_forward_fa_gb300 import build as BUILD

CSRC = Path(BUILD.CSRC)


@pytest.mark.parametrize("form,most", [("fa::kAppendPlaced", 0), ("fa::kAppend8", 20)])
def test_spills(tmp_path, form, most):
    names = [f"(void*)fa::fa_kv_append_kernel<{b}, 128, {i}, {m}, {form}>" for b in ("true", "false")
             for i in ("true", "false") for m in ("true", "false")]
    src = tmp_path / "append.cu"
    src.write_text('#include "fa_kv_append.cuh"\nvoid** all() {\n  static void* a[] = {%s};\n  return a;\n}\n' % ", ".join(names))
    r = subprocess.run([BUILD.nvcc_path(), *BUILD.ARCH, "-O3", "-std=c++17", "--expt-relaxed-constexpr", "-Xptxas", "-v",
                        "-I", str(CSRC), "-c", str(src), "-o", str(tmp_path / "append.o")], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    spills = [int(x) for x in re.findall(r"(\d+) bytes spill stores", r.stderr)]
    assert len(spills) == len(names) and max(spills) <= most, spills
