"""The append kernel's looping form: every page that holds tokens once, by a
block that keeps to one item; and no instance of the kernel spills registers
(a loop around all kinds of pieces did, and took a fifth longer over large
prompts than a block per piece)."""
import re
import subprocess
from pathlib import Path

import pytest

from attention_forward_fa_gb300 import build as BUILD

CSRC = Path(BUILD.CSRC)


def test_no_instance_spills(tmp_path):
    names = [f"(void*)fa::fa_kv_append_kernel<{b}, {d}, {i}, {m}>"
             for b in ("true", "false") for d in (64, 128) for i in ("true", "false") for m in ("true", "false")]
    src = tmp_path / "append.cu"
    src.write_text('#include "fa_kv_append.cuh"\nvoid** all() {\n  static void* a[] = {%s};\n  return a;\n}\n' % ", ".join(names))
    r = subprocess.run([BUILD.nvcc_path(), *BUILD.ARCH, "-O3", "-std=c++17", "--expt-relaxed-constexpr", "-Xptxas", "-v",
                        "-I", str(CSRC), "-c", str(src), "-o", str(tmp_path / "append.o")], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    spills = [int(x) for x in re.findall(r"(\d+) bytes spill stores", r.stderr)]
    assert len(spills) == len(names) and not any(spills), spills


def looped(pieces, items, sms, holds):
    """The (item, page) pairs that the looping form takes, block by block, in order."""
    loop = int(re.search(r"kAppendLoopBlocks = (\d+);", (CSRC / "fa_kv_append.cuh").read_text())[1])
    grid = max(1, loop * sms // items) * items
    assert grid <= pieces
    pages, step = pieces // items, grid // items
    for block in range(grid):
        at0 = block // items
        while at0 < pages:
            for lane in range(32):
                at = at0 + step * lane
                if at < pages and holds(at):
                    yield block % items, at
            at0 += 32 * step


@pytest.mark.parametrize("items,pages,sms", [(24, 520, 4), (3, 12336, 152), (7, 1389, 1), (1000, 40, 5), (1, 1 << 15, 152)])
def test_the_looping_form_takes_every_page_once(items, pages, sms):
    blocks = int(re.search(r"kAppendBlocks = (\d+);", (CSRC / "fa_kv_append.cuh").read_text())[1])
    assert items * pages > blocks * sms        # the form's own range
    for holds in (lambda at: True, lambda at: at % 257 == 0 or at % 11 == 3):
        got = list(looped(items * pages, items, sms, holds))
        want = {(i, at) for i in range(items) for at in range(pages) if holds(at)}
        assert len(got) == len(want) and set(got) == want
