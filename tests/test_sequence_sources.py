"""Orders in the kernels' sources that no run can show to be wrong without hanging a device."""
from __future__ import annotations

import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "mapreduce_prefix_scan_gb300", "csrc")


def _kernel(file, name):
    """A kernel's body without its comments."""
    with open(os.path.join(CSRC, file)) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    body = text[re.search(r"\b%s\s*\(" % name, text).end():]
    end = re.search(r"^}", body, re.M)
    return body[:end.start()]


def test_a_fold_has_its_tensor_memory_before_the_main_pass_may_start():
    """Blocks of the main pass allocate tensor memory and then wait for the fold pass to end. If they could start
    before every block of the fold pass has its own, a fold block could wait for them and they for it."""
    body = _kernel("linattn_mma.cu", "k_chunks")
    allocated, started = body.index("tmem_alloc("), body.index("griddep_launch_dependents(")
    assert allocated < body.index("__syncthreads()", allocated) < started
    assert body.count("griddep_launch_dependents(") == 1
    assert "return;" not in body[:allocated]


def test_nothing_is_issued_after_a_wait_that_ran_out():
    """Copies and products are issued by `leader` alone, which a wait of its own that ran out takes away; and the block
    gives up its tensor memory only after it has waited for the products and copies in flight."""
    body = _kernel("linattn_mma.cu", "k_chunks")
    assert re.search(r"!wait_long\([^;]*\)\) leader = 0;", body)
    walk = body[body.index("while (c.valid)"):]
    issued = re.findall(r"mma_(?:ss|ts|commit)\((?:[^;]*?)(\w+)\);", walk)
    assert len(issued) >= 8 and [x for x in issued if x != "leader"] == ["1"]  # the last one waits for all of them
    loads = [m.start() for m in re.finditer(r"tma_load_3d\(", body)]
    assert loads and all("if (leader) {" in body[at - 300:at] for at in loads)
    assert walk.index("mma_commit(&t.drained, 1)") < walk.index("mbar_wait(&t.drained") < walk.index("tmem_free(")
