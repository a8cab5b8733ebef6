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


def test_no_further_chunk_is_asked_for_after_a_wait_that_ran_out():
    """The issuing warp leaves its walk before it arms a barrier for another chunk's copies, whose last copies may still
    be under way; and the block gives up its tensor memory only after it has waited for the products and copies in
    flight."""
    body = _kernel("linattn_mma.cu", "k_chunks")
    walk = body[body.index("while (c.valid)"):]
    asked = [m.start() for m in re.finditer(r"load_[qv]\(c2", walk)]  # these announce a chunk's bytes
    left = [m.start() for m in re.finditer(r"if \(!?FOLD && lost\(\)\) break;", walk)]
    assert len(left) == 2 and min(left) < min(asked)
    assert walk.index("!FOLD && lost()") < walk.index("load_q(c2)")
    assert walk.index("if (lost())") < walk.index("mma_commit(&t.drained") < walk.index("mbar_wait(&t.drained")
    assert walk.index("mbar_wait(&t.qk[stage]") < walk.index("tmem_free(")
