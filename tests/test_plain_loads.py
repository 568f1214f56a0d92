"""Every kernel may start while the kernel before it on the stream still writes
(programmatic dependent launch), and the read-only path is defined for memory that
nothing writes while the kernel runs: what was loaded through it before the wait, or
lies in its cache, need not be what the kernel before wrote."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "combine_moonep_plan_gb300", "csrc")
# launched in the ordinary way, after all before them has ended
ORDINARY = {"plan.cu": ("plan_hist_kernel", "plan_balance_kernel", "plan_assign_kernel")}


@pytest.mark.parametrize("name", sorted(f for f in os.listdir(CSRC) if f.endswith((".cu", ".cuh"))))
def test_no_load_through_the_read_only_path(name):
    with open(os.path.join(CSRC, name)) as f:
        code = re.sub(r"//[^\n]*|/\*.*?\*/", "", f.read(), flags=re.S)
    for kernel in ORDINARY.get(name, ()):
        assert re.search(kernel + r"(<\w+>)?<<<", code)
        # the definition, to the brace in the first column
        code, n = re.subn(r"\n" + kernel + r"\(.*?\n}", "", code, flags=re.S)
        assert n == 1
    assert not re.search(r"__ldg\b|ld\.global(\.\w+)*\.nc\b|__restrict__", code)
