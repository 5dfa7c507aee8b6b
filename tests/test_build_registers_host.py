"""The build refuses kernels that were compiled to another number of registers than
the one that they share out between their warps (no GPU needed)."""
import os

import pytest

from causal_conv_backward_gb300 import build as cbuild

LINE = "ptxas info    : Used {} registers, used 2 barriers\n"


def source(name):
    return os.path.join(cbuild.CSRC, name)


@pytest.mark.parametrize("name", ["delta_chunks.cu", "delta_chunks_bwd.cu"])
def test_another_number_is_refused(name):
    n = cbuild.launch_registers(source(name))
    assert n > 0
    cbuild.check_registers(source(name), LINE.format(n) * 4)
    for log in (LINE.format(n) * 3 + LINE.format(n - 8), LINE.format(n + 8), ""):
        with pytest.raises(RuntimeError, match=name):
            cbuild.check_registers(source(name), log)


def test_other_sources_take_what_they_get():
    assert cbuild.launch_registers(source("delta_step.cu")) == 0
    cbuild.check_registers(source("delta_step.cu"), LINE.format(40))
