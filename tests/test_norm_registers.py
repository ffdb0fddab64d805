"""The norm's kernels hold a row in registers: what the compiler says of each variant when the
library is built."""
import os
import re

import pytest

from scaled_quantize_fp8_gb300 import build as B


def _usage(source):
    """Mangled name of a kernel -> (registers, bytes of spill stores), from the build's log."""
    log = os.path.join(B.OBJDIR, source[:-3] + ".log")
    B.build()
    if not os.path.exists(log):
        os.makedirs(B.OBJDIR, exist_ok=True)
        B._compile(B._nvcc(), os.path.join(B.CSRC, source))
    with open(log) as f:
        text = f.read()
    found = re.findall(r"Compiling entry function '(\S+)'.*?(\d+) bytes spill stores.*?"
                       r"Used (\d+) registers", text, re.S)
    return {name: (int(regs), int(spill)) for name, spill, regs in found}


@pytest.mark.parametrize("source,kernel,variants", [("norm.cu", "norm_row_kernel", 32),
                                                    ("norm_bwd.cu", "norm_bwd_kernel", 16)])
def test_no_variant_spills(source, kernel, variants):
    use = {n: v for n, v in _usage(source).items() if kernel in n}
    assert len(use) == variants
    assert {n: v for n, v in use.items() if v[1] != 0} == {}
