"""The build refuses a compiler that gives another register count to the kernels
that exchange registers, whose calls would all be refused."""
import os
import re

import pytest

from draft_verification_sdv_gb300 import build as sdv_build

LINE = ("ptxas info    : Compiling entry function '%s' for 'sm_103a'\n"
        "ptxas info    : Function properties for %s\n"
        "    0 bytes stack frame, 0 bytes spill stores, 0 bytes spill loads\n"
        "ptxas info    : Used %d registers, used 16 barriers\n")


def _report(*counts):
    return "".join(LINE % (("_ZN3sdv14attn_tc_kernelILb%dE" % i,) * 2 + (n,)) for i, n in enumerate(counts))


def test_register_counts():
    src = "k8_attn_tc.cu"
    other = LINE % ("_ZN3sdv5otherE", "_ZN3sdv5otherE", 40)
    sdv_build.check_registers(src, other + _report(168, 168))
    for report in (_report(168, 160), _report(), other, _report(170)):
        with pytest.raises(RuntimeError, match="168"):
            sdv_build.check_registers(src, report)


def test_the_count_is_the_kernels_own():
    for src, (kernel, want) in sdv_build.REGISTERS.items():
        text = open(os.path.join(sdv_build.CSRC, src)).read()
        assert kernel in text and re.search(r"kRegs = %d;" % want, text)
