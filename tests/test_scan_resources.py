"""CTAs per SM that the scan's forward counts on, from ptxas's report on the CPU: two in
bf16 where shared memory holds two (more than 8 states, the output pass over whole
rows of B and C; with 9 to 16 states in every form)."""
import os

import pytest

from linear_rnn_mlstm_b200 import build as libbuild
from test_kernel_resources import _named, _ptxas_report

REGISTERS = 65536


@pytest.fixture(scope="module")
def report():
    return _ptxas_report(os.path.join(libbuild.CSRC, "scan.cu"))


@pytest.mark.parametrize("lanes,out,whole,threads", [(8, 0, 0, 384), (8, 0, 1, 384), (8, 1, 0, 384), (8, 1, 1, 384), (16, 1, 1, 512),
                                                      (32, 1, 1, 512)])
def test_two_ctas_of_the_scan_fit_the_registers(report, lanes, out, whole, threads):
    found = _named(report, f"11scan_kernelI13__nv_bfloat16Li{lanes}ELb{out}ELb{whole}E")
    assert len(found) == 1
    for name, r in found.items():
        assert (r["regs"] + 7) // 8 * 8 * threads * 2 <= REGISTERS, (name, r["regs"])
