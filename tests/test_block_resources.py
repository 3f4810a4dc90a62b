"""Register and spill budgets of the block operators' kernels, from ptxas's
report on the CPU: an edit that makes one spill fails here before it reaches a
GPU."""
import concurrent.futures as cf
import os

import pytest

from linear_rnn_mlstm_b200 import build as libbuild
from test_kernel_resources import _named, _ptxas_report

SOURCES = ("rmsnorm.cu", "conv.cu", "scan.cu", "scan_bwd.cu", "sum_rows.cu")
NO_SPILLS = ("rmsnorm_kernel", "rmsnorm_bwd_kernel", "conv_fwd_kernel", "conv_step_kernel", "conv_bwd_kernel", "sum_rows_kernel",
             "scan_step_kernel", "scan_fold_kernel", "scan_bwd_summary_kernel", "scan_bwd_fold_kernel", "scan_bwd_finish_kernel")
# bytes a thread may spill: the scan's helper and scan warps share one allocation; the
# gradient pass with two pairs a lane
SOME_SPILLS = {"11scan_kernel": 32, "scan_bwd_grad_kernel": 8}
# launch width and CTAs per SM that the plans count on
RESIDENT = {"scan_bwd_grad_kernel": (256, 2), "conv_bwd_kernel": (256, 2)}


@pytest.fixture(scope="module")
def report():
    srcs = [os.path.join(libbuild.CSRC, s) for s in SOURCES]
    out = {}
    with cf.ThreadPoolExecutor(max_workers=os.cpu_count() or 4) as ex:
        for part in ex.map(_ptxas_report, srcs):
            out.update(part)
    return out


def test_spills(report):
    for short in NO_SPILLS:
        found = _named(report, short)
        assert found, short
        for name, r in found.items():
            assert r["spill"] == 0, f"{short}: {r['spill']} bytes ({name})"
    for short, most in SOME_SPILLS.items():
        found = _named(report, short)
        assert found, short
        for name, r in found.items():
            # spill stores and loads are counted together
            assert r["spill"] <= 2 * most, f"{short}: {r['spill']} bytes ({name})"


def test_registers_leave_room_for_the_planned_ctas(report):
    for short, (threads, ctas) in RESIDENT.items():
        for name, r in _named(report, short).items():
            assert r["regs"] * threads * ctas <= 65536, f"{short}: {r['regs']} registers ({name})"
