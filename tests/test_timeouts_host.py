"""Kernels that load through TMA and whose waits give up do not return while a copy may still be on its way into their
shared memory: what they report the timeout by waits for that."""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "eagle_tree_speculative_gb300", "csrc")
FILES = {os.path.basename(f): re.sub(r"//[^\n]*", "", open(f).read()) for f in glob.glob(os.path.join(CSRC, "*.cu*"))}


def test_a_timeout_is_reported_behind_copies_on_their_way():
    plain = {name for name, text in FILES.items() if re.search(r"flag_error\([^;]*EAGLE_DEV_TIMEOUT", text)}
    assert plain == {"tc_common.cuh"}                          # in report_timeout alone
    body = re.search(r"void report_timeout\(.*?\n}", FILES["tc_common.cuh"], re.S).group()
    assert body.index("while (clock64() - t0 < kLandCycles)") < body.index("flag_error")


def test_every_kernel_that_gives_up_reports_it_when_all_its_threads_are_done():
    aborting = {name for name, text in FILES.items() if re.search(r"\babort_flag = &?", text) and "__global__" in text}
    assert len(aborting) >= 6
    for name in aborting:
        assert re.search(r"__syncthreads\(\);\s*if \(\w+(?:\.x)? == 0 && \*abort_flag\) report_timeout\(", FILES[name]), name
