"""The counter summary of the gated scan and the norm with the residual describes the
kernels as they are: it carries a hash of each source's code, which a change of the code
(not of a comment) has to renew by another profiled run."""
import os
import re

import bench

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SOURCES = ["kda_scan.h", "kda_scan.hip", "kda_scan_decode.hip", "kda_add_norm.hip"]


def test_the_summary_describes_the_current_code():
    text = open(os.path.join(ROOT, "profiles", "scan_and_residual_norm.md"), encoding="utf-8").read()
    held = dict(re.findall(r"^- `(\S+)` ([0-9a-f]{16})$", text, flags=re.M))
    assert held == {name: bench._source_sha(name) for name in SOURCES}
