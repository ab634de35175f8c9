"""The counter summary of the linear attention and the per-head norms describes the
kernels as they are: it carries a hash of each source's code, which a change of the code
(not of a comment) has to renew by another profiled run."""
import os
import re

import bench

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SOURCES = ["kda_linattn.h", "kda_linattn.hip", "kda_linattn_f32.hip", "kda_linattn_decode.hip", "kda_norm.hip"]


def test_the_summary_describes_the_current_code():
    text = open(os.path.join(ROOT, "profiles", "linattn_and_norms.md"), encoding="utf-8").read()
    held = dict(re.findall(r"^- `(\S+)` ([0-9a-f]{16})$", text, flags=re.M))
    assert held == {name: bench._source_sha(name) for name in SOURCES}
