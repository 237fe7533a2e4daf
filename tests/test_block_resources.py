"""The feed-forward block's kernels keep nothing in scratch memory: an array
that the compiler cannot hold in registers costs a trip to memory per access
and is no spill in its report (no GPU needed)."""
import os
import re
import shutil
from concurrent.futures import ThreadPoolExecutor

import pytest

from test_kernel_resources import HIPCC, _report


@pytest.mark.skipif(not (shutil.which(HIPCC) or os.path.exists(HIPCC)), reason="no hipcc")
def test_no_scratch(tmp_path):
    sources = ["norm.hip", "gated.hip", "gated_bwd.hip", "segments.hip"]
    with ThreadPoolExecutor(4) as ex:
        reports = list(ex.map(lambda s: _report(s, str(tmp_path)), sources))
    seen = 0
    for src, text in zip(sources, reports):
        name = None
        for line in text.splitlines():
            m = re.search(r"remark: Function Name: (\S+)", line)
            name = m.group(1) if m else name
            m = re.search(r"remark:\s+ScratchSize \[bytes/lane\]: (\d+)", line)
            if m:
                seen += 1
                assert m.group(1) == "0", (src, name, m.group(1))
    assert seen >= 40
