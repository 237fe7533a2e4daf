"""The gated pair's matrix kernels (bf16, FP8) keep nothing in scratch memory
and spill no vector register (no GPU needed): they are the kernels nearest to
the register limit, and an array that the compiler cannot hold in registers is
no spill in its report."""
import os
import re
import shutil
from concurrent.futures import ThreadPoolExecutor

import pytest

from test_kernel_resources import HIPCC, _report


def gated(text):
    """Kernel name -> its report lines' values, of the gated instantiations and their reduction."""
    out, name = {}, None
    for line in text.splitlines():
        m = re.search(r"remark: Function Name: (\S+)", line)
        if m:
            name = m.group(1)
        m = re.search(r"remark:\s+(ScratchSize \[bytes/lane\]|VGPRs Spill): (\d+)", line)
        # the last template argument of the GEMMs is whether they are gated
        if m and name and re.search(r"k_gemm_\w+?I\w*Lb1EEEv|k_gated_reduceI", name):
            out.setdefault(name, {})[m.group(1)] = int(m.group(2))
    return out


@pytest.mark.skipif(not (shutil.which(HIPCC) or os.path.exists(HIPCC)), reason="no hipcc")
def test_no_scratch(tmp_path):
    sources = ["gemm.hip", "gemm_fp8.hip"]
    with ThreadPoolExecutor(2) as ex:
        reports = list(ex.map(lambda s: _report(s, str(tmp_path)), sources))
    for src, text in zip(sources, reports):
        found = gated(text)
        kind = "k_gemm_bf16" if src == "gemm.hip" else "k_gemm_fp8"
        # 256 x 256, 256 x 128, 128 x 128, 64 x 128 and 32 x 128 tiles, whole and in pieces
        tiles = {re.search(r"ILb[01]ELi(\d+)ELi(\d+)", n).groups() for n in found if kind in n}
        assert tiles == {("256", "256"), ("256", "128"), ("128", "128"), ("64", "128"), ("32", "128")}, tiles
        assert len([n for n in found if kind in n]) == 10, sorted(found)
        for name, info in found.items():
            assert info == {"ScratchSize [bytes/lane]": 0, "VGPRs Spill": 0}, (src, name, info)
