"""The kernels of the layer norm, of the linear layer with its epilogue and of the
orthogonalised updates keep nothing in scratch memory (no GPU needed)."""
import os
import re
import shutil
from concurrent.futures import ThreadPoolExecutor

import pytest

from test_kernel_resources import HIPCC, _report

# of the base GEMMs' files, the layer's whole tiles and its reductions
PARTS = {"layernorm.hip": ".", "ortho.hip": ".", "linear_act.hip": ".",
         "gemm.hip": r"k_gemm_bf16\w+Lb1ELb0EEE|k_splitk_reduce\w+Lb1EEE",
         "gemm_fp8.hip": r"k_gemm_fp8\w+Lb1ELb0EEE|k_splitk_reduce\w+Lb1EEE"}


@pytest.mark.skipif(not (shutil.which(HIPCC) or os.path.exists(HIPCC)), reason="no hipcc")
def test_no_scratch(tmp_path):
    with ThreadPoolExecutor(5) as ex:
        reports = list(ex.map(lambda s: _report(s, str(tmp_path)), PARTS))
    for (src, wanted), text in zip(PARTS.items(), reports):
        name, seen = "", 0
        for line in text.splitlines():
            m = re.search(r"remark: Function Name: (\S+)", line)
            name = m.group(1) if m else name
            m = re.search(r"remark:\s+ScratchSize \[bytes/lane\]: (\d+)", line)
            if m and re.search(wanted, name):
                seen += 1
                assert m.group(1) == "0", (src, name, m.group(1))
        assert seen >= 4, (src, seen)
