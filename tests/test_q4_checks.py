"""Every kernel of the 4-bit cache checks the indices it derives in the debug-bounds build, as jetlong.h says."""
import os
import re

import pytest

from rope_context_extension_sm_b200 import build

KERNELS = {"jl_q4.cuh": ["jl_kv_fill_q4_kernel", "jl_decode_append_q4_kernel", "jl_kv_read_q4_kernel"],
           "jl_decode_q4.cuh": ["jl_decode_q4_kernel", "jl_decode_q4_combine_kernel"]}


@pytest.mark.parametrize("file,kernel", [(f, k) for f, names in KERNELS.items() for k in names])
def test_kernel_checks_its_indices(file, kernel):
    text = open(os.path.join(build.CSRC, file)).read()
    kernels = re.split(r"\n__global__ ", text)[1:]
    body = [x for x in kernels if re.search(r"\b%s\(" % kernel, x.split("{")[0])]
    assert len(body) == 1
    assert "JL_CHECK(" in body[0].split("\n}\n")[0]


def test_the_decode_checks_rows_pages_tables_and_slots():
    text = open(os.path.join(build.CSRC, "jl_decode_q4.cuh")).read()
    checks = " ".join(re.findall(r"JL_CHECK\((.*?)\);", text, re.S))
    for name in ("cache_stride", "num_pages", "n_tab_rows", "slot0", "c0 + count <= p.n_cta"):
        assert name in checks
