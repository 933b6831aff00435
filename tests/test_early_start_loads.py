"""Kernels that start while the kernel before them still runs (they call
griddepcontrol.wait) read memory with ordinary loads only.  A read-only load
(__ldg, ld.global.nc, or what the compiler makes of a const pointer that is
declared __restrict__) is defined for memory that nothing writes as long as the
kernel lives, and such a kernel lives while its operands are being written."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "dense_fp32_matrix_03_gb300", "csrc")
READ_ONLY = re.compile(r"__ldg\s*\(|ld\.global(\.\w+)*\.nc\b|__restrict__")


def code(path):
    text = re.sub(r"/\*.*?\*/", "", open(path).read(), flags=re.S)
    return re.sub(r"//[^\n]*", "", text)


def early_starters():
    files = sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cuh")))
    return [f for f in files if re.search(r"dependent_wait\(\);|griddepcontrol\.wait", code(f))]


def test_the_early_starters_are_found():
    names = {os.path.basename(f) for f in early_starters()}
    assert {"experts.cu", "quant.cu", "i8_gemm.cu", "i8_few.cuh", "i8_tc.cuh", "tc_ss.cuh",
            "api.cu"} <= names


@pytest.mark.parametrize("path", early_starters(), ids=os.path.basename)
def test_no_read_only_loads(path):
    found = [m.group(0) for m in READ_ONLY.finditer(code(path))]
    assert not found, found


def test_kernels_with_read_only_loads_start_late():
    """The files that do use such loads launch nothing as a programmatic
    dependent."""
    for path in glob.glob(os.path.join(CSRC, "*.cu*")):
        text = code(path)
        if READ_ONLY.search(text):
            assert "ProgrammaticStreamSerialization" not in text, path
            assert "launch_dependent(" not in text, path
