"""CPU-only checks of the 8-bit products' test hooks (include/int8_gemm.h)."""
import os
import re

import pytest

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include",
                      "int8_gemm.h")


@pytest.fixture(scope="module")
def lib():
    from dense_fp32_matrix_03_gb300 import build
    build.build()
    import dense_fp32_matrix_03_gb300 as m
    m.load()
    yield m
    assert m.sgemm_i8_tune_force("auto") == m.SGEMM_OK


def test_force_validates_its_argument(lib):
    for bad in (-1, 6, 2 ** 31 - 1):
        assert lib.sgemm_i8_tune_force(bad) == lib.SGEMM_ERR_INVALID_ARG
    with pytest.raises(KeyError):
        lib.sgemm_i8_tune_force("fastest")
    for name in lib.I8_KERNELS:
        assert lib.sgemm_i8_tune_force(name) == lib.SGEMM_OK


def test_names_match_the_header(lib):
    text = open(HEADER).read()
    found = {m.group(1).lower(): int(m.group(2))
             for m in re.finditer(r"#define SGEMM_I8_KERNEL_(\w+) (\d+)", text)}
    assert found == lib.I8_KERNELS


def test_refused_products_leave_no_record(lib):
    before = lib.sgemm_i8_last_kernel(), lib.sgemm_i8_last_split_count()
    assert lib.sgemm_i8("bf16", 4, 4, 8, 0, 8, 0, 0, 8, 0, 0, 4) == lib.SGEMM_ERR_INVALID_ARG
    assert (lib.sgemm_i8_last_kernel(), lib.sgemm_i8_last_split_count()) == before
