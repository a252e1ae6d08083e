"""Rows that a launch may also write (an output over an input, rows read back after they were stored) are not read through the
read-only path, of which the compiler and the caches may take it that nothing writes there."""
import os
import re

from ragged_grouped_gemm_device_gb300 import _lib

CSRC = os.path.join(os.path.dirname(os.path.abspath(_lib.__file__)), "csrc")


def _code(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//.*", "", f.read())


def test_elements_of_rows():
    chunks = re.findall(r"struct Chunk<(\w+, \d)> \{(.*?)\n\};", _code("rows.cuh"), flags=re.S)
    assert {"float, 1", "bf16, 1"} <= {n for n, _ in chunks}
    assert all("__ldg" not in body and ".nc" not in body for _, body in chunks)


def test_the_join_reads_only_statistics_so():
    for line in _code("residual_norm.cu").splitlines():
        assert "__ldg" not in line or "stats" in line or "__ldg(p + static_cast<size_t>(q) * a.T)" in line, line
