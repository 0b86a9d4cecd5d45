"""The linear layer's choice of operands and the addresses that its kernels read,
on the CPU: the header that the library is built from, run over small sizes and
layouts (tests/xcheck/product_operands.cpp)."""

import os
import shutil
import subprocess

import pytest

from momentum_compression_amd import build as B

SRC = os.path.join(B.ROOT, "tests", "xcheck", "product_operands.cpp")


def run(tmp_path, include):
    exe = str(tmp_path / "operands")
    res = subprocess.run(["g++", "-O2", "-std=c++17", "-Wall", "-Wextra", "-Werror",
                          f"-I{include}", SRC, "-o", exe], capture_output=True, text=True)
    assert res.returncode == 0, res.stderr
    return subprocess.run([exe], capture_output=True, text=True, timeout=300)


@pytest.mark.skipif(shutil.which("g++") is None, reason="no g++")
def test_no_read_leaves_the_operands_rows(tmp_path):
    res = run(tmp_path, B.CSRC)
    assert res.returncode == 0, res.stdout


@pytest.mark.skipif(shutil.which("g++") is None, reason="no g++")
def test_the_check_sees_reads_in_front(tmp_path):
    """With rows laid out anew taken for as long as the matrix's own, reads start in
    front of them, and the check says so."""
    text = open(os.path.join(B.CSRC, "operands.h")).read()
    short = text.replace("ProductIn{room, padded(cols), padded(cols)",
                         "ProductIn{room, padded(cols), cols")
    assert short != text
    (tmp_path / "operands.h").write_text(short)
    res = run(tmp_path, str(tmp_path))
    assert res.returncode == 1 and "row 0 elements -" in res.stdout, res.stdout
