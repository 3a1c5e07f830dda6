"""What fsa_get_device_error makes of an error word that several kernels left
their codes in: evaluated by the compiler, no GPU."""
import os
import shutil
import subprocess

import pytest

from matrix_core_softmax_gb300 import build as fsa_build

CASES = """
static_assert(error_word_status(0) == FSA_OK);
static_assert(error_word_status(kErrTimeout) == FSA_ERR_TIMEOUT);
static_assert(error_word_status(kErrMisaligned) == FSA_ERR_CUDA);
static_assert(error_word_status(kErrBadIndex) == FSA_ERR_INVALID_ARGUMENT);
static_assert(error_word_status(kErrTimeout | kErrMisaligned | kErrBadIndex) == FSA_ERR_TIMEOUT);
static_assert(error_word_status(kErrTimeout | kErrBadIndex) == FSA_ERR_TIMEOUT);
static_assert(error_word_status(kErrMisaligned | kErrBadIndex) == FSA_ERR_CUDA);
static_assert(error_word_status(1u << 20 | kErrBadIndex) == FSA_ERR_CUDA);
"""


def test_order_of_the_codes(tmp_path):
    if not shutil.which("g++"):
        pytest.skip("no host compiler")
    src = tmp_path / "codes.cpp"
    src.write_text('#include "fsa_internal.h"\nnamespace fsa {' + CASES + "}\n")
    cuda = os.path.join(os.path.dirname(os.path.dirname(shutil.which(fsa_build._nvcc()) or "/usr/local/cuda/bin/nvcc")), "include")
    r = subprocess.run(["g++", "-std=c++17", "-fsyntax-only", "-I", fsa_build.CSRC, "-I", os.path.join(fsa_build.ROOT, "include"),
                        "-I", cuda, str(src)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
