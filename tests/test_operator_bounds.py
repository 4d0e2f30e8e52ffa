"""What the bounds-checked build of the training and adapter operators checks:
the width of every access, and every array that an index is computed for.  The
comparisons are compiled for the host and the kernels' source is read; on a GPU
the operators' other suites run under that build too."""
import os
import re
import shutil
import subprocess

import pytest

import test_checked_operators as checked

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "partial_sum_reduction_gb300", "csrc")


def test_a_piece_is_inside_as_a_whole(tmp_path):
    if not shutil.which("g++"):
        pytest.skip("g++ not available")
    exe = str(tmp_path / "checked_pieces")
    r = subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Wextra", "-Werror", "-I", CSRC, "-I",
                        os.path.join(ROOT, "include"), os.path.join(ROOT, "tests", "c", "checked_pieces.cpp"), "-o", exe],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0 and r.stdout == "ok\n", r.stdout


def test_pieces_of_eight_are_checked_as_such():
    """The four places that take eight values at a time say so."""
    src = open(os.path.join(CSRC, "adapters.cu")).read()
    for name, end in (("auto x_piece = ", "};"), ("auto w_piece = ", "};"), ("auto has = ", "};"), ("auto load_w = ", "};\n    int slot")):
        body = src[src.index(name):]
        body = body[:body.index(end)]
        assert "piece_in_bounds<VEC>(" in body and not re.search(r"(?<!piece_)in_bounds\(", body), name


@pytest.mark.parametrize("name,array", [("adapters.cu", r"k\.s\[at"), ("adapters.cu", r"\bw\[at\]"), ("adapters.cu", r"J\.s\[at\]"),
                                        ("adapters.cu", r"(?<!_)as_float\(w\["), ("adapters.cu", r"k\.out\[t0 \* k\.R"),
                                        ("adapters.cu", r"__stcg\("), ("layernorm_train.cu", r"\? part\[at\]")])
def test_indexed_arrays_are_checked(name, array):
    """Each access has its check within the three lines up to it."""
    lines = open(os.path.join(CSRC, name)).read().split("\n")
    hits = [i for i, text in enumerate(lines) if re.search(array, text)]
    assert hits
    for i in hits:
        assert "in_bounds(" in "\n".join(lines[max(0, i - 3):i + 1]), "%s:%d" % (name, i + 1)


@pytest.mark.gpu
@pytest.mark.parametrize("suite", ["test_adapters_exactness.py", "test_operator_ordering.py",
                                   "test_layernorm_training_extremes.py"])
def test_other_suites_pass_under_bounds_checks(suite):
    checked.test_suite_passes_under_bounds_checks(suite)
