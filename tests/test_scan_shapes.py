"""The scan's loop over a tile takes its rows in batches: a shape whose tile the batches do not fill, or
that has one batch alone, does not compile."""
import os
import subprocess

import pytest

from pointwise_conv_cnn_gb300 import build

CSRC = build.CSRC


@pytest.mark.parametrize("spt,lpc,rows,message", [
    (4, 4, None, None),
    (8, 16, None, None),
    (2, 8, None, "whole 16-byte loads"),
    (4, 4, 4, "two batches are loaded"),
    (4, 4, 10, "batches fill the tile")])
def test_shapes(tmp_path, spt, lpc, rows, message):
    """rows: a tile's, in place of the rule for them."""
    text = open(os.path.join(CSRC, "seq_scan.cuh")).read()
    rule = "TT = scan_rows(CH, NP);"
    assert text.count(rule) == 1
    if rows:
        text = text.replace(rule, f"TT = {rows};")
    (tmp_path / "scan.cuh").write_text(text)
    (tmp_path / "one.cu").write_text(
        '#include <atomic>\n#include "scan.cuh"\nnamespace fcm { namespace seq {\n'
        f"template __global__ void scan_kernel<float, {spt}, {lpc}, 0, false>(const ScanArgs);\n}} }}\n")
    r = subprocess.run([build.nvcc(), *build.ARCH, "-std=c++17", "--expt-relaxed-constexpr", "-I", CSRC, "-I", build.INCLUDE,
                        "-c", "-o", str(tmp_path / "one.o"), str(tmp_path / "one.cu")], capture_output=True, text=True)
    if message:
        assert r.returncode != 0 and message in r.stderr, r.stderr
    else:
        assert r.returncode == 0, r.stderr
