"""The loads of the 8-bit products' large tiles stay inside an operand whose last tile is short: the address
arithmetic that the kernel uses (csrc/fp8_panel.h), compiled for the CPU and walked through for every number
of rows, under every reading of the hardware's range check; and that the kernel takes its addresses from there."""
import os
import re
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "muon_newton_schulz_momentum_amd", "csrc")


def test_panel_loads_stay_inside(tmp_path):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("g++ not available")
    exe = tmp_path / "panel_bounds"
    build = subprocess.run([gxx, "-std=c++17", "-O2", "-Wall", "-I", CSRC, os.path.join(ROOT, "tests", "native", "panel_bounds.cpp"),
                            "-o", str(exe)], capture_output=True, text=True)
    assert build.returncode == 0, build.stderr[-2000:]
    run = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300)
    assert run.returncode == 0 and "panels ok" in run.stdout, run.stdout[-2000:]


def test_product_kernel_uses_these_addresses():
    text = open(os.path.join(CSRC, "fp8_product.hip")).read()
    loads = re.findall(r"raw_buffer_load_b128\(([^;]*)\);", text)
    assert len(loads) == 1
    _, vector, scalar, _ = [a.strip() for a in loads[0].split(",")]
    assert f"int32_t {vector} = (d < LA ? va : vb) + rows_on;" in text
    assert "int32_t rows_on = Panel::rows(64 * i, (int)(d < LA ? p.lda : p.ldb));" in text
    assert "va = Panel::lane(lrow, lchunk, (int)p.lda), vb = Panel::lane(lrow, lchunk, (int)p.ldb);" in text
    assert f"int32_t {scalar} = Panel::block(step) & keep;" in text
    for operand in "ab":
        assert f"bytes_{operand} = Panel::bytes(x.rows_{operand}, (int)p.ld{operand}, kp);" in text
