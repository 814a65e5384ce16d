"""What the compiler makes of the routed-expert kernels for gfx950: occupancy that their text relies on, and no register
spilled to memory inside a main loop of the large products (a scratch access there would wait for the loads in flight).
"""
import os
import re
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "..", "muon_newton_schulz_momentum_amd", "csrc")
INCLUDE = os.path.join(HERE, "..", "include")
HIPCC = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"

pytestmark = pytest.mark.skipif(not os.path.exists(HIPCC), reason="hipcc not installed")


def _compile(src, tmp_path):
    """(resources by function, assembly text)"""
    out = str(tmp_path / "out.s")
    cmd = [HIPCC, "--offload-arch=gfx950", "-O3", "-std=c++17", "-I", INCLUDE, "-I", CSRC, "-Xclang", "-target-feature", "-Xclang",
           "-packed-fp32-ops", "--cuda-device-only", "-S", os.path.join(CSRC, src), "-o", out,
           "-Rpass-analysis=kernel-resource-usage"]
    run = subprocess.run(cmd, capture_output=True, text=True, timeout=600)
    assert run.returncode == 0, run.stderr[-2000:]
    res, name = {}, None
    for line in run.stderr.splitlines():
        m = re.search(r"Function Name: (\S+)", line)
        if m:
            name = m.group(1)
            res[name] = {}
            continue
        m = re.search(r"remark:\s+(VGPRs|AGPRs|LDS Size|ScratchSize|Occupancy) ?(?:\[[^\]]*\])?: (\d+)", line)
        if m and name:
            res[name][m.group(1)] = int(m.group(2))
    return res, open(out).read()


def test_large_products_spill_outside_their_loops_only(tmp_path):
    res, text = _compile("fp8_product.hip", tmp_path)
    large = {k: r for k, r in res.items() if "14product_kernel" in k}
    few = {k: r for k, r in res.items() if "18product_few_kernel" in k}
    assert len(large) == 6 and len(few) == 12, sorted(res)
    for k, r in large.items():
        assert r["VGPRs"] + r.get("AGPRs", 0) <= 256 and r["LDS Size"] <= 160 * 1024 and r["Occupancy"] == 2, (k, r)
    for k, r in few.items():
        # a workgroup is 2 waves a SIMD; of the 32 x 16 tiles' there are two on a compute unit
        assert r["ScratchSize"] == 0 and r["Occupancy"] >= (4 if "Li1ELi4E" in k else 2) and 2 * r["LDS Size"] <= 160 * 1024, (k, r)
    seen = 0
    for k in large:
        body = re.search(r"\n%s:(.*?)\.Lfunc_end" % re.escape(k), text, re.S).group(1)
        for block in re.split(r"\n(?=\.LBB\S+:)", body):
            if "v_mfma" in block:
                seen += 1
                assert "scratch_" not in block, (k, block.splitlines()[0])
    assert seen >= 6 * 4                                       # four numbers of row blocks each


def test_routing_kernels_keep_their_waves(tmp_path):
    res, _ = _compile("route.hip", tmp_path)
    for k, r in res.items():
        assert r["ScratchSize"] == 0, (k, r)
    narrow = {k: r for k, r in res.items() if "12route_kernel" in k and "Li16E" in k}
    assert len(narrow) == 8, sorted(res)
    for k, r in narrow.items():
        assert r["Occupancy"] >= 4, (k, r)


def test_quantisation_keeps_its_waves(tmp_path):
    res, _ = _compile("fp8_quantize.hip", tmp_path)
    assert len(res) == 8, sorted(res)
    for k, r in res.items():
        assert r["ScratchSize"] == 0 and r["Occupancy"] >= 3, (k, r)
