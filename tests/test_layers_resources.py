"""What the compiler makes of the expert layers' kernels for gfx950: nothing spilled to memory, the occupancy that their text
relies on, and main loops of the big tiles that wait for the oldest of the loads in flight only.
"""
import os
import re

import pytest

from test_experts_resources import HIPCC, _compile

pytestmark = pytest.mark.skipif(not os.path.exists(HIPCC), reason="hipcc not installed")


def test_big_tiles_keep_their_loads_in_flight(tmp_path):
    res, text = _compile("layer_product.hip", tmp_path)
    big = {k: r for k, r in res.items() if "12layer_kernel" in k}
    few = {k: r for k, r in res.items() if "16layer_few_kernel" in k}
    assert len(big) == 7 * 3 and len(few) == 4 * 3, sorted(res)
    for k, r in big.items():
        assert r["ScratchSize"] == 0 and r["VGPRs"] + r.get("AGPRs", 0) <= 256 and r["LDS Size"] <= 160 * 1024 and r["Occupancy"] == 2, (k, r)
    for k, r in few.items():
        assert r["ScratchSize"] == 0 and r["Occupancy"] >= 2 and 2 * r["LDS Size"] <= 160 * 1024, (k, r)
    for k in big:
        body = re.search(r"\n%s:(.*?)\.Lfunc_end" % re.escape(k), text, re.S).group(1)
        loads = 4 + int(re.search(r"Li(\d+)EEEv", k).group(1)) // 64
        loops = 0
        for block in re.split(r"\n(?=\.LBB\S+:)", body):
            if "v_mfma" not in block:
                continue
            step = block.split("s_barrier")[0] if "s_barrier" in block else ""
            waits = [int(v) for v in re.findall(r"vmcnt\((\d+)\)", step)]
            if step.count("buffer_load_dwordx4") == loads:
                loops += 1
                assert waits and min(waits) == loads - 1, (k, waits)
        assert loops >= 1, k


def test_row_kernels_do_not_spill(tmp_path):
    res, _ = _compile("layer_rows.hip", tmp_path)
    assert len(res) >= 10, sorted(res)
    for k, r in res.items():
        assert r["ScratchSize"] == 0, (k, r)
