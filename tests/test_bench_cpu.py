"""The oracle arm of bench.py runs on the host cores alone and prints the
benchmark's JSON line (the metric, its unit, the oracle baseline and the
zero-copy end-to-end fields) without touching a GPU."""

import json
import os
import re
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_reference_arm_json_line():
    env = dict(os.environ, CUDA_VISIBLE_DEVICES="")
    out = subprocess.run([sys.executable, os.path.join(ROOT, "bench.py"), "--impl", "reference", "--steps", "1",
                          "--warmup", "1"], capture_output=True, text=True, timeout=600, env=env, cwd=ROOT)
    assert out.returncode == 0, out.stderr[-2000:]
    lines = [l for l in out.stdout.splitlines() if l.startswith("{")]
    assert len(lines) == 1
    d = json.loads(lines[0])
    assert d["impl"] == "reference"
    for key in ("metric", "value", "unit", "n_gpus", "steps", "warmup", "ms_per_step", "higher_is_better",
                "scaling", "vs_baseline", "dtype", "data", "config", "cpu_baseline", "e2e"):
        assert key in d, key
    assert d["value"] > 0 and d["unit"] == "TFLOP/s" and d["n_gpus"] == 1
    assert d["cpu_baseline"]["kind"] == "oracle" and d["cpu_baseline"]["value"] == d["value"]
    assert d["e2e"]["h2d_bytes_per_step"] == 0 and d["e2e"]["d2h_bytes_per_step"] == 0
    assert d["config"]["workload"].startswith("llama65b-decoder-layer")


def test_traffic_record_covers_every_source_of_the_gemms():
    """The DRAM record of the dequant GEMMs is dropped when their sources
    change: the hash covers the two kernels and all that they include."""
    sys.path.insert(0, ROOT)
    import bench
    csrc = os.path.join(ROOT, "bit_nf4_quantized_11_b200", "csrc")
    todo, seen = ["gemm_pair_sm100.cuh", "gemm_sm100.cuh"], set()
    while todo:
        name = todo.pop()
        if name not in seen:
            seen.add(name)
            with open(os.path.join(csrc, name)) as f:
                todo += re.findall(r'#include "([^"]+)"', f.read())
    assert seen == set(bench.GEMM_SOURCES)
