"""bench.py's printed line, on the CPU: short enough for a reader that keeps only the end
of the output, with every key such a reader looks for."""

from __future__ import annotations

import json
import math
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)

import bench  # noqa: E402
from lora_adapter_execution_b200 import workloads as wl  # noqa: E402


def entry(name):
    """A workload's record with the lengths that a run's records have."""
    x = 1234567.8901234567
    inp = wl.make_inputs("tiny")
    return {"metric": "tokens/s per fused multi-LoRA linear at 1 B200; % of bf16 TC peak / HBM roofline", "value": x * 10,
            "unit": "tokens/s", "n_gpus": 1, "steps": 20, "warmup": 5, "ms_per_step": x / 1e6, "higher_is_better": True,
            "scaling": "weak", "vs_baseline": None, "dtype": "bf16", "data": "synthetic",
            "config": {**bench.config_record("tiny", inp, 8), "workload": max(bench.WORKLOAD_TEXT.values(), key=len),
                       "l2": "inputs rotate over 2 copies (1344 MiB > 126 MiB L2)"},
            "timing": "t" * 120, "gpu_launches": 180,
            "roofline": {"bound": "tensor", "achieved": x / 1e3, "peak": 1669.2, "unit": "TFLOP/s", "frac": 0.78079694,
                         "peak_kind": "k" * 40, "traffic": 420225536, "kernel": "k" * 60, "timed": "k" * 40},
            "layer_roofline": {"bound": "tensor", "frac": 0.6776020282516099, "what": "w" * 100},
            "clocks": {"sm_mhz": 1552.0, "sm_max_mhz": 1965.0, "reasons": ["sw_power_cap"], "samples": 149},
            "layer": {str(i): x for i in range(12)},
            "e2e": {"value": x, "unit": "tokens/s", "h2d_bytes_per_step": 268500992, "d2h_bytes_per_step": 268435456,
                    "steps": 20, "what": "w" * 300},
            "cpu_baseline": {"value": 559.7820445441624, "unit": "tokens/s", "cores": 16, "kind": "oracle",
                             "sample": "s" * 80}}


NAMES = [*wl.WORKLOADS, "switch", "factor_qr", "compress"]


def test_the_line_is_short_and_complete():
    entries = {n: entry(n) for n in NAMES}
    del entries["compress"]["e2e"]
    line = bench.result_line(bench.HEADLINE, entries)
    assert len(line) < bench.LINE_MAX == 2000 and "\n" not in line
    d = json.loads(line)
    for k in ("metric", "value", "unit", "n_gpus", "steps", "warmup", "ms_per_step", "higher_is_better", "scaling",
              "vs_baseline", "dtype", "data", "config", "clocks", "e2e", "gpu_launches"):
        assert k in d, k
    full = entries[bench.HEADLINE]
    assert d["config"] == full["config"] and d["higher_is_better"] is True and d["vs_baseline"] is None
    assert set(d["e2e"]) == {"value", "unit", "h2d_bytes_per_step", "d2h_bytes_per_step"}
    assert d["e2e"]["h2d_bytes_per_step"] == 268500992 and d["clocks"]["reasons"] == ["sw_power_cap"]
    # six significant digits: half a unit of the sixth at most
    for got, want in ((d["value"], full["value"]), (d["ms_per_step"], full["ms_per_step"]),
                      (d["e2e"]["value"], full["e2e"]["value"])):
        assert math.isclose(got, want, rel_tol=5e-6)
    cols = d["configs"].pop("columns")
    assert set(d["configs"]) == set(NAMES)
    row = dict(zip(cols, d["configs"]["decode"]))
    assert math.isclose(row["value"], entries["decode"]["value"], rel_tol=5e-4)
    assert d["configs"]["compress"][cols.index("e2e")] is None


def test_one_workload_alone_has_no_table():
    d = json.loads(bench.result_line("decode", {"decode": entry("decode")}))
    assert "configs" not in d and "headline" not in d and d["unit"] == "tokens/s"
