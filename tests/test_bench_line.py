"""The benchmark's printed line: one JSON object, short enough for a reader that
keeps the last 3000 bytes of the output, with the headline's keys."""
import json

import pytest

import bench

LONG = 123.45678901234567


def full_result():
    part = {"us": LONG, "kernel": "k" * 40, "bytes": LONG * 1e9, "GB/s": LONG, "bound": "tensor_bf16", "frac_hbm": LONG,
            "t_roof_us": LONG, "frac_roof": LONG}
    config = dict(workload="gemma_gate_4096x2048x16384", step_us=LONG, tflops=LONG, t_roof_us=LONG, roof_frac=LONG,
                  kernels={p: part for p in bench.PART_KERNELS})
    return {"metric": bench.METRIC, "value": LONG * 10, "unit": bench.UNIT, "n_gpus": 8, "steps": 20, "warmup": 5,
            "ms_per_step": LONG, "higher_is_better": True, "scaling": "weak", "vs_baseline": None, "dtype": "bf16",
            "data": "synthetic (seeded; random-init weights of the 4096x4096 layer)", "config": bench.head_config(8),
            "e2e": {"value": LONG, "unit": bench.UNIT, "h2d_bytes_per_step": 268435456, "d2h_bytes_per_step": 147456},
            "gpu_launches": 120,
            "roofline": {"bound": "tensor", "achieved": LONG * 10, "peak": 1639.8, "unit": "TFLOP/s", "frac": LONG / 1e3,
                         "traffic": 259798272, "kernel": "k3_dx_pair_kernel (gemm_dx, 16384x4096x4096 bf16)",
                         "peak_source": "measured bf16 dense burst x 2 (nominal int8:bf16 ratio)", "avg_launch_us": LONG,
                         "algorithmic_per_launch": 549755813888.0, "launches_timed": 20},
            "step_roofline": {"t_roof_us": LONG, "t_measured_us": LONG, "frac": LONG, "rule": "r" * 120},
            "kernels": {p: part for p in bench.PART_KERNELS},
            "cpu_baseline": {"value": LONG, "unit": "TFLOP/s", "cores": 128, "cpu": "c" * 60, "kind": "oracle",
                             "sample": "s" * 160},
            "clocks": {"sm_mhz": 1965.0, "sm_max_mhz": 1965.0, "samples": 100,
                       "reasons": ["hw_slowdown", "hw_thermal_slowdown", "sw_power_cap", "sw_thermal_slowdown"]},
            "peaks": {"hbm_gbs": 6529.1, "bf16_tflops": 1639.8, "bf16_tflops_sustained": 1392.5, "source": "measured"},
            "merge": part, "configs": [config] * 31}


def test_the_line_is_short_and_whole():
    text = bench.headline(full_result())
    assert len(text) <= bench.LINE_BYTES and "\n" not in text
    line = json.loads(text)
    for key in ("metric", "value", "unit", "n_gpus", "steps", "warmup", "ms_per_step", "higher_is_better", "scaling",
                "vs_baseline", "dtype", "data", "config", "e2e", "gpu_launches", "clocks", "roofline"):
        assert key in line, key
    assert line["value"] == pytest.approx(1234.57) and line["roofline"]["traffic"] == 259798272
    assert line["e2e"]["h2d_bytes_per_step"] == 268435456 and set(line["kernels_us"]) == set(bench.PART_KERNELS)


def test_a_line_too_long_drops_what_is_not_the_headline():
    full = full_result()
    full["cpu_baseline"]["sample"] = "s" * 2000
    text = bench.headline(full)
    assert len(text) <= bench.LINE_BYTES
    line = json.loads(text)
    assert "cpu_baseline" not in line and "e2e" in line and "clocks" in line and "roofline" in line


def test_config_rows():
    row = bench.config_row(full_result()["configs"][0])
    assert row.startswith("gemma_gate_4096x2048x16384") and "123.5 us" in row
