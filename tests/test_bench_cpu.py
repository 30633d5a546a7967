"""The bench's reference arm on the host: one JSON line with the keys the
driver reads, the oracle as the timed program, and the same workload config
as the GPU arm (no GPU needed)."""
import json
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_reference_arm_prints_one_contract_line():
    out = subprocess.run([sys.executable, "bench.py", "--impl", "reference", "--steps", "1", "--warmup", "1"],
                         cwd=ROOT, capture_output=True, text=True, timeout=600)
    assert out.returncode == 0, out.stderr[-2000:]
    lines = [ln for ln in out.stdout.splitlines() if ln.strip().startswith("{")]
    assert len(lines) == 1
    d = json.loads(lines[0])
    for key in ("metric", "value", "unit", "n_gpus", "steps", "warmup", "ms_per_step", "higher_is_better",
                "scaling", "vs_baseline", "dtype", "data", "config", "cpu_baseline", "e2e"):
        assert key in d, key
    assert d["impl"] == "reference"
    assert d["steps"] == 1 and d["warmup"] == 1 and d["n_gpus"] == 1
    assert d["value"] > 0 and d["higher_is_better"] is True
    assert d["cpu_baseline"]["kind"] == "oracle" and d["cpu_baseline"]["value"] == d["value"]
    assert d["cpu_baseline"]["cores"] >= 1
    assert d["e2e"] == {"value": d["value"], "unit": d["unit"], "h2d_bytes_per_step": 0, "d2h_bytes_per_step": 0}
    assert "paired Q8_0" in d["config"]["workload"]


def test_traffic_record_follows_the_kernels_sources(tmp_path, monkeypatch):
    """The recorded traffic holds for the sources it was measured on: the
    kernel's own file and every header beside it that it includes."""
    import shutil

    import bench
    args = ("gemv_kernel", "paired_f32_q8_0_2x8192x4096")
    assert bench.traffic_record(*args) > bench.paired_bytes_per_call()["fused"] * 0.9
    csrc = os.path.join("block_quantized_dsq_b200", "csrc")
    monkeypatch.setattr(bench, "ROOT", str(tmp_path))
    for name in ("gemv.cu", "units.cuh", "act_q8.cuh", "dsq_host.h", "dsq_device.cuh"):
        for part in (csrc, "profiles"):
            shutil.copytree(os.path.join(ROOT, part), tmp_path / part, dirs_exist_ok=True)
        assert bench.traffic_record(*args) is not None
        with open(tmp_path / csrc / name, "a") as f:
            f.write("\n")
        assert bench.traffic_record(*args) is None, name


def test_rows_of_the_result_line_are_short():
    """The line is read from the end of a log: with all figures of its 56 rows it was
    21 KB, and a reader that keeps less lost its beginning.  Rows of some 110
    characters with their names keep it under 10."""
    import bench
    full = {"us_per_call": 1234.567, "median_us": 1234.567, "min_us": 1234.5, "max_us": 1299.9, "replays": 21, "calls_per_replay": 35,
            "GB/s": 1234.5, "hbm_frac": 0.1234, "algorithmic_bytes": 123456789, "weight_copies": 35}
    prefill = full | {"TFLOP/s": 1148.7, "bf16_peak_frac": 0.7002, "bound": "tensor", "roofline_frac": 0.7002}
    memory = prefill | {"bound": "hbm", "roofline_frac": 0.1234}
    assert bench.short_row(full) == {"us_per_call": 1234.567, "GB/s": 1234.5, "frac": 0.1234}
    assert bench.short_row(prefill) == {"us_per_call": 1234.567, "TFLOP/s": 1148.7, "frac": 0.7002}
    assert bench.short_row(memory) == {"us_per_call": 1234.567, "GB/s": 1234.5, "frac": 0.1234}
    assert bench.short_row(full | {"m_single_calls_us": 33.28})["m_single_calls_us"] == 33.28
    assert len(json.dumps({"prefill_grouped_q4_k_4096+1024_m2048": bench.short_row(prefill | {"single_calls_us": 119.897})})) <= 150
    assert len(json.dumps({"prefill_q8_0_n8192_m2048": bench.short_row(prefill)})) <= 110
