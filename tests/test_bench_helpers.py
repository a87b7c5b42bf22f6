"""The bench's arithmetic, on the CPU: the algorithmic bytes behind the
roofline's numerator agree with the oracle's packed-layout size and with the
decode figures stated for the workload (36 700 160 B of compressed weight,
37 281 856 B per GEMM launch at M=16, K=4096, N=14336), and the argument
parser accepts every workload mode."""
import os
import subprocess
import sys

import pytest

import bench
import oracle

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("n,k", [(1, 128), (64, 128), (129, 384), (14336, 4096), (4096, 14336),
                                 (28672, 8192)])
def test_compressed_bytes_match_the_layout(n, k):
    assert bench.compressed_weight_bytes(n, k) == oracle.packed_bytes(n, k)


def test_decode_algorithmic_bytes():
    assert bench.compressed_weight_bytes(14336, 4096) == 36700160
    assert bench.gemm_algorithmic_bytes(16, 14336, 4096) == 37281856
    # weight + s_w + A_q + s_a + y
    assert bench.gemm_algorithmic_bytes(1, 14336, 4096) == (
        36700160 + 4 * 14336 + 4096 + 4 + 2 * 14336)


def test_parser_accepts_every_mode():
    r = subprocess.run([sys.executable, os.path.join(ROOT, "bench.py"), "--help"],
                       capture_output=True, text=True, timeout=120)
    assert r.returncode == 0
    for mode in ("decode_gate_up_8b", "prefill_8b", "quantize_tensorwise", "dtype_sweep_8b_up",
                 "stress_70b_mlp"):
        assert mode in r.stdout


class _FakeNvml:
    """Stands in for pynvml: a clock the test sets and a power-cap reason."""
    NVML_CLOCK_SM = 0

    def __init__(self):
        self.mhz = 1965

    def nvmlInit(self):
        pass

    def nvmlDeviceGetHandleByIndex(self, i):
        return i

    def nvmlDeviceGetMaxClockInfo(self, h, kind):
        return 1965

    def nvmlDeviceGetClockInfo(self, h, kind):
        return self.mhz

    def nvmlDeviceGetCurrentClocksThrottleReasons(self, h):
        return 0x4          # sw_power_cap


def test_clock_sampler_pause_keeps_host_only_time_out(monkeypatch):
    """Samples taken while paused (host-only work, idle GPU clocks) must not
    enter the record; the throttle reasons are named."""
    import time
    fake = _FakeNvml()
    monkeypatch.setitem(sys.modules, "pynvml", fake)
    with bench.ClockSampler(0, period_s=0.001) as clk:
        time.sleep(0.05)
        clk.pause()
        n_before = len(clk.samples)
        fake.mhz = 345                      # what an idle GPU would report
        time.sleep(0.05)
        n_paused = len(clk.samples)
        fake.mhz = 1965
        clk.resume()
        time.sleep(0.05)
    s = clk.summary()
    assert n_before > 0
    assert n_paused <= n_before + 1          # at most one sample already in flight
    assert 345 not in clk.samples[n_before + 1:]
    assert s["sm_mhz"] == 1965 and s["sm_max_mhz"] == 1965
    assert s["reasons"] == ["sw_power_cap"] and s["samples"] == len(clk.samples)


def test_oracle_sample_extrapolates_linearly():
    """The oracle baseline on a bounded sample: a positive dense-equivalent
    rate, labelled as extrapolated from the rows and columns it timed."""
    from semi_structured_sparse_rowwise_b200 import synthetic
    x = synthetic.activation(11, 8, 256)
    w = synthetic.weight(12, 96, 256)
    rate, cores, note = bench.oracle_prefill_rate(x, w, seconds=0.05, rows=4, n_sample=32)
    assert rate > 0 and cores >= 1
    assert note.startswith("extrapolated") and "4 of 8 activation rows" in note
    assert "32 of 96 output columns" in note


def test_oracle_offline_sample_scales_to_all_rows():
    """The offline oracle baseline (prune + quantise + compress) on a sample
    of rows: a positive time for the whole weight, labelled as extrapolated."""
    from semi_structured_sparse_rowwise_b200 import synthetic
    w = synthetic.weight(13, 64, 256)
    t, cores, note = bench.oracle_offline_time(w, seconds=0.05, n_sample=16)
    assert t > 0 and cores >= 1
    assert note.startswith("extrapolated") and "16 of 64 weight rows" in note


def _record():
    """A record of the default run's form, with its longest notes."""
    note = "median of 1345 replays of one CUDA graph, each between events " * 4
    clocks = {"sm_mhz": 1965.0, "sm_max_mhz": 1965, "reasons": ["sw_power_cap"], "samples": 3696}
    third = 1234.5678901234567
    linear = {"shape": "", "m": 8192, "k": 4096, "n": 6144, "gemm_us": third, "TFLOP/s": third,
              "roofline": {"frac_sustained": third / 5819.2, "timing": note}, "seeds": {"a": 1}}
    table = [{"m": m, "k": 4096, "n": 14336, "a": a, "w": w, "step_us": third, u: third,
              "cpu_baseline": {"value": third, "sample": note}}
             for m, u in ((1, "GB/s"), (16, "GB/s"), (128, "GB/s"), (1024, "TFLOP/s"),
                          (8192, "TFLOP/s"))
             for a in ("e4m3", "e5m2") for w in ("e4m3", "e5m2")]
    return {
        "metric": bench.METRIC, "value": third, "unit": "GB/s", "n_gpus": 1, "steps": 20,
        "warmup": 5, "ms_per_step": third, "higher_is_better": True, "scaling": "weak",
        "vs_baseline": None, "dtype": "e4m3", "data": "synthetic",
        "config": {"workload": bench.WORKLOAD, "m": 16, "k": 4096, "n": 14336, "a_dtype": "e4m3",
                   "w_dtype": "e4m3", "bias": False, "l2": bench.L2_NOTE, "step": note,
                   "timing": note, "weight_bytes_per_step": 36700160,
                   "seeds": {"a": 100121, "w": 100122, "bias": None}, "parallelism": "single"},
        "roofline": {"bound": "hbm", "achieved": third, "peak": 6452.5, "unit": "GB/s",
                     "frac": third, "traffic": 37432320, "peak_datasheet": 8000.0,
                     "frac_datasheet": third, "kernel": "sparse_linear_kernel",
                     "algorithmic_bytes_per_launch": 37281856,
                     "algorithmic_flop_per_launch": 1879048192.0, "us_per_launch": third,
                     "launches_timed": note, "peak_source": note},
        "quantize_us_per_launch": third,
        "fused_step": {"call": note, "step_us": third, "chained_step_us": third, "timing": note},
        "e2e": {"value": third, "unit": "GB/s", "h2d_bytes_per_step": 131072,
                "d2h_bytes_per_step": 458752, "ms_per_step": third, "replays": 683, "path": note},
        "gpu_launches": 40, "clocks": clocks,
        "offline": {k: {"ms": third, "GB/s": third} for k in (
            "prune_24", "quantize_weight", "compress_24", "prepare_weight_24")},
        "e2e_pipelined": {"value": third, "unit": "GB/s", "ms_per_step": third, "path": note},
        "per_workload": {"prefill_8b": [dict(linear, shape=s) for s in ("qkv", "o", "up", "down")],
                         "dtype_sweep_8b_up": {"table": table, "clocks": clocks, "timing": note},
                         "stress_70b_mlp": {"table": [dict(table[0], m=16384)], "clocks": clocks}},
        "cpu_baseline": {"value": third, "unit": "GB/s", "cores": 16, "kind": "oracle",
                         "sample": note},
        "offline_cpu_baseline": {"value": third, "unit": "GB/s", "ms": third, "cores": 16,
                                 "kind": "oracle", "sample": note},
    }


def test_printed_line_is_short_and_has_every_key():
    """The last kilobytes of the output hold the whole line: every key of the
    record, the headline's figures to their last digit."""
    import json
    record = _record()
    text = json.dumps(bench.brief_line(record))
    assert len(text) < 2000 and "\n" not in text
    line = json.loads(text)
    assert list(line) == list(record)
    for key in ("metric", "value", "unit", "n_gpus", "steps", "warmup", "ms_per_step",
                "higher_is_better", "scaling", "vs_baseline", "dtype", "data", "gpu_launches",
                "clocks"):
        assert line[key] == record[key]
    for key in ("m", "k", "n", "a_dtype", "w_dtype", "l2", "parallelism"):
        assert line["config"][key] == record["config"][key]
    assert line["e2e"]["h2d_bytes_per_step"] == 131072
    assert line["e2e"]["value"] == pytest.approx(record["e2e"]["value"], rel=1e-4)
    assert len(line["per_workload"]["prefill_8b"]) == 4
    sweep = line["per_workload"]["dtype_sweep_8b_up"]
    assert {u: list(r) for u, r in sweep.items()} == {"GB/s": ["m=1", "m=16", "m=128"],
                                                      "TFLOP/s": ["m=1024", "m=8192"]}
    assert record == _record()          # the record itself is left whole
