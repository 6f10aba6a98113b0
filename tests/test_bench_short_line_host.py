"""The line bench.py prints stays short (readers keep the end of a log only) and keeps the
contract's keys, whatever the full record holds (no GPU)."""
import copy
import json
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import bench  # noqa: E402

X = 1234.5678901234567


def record():
    clocks = {"sm_mhz": 1552.0, "sm_max_mhz": 2070.0, "reasons": ["sw_power_cap"],
              "samples_under_load": 149, "sm_mhz_min": 1492.0, "sm_mhz_max": 2070.0,
              "power_w_max": 1388.313, "region_s": X, "source": "nvml every 10 ms"}
    kernels = {"kernel_number_%d" % i: {"launches_per_step": 26.0, "ms_per_step": X, "share": X}
               for i in range(12)}
    roofline = {"bound": "tensor", "kernel": "bwd_all_gemm", "achieved": X, "peak": X, "unit": "TFLOP/s",
                "frac": 1.0, "frac_of_burst_peak": X, "traffic": 9341471616, "peak_kind": "sustained",
                "peak_source": "x" * 60, "timed_region_s": X, "flops_per_launch": X,
                "counted_note": "n" * 150}
    oracle = {"value": X, "unit": "tokens/s", "cores": 16, "kind": "oracle", "sample": "s" * 120,
              "gpu_over_oracle": X, "scaled": True, "scaled_note": "n" * 150,
              "parity_on_sample": {"rows": 128, "logp": X, "entropy": X, "lse": X, "d_hidden": X}}
    one = {"config": "c" * 70, "steps_per_region": 6, "regions": 3, "ms_per_step": X,
           "ms_per_step_all": [X] * 3, "tokens_per_s": X, "tflops_counted": X, "tflops_executed": X,
           "frac_peak_counted": X, "peak_kind": "sustained", "clocks": clocks,
           "tokens_per_s_per_mhz": X, "fwd": {"ms": X, "tokens_per_s": X, "tflops": X},
           "roofline": roofline, "kernels": kernels, "oracle": oracle, "input_generation_s": X,
           "single_call_fwd_bwd": {"strategy": "keep_logits", "block_tokens": 3840, "ms_per_step": X}}
    return {"metric": "m" * 80, "value": X, "unit": "tokens/s", "n_gpus": 1, "steps": 20, "warmup": 5,
            "ms_per_step": X, "higher_is_better": True, "scaling": "weak", "vs_baseline": None,
            "dtype": "bf16", "data": "synthetic", "config": {"workload": "w" * 80},
            "repeats": {"regions": 5, "ms_per_step_all": [X] * 5, "note": "n" * 80},
            "clocks": clocks, "gpu_launches": 160, "gpu_launches_note": "n" * 60,
            "e2e": {"value": X, "unit": "tokens/s", "h2d_bytes_per_step": 1, "d2h_bytes_per_step": 2},
            "roofline": roofline, "kernels": kernels, "cpu_baseline": oracle,
            "workloads": {n: copy.deepcopy(one) for n in bench.ALL_WORKLOADS}}


def test_short_line():
    full = record()
    before = copy.deepcopy(full)
    d = bench.short_line(full)
    assert full == before
    assert len(json.dumps(d, separators=(",", ":"))) < 8192 < len(json.dumps(full))
    for k, v in full.items():
        if k not in ("workloads", "gpu_launches_note", "roofline", "repeats", "cpu_baseline"):
            assert d[k] == v, k
    assert d["roofline"]["frac"] == 1.0 and d["roofline"]["traffic"] == 9341471616
    assert d["cpu_baseline"]["sample"] and d["repeats"]["regions"] == 5
    assert list(d["workloads"]) == list(bench.ALL_WORKLOADS)
    for w in d["workloads"].values():
        assert w["ms_per_step"] == w["tokens_per_s"] == X and w["oracle"]["kind"] == "oracle"
        assert w["oracle"]["scaled"] is True and set(w["oracle"]["parity_on_sample"]) >= {"logp", "d_hidden"}
    assert bench.short_line({"metric": "m", "value": 1.0}) == {"metric": "m", "value": 1.0}
