"""The benchmark's line: the headline is kept whole, and the line is short enough
that the last 8000 characters of the output hold it."""
import json

import bench


def _record():
    third = 1000.0 / 3.0
    kernels = {f"kernel_{i}": {"launches": 16, "avg_us": third, "us_per_step": third,
                               "algorithmic_bytes": 521338880.0, "GBs": third} for i in range(9)}
    work = {"config": 2, "T": 64, "tokens_per_s": 1e5 / 3, "ms_per_step": third, "host_wall_ms_per_step": third,
            "layer_hbm_GBs": third, "layer_hbm_frac": 1 / 3, "layer_tflops": third,
            "mfma_frac_bf16_peak": 1 / 3, "kernels": kernels}
    stack = {"T": 1, "tokens_per_s": third, "ms_per_step": third, "hbm_frac": 1 / 3, "hit_rate": 1 / 3,
             "h2d_frac_of_link": 1 / 3, "resize": [third] * 8, "popularity_phases": {"0": {"hit_rate": 1 / 3}}}
    sweep = {f"workload_{i}": dict(work) for i in range(11)}
    sweep["stack43_resident"] = {f"T{t}": dict(stack) for t in (1, 2, 4, 8, 16)}
    sweep["stack43_cache32GB"] = {"pool_bytes": 32 * 10 ** 9, **{f"T{t}": dict(stack) for t in (1, 2, 4, 8, 16)}}
    sweep["stack43_qstar"] = {"host_s_per_expert": third,
                              "runs": [{"link": "native", "mode": "qstar", "T": 1, "steps": 24,
                                        "tokens_per_s": third, "ms_per_step": third}] * 6}
    return {"metric": "m" * 80, "value": third, "unit": "tokens/s", "n_gpus": 1, "steps": 20, "warmup": 5,
            "ms_per_step": third, "higher_is_better": True, "scaling": "weak", "vs_baseline": None,
            "dtype": "bf16", "data": "synthetic", "config": {"workload": "w" * 120, "T": 64, "kernels": kernels},
            "roofline": {"bound": "hbm", "achieved": third}, "cpu_baseline": {"value": third},
            "cpu_baseline_sweep": {"runs": [work] * 9}, "micro": {"read_stream": [work] * 8}, "sweep": sweep}


def test_line_keeps_the_headline_and_is_short():
    record = _record()
    text = json.dumps(bench.short_line(record))
    assert len(json.dumps(record)) > 20000 and len(text) < 7000
    line = json.loads(text)
    for k in ("metric", "value", "unit", "n_gpus", "steps", "warmup", "ms_per_step", "higher_is_better",
              "scaling", "vs_baseline", "dtype", "data", "roofline", "cpu_baseline"):
        assert line[k] == record[k]
    assert line["config"] == {"workload": "w" * 120, "T": 64}
    assert set(line["sweep"]) == set(record["sweep"])
    assert line["sweep"]["workload_3"] == {"tokens_per_s": 33333.3, "ms_per_step": 333.333,
                                           "layer_hbm_frac": 0.333333, "layer_tflops": 333.333,
                                           "mfma_frac_bf16_peak": 0.333333}
    assert line["sweep"]["stack43_cache32GB"]["T16"]["hit_rate"] == 0.333333
    assert line["sweep"]["stack43_qstar"]["runs"][0]["mode"] == "qstar"
