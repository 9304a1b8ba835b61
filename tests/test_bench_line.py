"""The benchmark's line stays short enough to be kept whole, and says what it has to."""
import json

import bench

MUST = ("metric", "value", "unit", "n_gpus", "steps", "warmup", "ms_per_step", "higher_is_better",
        "scaling", "vs_baseline", "dtype", "data", "config", "clocks", "gpu_launches", "e2e")


def test_long_tables_are_not_in_the_line():
    point = {"us": 12.3456789012, "hbm_gbs": 4321.123456789, "tflops": 987.654321987}
    big = {f"config_{i}": {f"variant_{j}": dict(point) for j in range(20)} for i in range(20)}
    out = {k: 1.0 for k in MUST}
    out.update(value=68603049.12926175, n_gpus=1, vs_baseline=None, config={"M": 256},
               roofline={"frac": 0.3402575948860326}, variants={"det": dict(point)},
               cpu_baseline={"value": 1.5, "cores": 1, "per_config": big, "per_config_how": "x"},
               prefill={"timing": "x", "stacked": {"a": {"det": dict(point), "how": "x"}}, "large": big})
    for k in bench.DETAILS:
        out.setdefault(k, big)
    line, details = bench.result_lines(out)
    assert all(k in line for k in MUST)
    assert len(json.dumps(line)) < 2000 < len(json.dumps(details))
    assert line["n_gpus"] == 1 and line["vs_baseline"] is None
    assert abs(line["value"] / out["value"] - 1) < 1e-5
    assert line["prefill_us"] == {"a": {"det": 12.3457}}
    assert line["cpu_baseline"] == {"value": 1.5, "cores": 1}
    assert details["cpu_baseline"]["per_config"].keys() == big.keys()
    assert all(k in details for k in bench.DETAILS)


def test_without_the_optional_tables():
    line, details = bench.result_lines({"metric": "m", "value": 2.0, "prefill": {}})
    assert line == {"metric": "m", "value": 2.0} and details == {"prefill": {}}
