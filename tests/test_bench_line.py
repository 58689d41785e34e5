"""The benchmark's line stays short enough to be kept whole: contract and headlines on stdout, records on stderr."""
import json

from test_bench_contract import _measurement, bench, gen


def test_line_and_details():
    cfg = gen.CONFIGS["qwen3_30b_a3b"]
    side = bench.summarize(_measurement(cfg), 1900.0, "measured bf16_tflops (burst)")
    line = {"metric": bench.METRIC, "value": 1.0, "unit": "TFLOP/s", "n_gpus": 1, "steps": 20, "warmup": 5, "ms_per_step": 4.1,
            "config": {"workload": "w" * 200}, "e2e": {"value": 1.0, "copies": "c" * 300}, "data": "d" * 100}
    line.update(side)
    names = ("fused_combine", "mxfp8", "fp8_bwd", "fp8_fp4_fwd")
    for n in names:
        line[n] = dict(side)
    line["workloads"] = {n: dict(side) for n in bench.EXTRA_WORKLOADS}
    line["router"] = {"fwd_us": 11.0, "bwd_us": 3.6}
    line["cpu_baseline"] = {"value": 0.07, "sample": "s" * 200}
    line["summary"] = {n: bench.compact(cfg.name, side) for n in names + tuple(bench.EXTRA_WORKLOADS) + (cfg.name,)}
    out, details = bench.split_line(line)
    assert {**out, **details} == line and not set(out) & set(details)
    assert list(out)[-1] == "summary"
    for key in ("metric", "value", "unit", "n_gpus", "steps", "warmup", "ms_per_step", "config", "e2e", "clocks", "roofline",
                "gpu_launches", "kernels", "cpu_baseline", "summary"):
        assert key in out, key
    assert len(json.dumps(out)) < 8192
    assert set(details) == set(names) | {"workloads"}
