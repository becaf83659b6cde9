"""The line that bench.py prints, on the CPU: one JSON line on standard output, short enough for a reader that keeps
the end of the output, with every field of its contract; a longer one goes whole to standard error."""
import json

import pytest


def entry(name, **more):
    return {"us_per_step": 344.97, "median_us_per_step": 341.95, "tokens_per_s": 185522.4, "value": 26876.41, "unit": "GB/s",
            "dtype": "bf16, fp32 accumulate", "steps": 100, "gpu_launches": 100,
            "clocks": {"sm_mhz": 2070.0, "sm_max_mhz": 2070.0, "reasons": [], "samples": 15},
            "parity": {"rows": 64, "max_abs_err": 0.000866600696410702, "tol": 0.01, "within_tolerance": True,
                       "pools_bit_exact": True, "basis": "b" * 180},
            "cpu_baseline": {"value": 6.1857, "unit": "GB/s", "cores": 16, "kind": "oracle", "sample": "s" * 90,
                             "single_thread": {"value": 0.4, "unit": "GB/s", "cores": 1, "sample": "s" * 30}},
            "e2e": {"value": 6990.75, "unit": "GB/s", "h2d_bytes_per_step": 1638656, "d2h_bytes_per_step": 524288, "steps": 200,
                    "copies": "c" * 270},
            "roofline": {"bound": "hbm", "achieved": 7014.4, "peak": 6786.9, "unit": "GB/s", "frac": 1.0335, "traffic": 2398353920.0,
                         "peak_kind": "measured", "kernel": "k" * 70, "mean_launch_us": 340.63, "bytes_basis": "b" * 50,
                         "algorithmic_bytes_per_launch": 2389316012, "launch_timing": "t" * 50},
            "config": {"workload": name, "num_seqs": 64, "q_heads": 32, "kv_heads": 32, "head_size": 128, "block_size": 16,
                       "kv_dtype": "bf16", "num_blocks": 10045, "max_seq_len": 4042, "mean_seq_len": 2275.59375,
                       "partition_tokens": 4048, "cow_pairs": 0, "appended_tokens": 64, "decode": "plain", "l2": "l" * 56,
                       "parallelism": "replicas x1", "launch": "e" * 50, "cta_order": "host plan, longest unit first",
                       "bytes_per_step": {k: 2387218348 for k in ("kv", "decode", "append", "copy", "total", "unique_kv")}}, **more}


def default_line():
    import bench
    names = ["tiny_fp16", "llama7b_mha", "llama3_8b_gqa", "longctx_fp8", "prefix_share", "prefix_share_cascade"]
    return entry("llama7b_mha", metric=bench.METRIC, n_gpus=1, warmup=10, ms_per_step=0.34497, pct_of_hbm_peak=102.05,
                 pct_of_nominal_8tbs=86.58, higher_is_better=True, scaling="weak", vs_baseline=None, data="synthetic",
                 kv_utilisation={"utilisation": 0.99687, "bound": "b" * 50}, configs={n: entry(n) for n in names},
                 next={"prefill_chunked_gqa": entry("prefill_chunked_gqa"), "prefill_chunked_gqa_fp8": entry("prefill_chunked_gqa_fp8"),
                       "prefix_cache_host": {"metric": "m" * 90, "value": 24319.1, "unit": "requests/s", "config": {"n": 1}},
                       "swap_blocks": {"metric": "m" * 60, "unit": "GB/s", "device_to_host": {"us": 2956.95, "GB/s": 193.3},
                                       "host_to_device": {"us": 2708.56, "GB/s": 211.0}}})


CONTRACT = ["metric", "value", "unit", "n_gpus", "steps", "warmup", "ms_per_step", "higher_is_better", "scaling", "vs_baseline",
            "dtype", "data", "config", "e2e", "gpu_launches", "roofline", "clocks", "parity", "cpu_baseline"]


def test_a_long_line_is_printed_short_and_whole_elsewhere(monkeypatch, capsys):
    import bench
    line = default_line()
    assert len(json.dumps(line)) > 4 * bench.LINE_LIMIT
    monkeypatch.setattr(bench, "run_ours", lambda *a: line)
    bench.main([])
    out, err = capsys.readouterr()
    assert out.count("\n") == 1 and len(out) <= bench.LINE_LIMIT
    got = json.loads(out)
    assert all(k in got for k in CONTRACT)
    for k in CONTRACT:
        if not isinstance(line[k], dict):
            assert got[k] == line[k]
    for k in ("value", "unit", "h2d_bytes_per_step", "d2h_bytes_per_step"):
        assert got["e2e"][k] == line["e2e"][k]
    assert got["clocks"] == line["clocks"] and got["roofline"]["frac"] == 1.0335
    assert got["config"]["workload"] == "llama7b_mha" and got["config"]["l2"] == line["config"]["l2"]
    assert set(got["configs"]) == set(line["configs"]) and set(got["next"]) == set(line["next"])
    assert got["configs"]["longctx_fp8"] == {"us_per_step": 344.97, "value": 26876.41, "frac": 1.0335, "ok": True}
    assert got["next"]["swap_blocks"] == {"unit": "GB/s", "device_to_host": 193.3, "host_to_device": 211.0}
    assert json.loads(err) == line


@pytest.mark.parametrize("drop", [("configs", "next"), ("configs", "next", "cpu_baseline", "parity")])
def test_a_short_line_is_printed_as_it_is(drop):
    import bench
    line = {k: v for k, v in default_line().items() if k not in drop}
    line["e2e"] = {**line["e2e"], "copies": "c"}
    if len(json.dumps(line)) <= bench.LINE_LIMIT:
        assert bench.printed_line(line) == json.dumps(line)
    else:
        assert len(bench.printed_line(line)) <= bench.LINE_LIMIT
