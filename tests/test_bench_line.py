"""The bench prints one line that a reader of a log's end gets whole: its length stays below a limit with
every measurement in it, and what the contract names is in it unchanged."""

import json

import bench


def _record():
    x = 41.551999561488626
    us = {"mean": x, "median": x, "p90": x}
    cpu = {"value": 7.546611438514775, "unit": "rounds/s", "cores": 16, "kind": "oracle", "sample": "s" * 300,
           "one_core": {"value": x, "unit": "rounds/s", "cores": 1, "sample": "s" * 170}}
    split = {k: x for k in ("accept_sampled_us", "commit_accepted_us", "prologue_us", "attend_us", "sum_us")}
    prefixes = [4096, 16384, 32768, 65536, 131072]
    cfg = {"workload": "w" * 190, "prefix_rows": 524288, "prefill": {k: x for k in ("ms", "bytes", "achieved_GBps", "frac", "calls")},
           "rounds": 253, "us_per_round": us, "rounds_per_s": x, "realised_accept_mean": x, "round_bytes": 186464051,
           "round_frac": x, "state_bytes_per_sequence": x, "cpu_oracle": cpu}
    point = {k: x for k in ("prefix", "batch", "accept_mean", "us_per_round", "us_mean", "rounds", "realised_accept_mean", "round_frac",
                            "state_bytes", "state_bytes_per_sequence")}
    return {
        "metric": bench.METRIC, "value": 24066.23051966971, "unit": "rounds/s", "n_gpus": 1, "steps": 20, "warmup": 5,
        "ms_per_step": 0.041551999561488626, "higher_is_better": True, "scaling": "weak", "vs_baseline": None, "dtype": "bf16",
        "data": "synthetic", "config": {"workload": "w" * 400}, "gpu_launches": 40,
        "e2e": {"value": 2336.666899907877, "unit": "rounds/s", "h2d_bytes_per_step": 21760256, "d2h_bytes_per_step": 8389120},
        "clocks": {"sm_mhz": 1965.0, "sm_max_mhz": 1965.0, "reasons": []}, "cpu_baseline": cpu,
        "configs": {n: dict(cfg) for n in ("tiny", "qwen3_4b_32k", "qwen3_8b_128k_ragged")},
        "sweep": {"points": [dict(point) for _ in range(60)], "flatness": {f"batch{i}_mean2.5": x for i in range(12)}, "rounds_per_point": 125,
                  "state_bytes_identical_across_prefixes": True},
        "view_ablations": {f"without_{i}": {"views": 7, "attend_us": x, "bytes": 177473536, "GBps": x, "state_bytes_per_sequence": 13336704.0}
                           for i in range(4)},
        "other_output_dtype": {"out_dtype": "f32", "us_per_round": us, "attend_us": us, "attend_bytes": 185862144},
        "state_bytes_per_sequence": 13517280.0,
        "paged": {"page_size": 16, "num_pages": 65907, "prefill": {"ms": x, "frac": x}, "prefill_page_size_256": {"ms": x, "frac": x},
                  "round_us": {"mean": x, "median": x}, "round_bytes": 187029989, "round_slots_us": {"mean": x, "median": x, "rounds": 7}},
        "drafting_round": {"kernels": "k" * 90, "rounds": 17, "bytes": 424848947, "frac": x, "us_per_round": us, "split": dict(split, note="n" * 70),
                           "over_prefix": {
            "us_per_round_median": {str(p): x for p in prefixes}, "flatness": x, "split": {str(p): dict(split) for p in prefixes}}},
        "others": {f"measurement{i}": x for i in range(65)},  # per layer, rooflines, ...
    }


def test_the_line_is_short_and_holds_the_contract():
    full = _record()
    before = json.dumps(full)
    text = json.dumps(bench.short_line(full))
    assert json.dumps(full) == before  # the whole record is not touched
    assert len(before) > 20000 and len(text) < 5000
    d = json.loads(text)
    for key in ("metric", "value", "unit", "n_gpus", "steps", "warmup", "ms_per_step", "higher_is_better", "scaling", "vs_baseline", "dtype",
                "data", "config", "gpu_launches", "clocks"):
        assert d[key] == full[key], key
    assert d["e2e"]["h2d_bytes_per_step"] == 21760256 and d["e2e"]["d2h_bytes_per_step"] == 8389120
    assert abs(d["e2e"]["value"] / full["e2e"]["value"] - 1) < 1e-5
    assert d["sweep"]["points"] == 60 and d["configs"]["tiny"]["cpu_oracle"] == 7.54661
    assert d["state_bytes_per_sequence"] == 13517280 and d["cpu_baseline"]["one_core"] == 41.552
    assert "split" in d["drafting_round"] and "split" not in d["drafting_round"]["over_prefix"]


def test_a_run_that_skipped_its_parts():
    full = {**_record(), "sweep": None, "configs": None, "drafting_round": None,
            "view_ablations": None, "other_output_dtype": None}
    full.pop("cpu_baseline")
    d = bench.short_line(full)
    assert d["sweep"] is None and d["configs"] is None and d["drafting_round"] is None and d["value"] == full["value"]
