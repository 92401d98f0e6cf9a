"""bench.py's line, what needs no GPU: the DRAM traffic figures it reports belong to
the kernels as they are."""
import bench


def test_traffic_figures_describe_the_current_kernels():
    """A figure is reported while the sources it was captured with stand; the default
    run's calls (down at M = 128 under both partition rules, decode attention) and
    gate at M = 32 keep theirs."""
    assert {h for _, h in bench.NCU_TRAFFIC.values()} == {bench.tc_source_hash()}
    assert {("down", 128, 4), ("down", 128, 7), ("gate", 32, 2)} <= set(bench.NCU_TRAFFIC)
    assert {h for _, h in bench.ATTN_TRAFFIC.values()} == {bench.tc_source_hash(bench.ATTN_SOURCES)}


def test_line_is_short_and_loses_nothing():
    """14 calls, 35 swept shapes and the rest of a run's keys at their usual sizes fit
    16 KB, on one line; the tables give back every row."""
    import json
    call = {"proj": "down", "M": 128, "Kred": 9728, "Nout": 2560, "split": 4, "us_split": 12.345,
            "us_unsplit": 123.456, "bytes": 16093696, "flops": 6710886400.0, "bound": "hbm",
            "roof_frac_split": 0.1785, "roof_frac_unsplit": 0.0934, "tbps_split": 1.2134,
            "tflops_split": 100.36, "split_near_equal": 7, "us_near_equal": 6.687,
            "roof_frac_near_equal": 0.1785, "copies": 52}
    row = {"proj": "gate", "M": 2048, "Kred": 2560, "Nout": 9728, "split": 1, "base_ctas": 1234,
           "us": 123.456, "control_split": 2, "control_us": 123.456, "speedup_vs_control": 1.057,
           "bound": "tensor", "roofline_frac": 0.1292, "planned_split": 2, "planned_us": 123.456}
    out = {"metric": "µs/call", "value": 8.7575, "rest": "x" * 7000,
           "per_call": [dict(call, M=i) for i in range(14)],
           "split_vs_control": {"summary": {"shapes": 35},
                                "rows": [dict(row, M=i) for i in range(35)]}}
    line = bench.json_line(out)
    assert len(line.encode()) < 16384 and "\n" not in line
    got = json.loads(line)
    for name, rows in (("per_call", out["per_call"]),
                       ("split_vs_control", out["split_vs_control"]["rows"])):
        t = got[name]
        assert [dict(zip(t["columns"], r)) for r in t["rows"]] == rows
    assert got["split_vs_control"]["summary"] == {"shapes": 35} and got["value"] == 8.7575
    assert bench.as_table([{"a": 1}, {"a": 2, "b": 3}]) == {"columns": ["a", "b"],
                                                           "rows": [[1, None], [2, 3]]}
