"""bench.py's JSON line stays short: who reads the last 16000 characters of its output
finds the whole line there."""
import json

import bench


def arm(us, against=None):
    a = {"decision": "DataParallel", "units_or_splits": 256, "median_us": us, "p10_us": us, "p90_us": us, "min_us": us,
         "round_medians_us": [us] * 9, "tflops": 1234.56, "pct_peak": 49.38, "compulsory_gbps": 1234.5,
         "pct_hbm_peak": 12.34, "pack1": {"median_us": us, "p10_us": us, "p90_us": us, "min_us": us}}
    if against:
        a[f"speedup_vs_{against}"] = {"median": 1.234, "min": 1.2, "max": 1.3}
        a["pack1"][f"speedup_vs_{against}"] = {"median": 1.234, "min": 1.2, "max": 1.3}
    return a


def test_the_line_with_every_arm_stays_short():
    # more arms than the benchmark has: ten shapes of nine
    shapes = {f"c{i}_some_workload": {"M": 2048, "N": 2176, "K": 16384, "dtype": "bf16", "b_layout": "kn",
                                      "protocol": {"rounds": 9, "order": "rotated every sample, reversed every other round"},
                                      **{f"streamk32_in_launch_{j}": arm(1234.567, "dp" if j else None) for j in range(9)}}
              for i in range(10)}
    full, short = json.dumps(shapes), json.dumps(bench.brief(shapes))
    assert len(full) > 16000
    assert len(short) < 13000   # beside it the line holds about 3 KB


def test_an_arm_keeps_its_medians():
    shapes = {"x4_grouped": {"Ms": [448, 96], "N": 2048, "protocol": {}, "separate": {"median_us": 147.9, "tflops": 232.1},
                             "grouped": arm(57.2, "separate")}}
    got = bench.brief(shapes)["x4_grouped"]
    assert got == {"Ms": [448, 96], "N": 2048, "separate": {"median_us": 147.9, "tflops": 232.1},
                   "grouped": {"median_us": 57.2, "tflops": 1234.56, "compulsory_gbps": 1234.5,
                               "speedup_vs_separate": 1.234}}
