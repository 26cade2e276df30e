"""The headline's line stays short enough to be read from the end of a log."""
import json

import bench


def test_compact_sweep():
    rows = []
    for config in ("tiny", "2A2F", "2A2F-H4096", "skew-3A1F", "fp8-2A2F"):
        for T in (1, 512, 2048):
            for combine in ("fused", "two-stage-fp8"):
                for variant in ("full", "batched collect"):
                    rows.append({"config": config, "T": T, "combine": combine, "variant": variant, "us": 123.45,
                                 "us_back_to_back": 120.01, "bytes": 303300608, "gbs": 5242.3,
                                 "frac": 0.7735 if T >= 512 else None, "context": {"note": "x" * 100}, "oracle_us": 1.0,
                                 "oracle_reps": 3})
    out = bench.compact_sweep(rows)
    assert len(out) == len(rows) == 60
    assert out["2A2F T=2048"] == [123.45, 120.01, 0.7735]
    assert out["tiny T=1 two-stage-fp8 batched collect"] == [123.45, 120.01]
    assert len(json.dumps(out)) < 4000
