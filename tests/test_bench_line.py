"""The benchmark's result line stays short: what is longer than a number or two per batch size goes to stderr."""

import json
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_tables_of_the_result_line_are_short():
    sys.path.insert(0, ROOT)
    import bench

    entry = {"us_per_layer": 12345.67, "unique_MB": 12345.67, "frac": 0.1234, "GBps": 1234.5,
             "stage_us": {f"stage{i}": 1234.56 for i in range(6)}, "ffn_path": "cuda-core/tensor-core"}
    tables = {w: {str(T): dict(entry) for T in bench.WORKLOADS[w].batches} for w in bench.SUITE + bench.NEXT}
    short = bench.short_table(tables)
    assert set(short) == set(tables)
    for w in tables:
        assert set(short[w]) == set(tables[w]) and all(v == [12345.67, 0.1234] for v in short[w].values())
    assert len(json.dumps(short)) < 3000
