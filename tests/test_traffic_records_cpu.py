"""The HBM byte counts that bench.py prints beside its rooflines come from committed
counter runs, and are dropped once a kernel's source has changed: each record belongs
to the source as it is."""
import json
import os

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("record", ["fprop_gemm_traffic.json", "quant_rows_traffic.json"])
def test_traffic_record_belongs_to_the_present_source(record):
    import bench
    rec = json.load(open(os.path.join(ROOT, "profiles", record)))
    assert rec["hbm_bytes_per_launch"] == rec["fetch_bytes_per_launch"] + rec["write_bytes_per_launch"]
    assert bench.traffic_from_profiles(record, rec["source"]) == rec["hbm_bytes_per_launch"], \
        f"take {record} again ({rec['source']} has changed)"
