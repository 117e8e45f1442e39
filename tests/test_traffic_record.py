"""The committed DRAM-traffic record belongs to the decode kernel's present
sources, so that the bench line has its roofline's traffic."""
import json
import os

import bench


def test_record_is_of_the_kernels_sources():
    with open(os.path.join(bench.ROOT, "profiles", "traffic.json")) as f:
        record = json.load(f)
    assert bench.load_traffic() == record
    assert bench.traffic_for(record, record["layers"]) == record["bytes_per_launch"]
