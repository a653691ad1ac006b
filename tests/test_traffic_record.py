"""The record of the draft kernel's DRAM traffic that bench.py reports as roofline.traffic."""
import json

import bench


def test_the_record_is_of_the_present_sources():
    """bench.py reports an entry only while the draft kernel's sources are those it was captured from: an entry that
    no longer is reports nothing, and is captured anew or taken out."""
    entries = json.load(open(bench.TRAFFIC))["entries"]
    for e in entries:
        assert e["source_sha16"] == bench.draft_source_hash(), (e["kernel"], e["workload"])
        assert bench.profiled_traffic(e["kernel"], e["workload"]) == e["bytes_per_launch"] > 0
