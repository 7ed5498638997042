"""bench.py reports HBM bytes a launch from committed counter summaries, which belong to the sources
they were taken on: an edit of those sources takes the figure out of its output until the counters
are taken again."""
import json

import pytest

import bench


@pytest.mark.parametrize("op", bench.COUNTED)
def test_the_summary_belongs_to_the_sources(op):
    traffic, note = bench.counters_traffic(op)
    assert traffic is not None, f"{note}: take FETCH_SIZE and WRITE_SIZE again (the commands are in {bench.counters_path(op).with_suffix('.md').name})"
    c = json.loads(bench.counters_path(op).read_text())
    assert traffic == c["fetch_bytes_per_launch"] + c["write_bytes_per_launch"]
    # every byte the result depends on is read once, and little more than twice at most
    assert bench.COUNTED[op]["alg"] <= traffic < 2.2 * bench.COUNTED[op]["alg"]
