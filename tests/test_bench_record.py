"""CPU tests of the HBM traffic record in bench.py: it belongs to the sources
as they are, and those are the linear layer's alone."""
import os
import re

import bench


def test_the_traffic_record_is_of_these_sources():
    rec = bench.TRAFFIC
    assert bench.src_sha(rec["sources"]) == rec["src_sha256"], \
        "the roofline call's sources changed: take its HBM counters again (bench.py --only fwd_up)"
    assert rec["fetch_bytes"] > 0 and rec["write_bytes"] > 0


def test_the_traffic_record_leaves_out_the_row_operators():
    csrc = os.path.join(bench.ROOT, "qlora_fine_tuning_blockwise_amd", "csrc")
    for name in bench.TRAFFIC["sources"]:
        text = open(os.path.join(csrc, name)).read()
        assert not re.search(r"\bqlora_(embed|norm|distill)_\w+\(", text), name
