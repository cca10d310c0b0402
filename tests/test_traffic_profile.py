"""The DRAM traffic that bench.py reports comes from a committed capture, which
counts only for the kernel sources it was taken of."""
import json
import os

import bench
from block_sparse_attention_fa_gb300 import synth


def test_capture_is_of_these_sources():
    with open(os.path.join(bench.ROOT, "profiles", "dram_traffic.json")) as f:
        d = json.load(f)
    assert d["source_files"] == bench.KERNEL_SOURCES
    assert d["source_digest"] == bench.kernel_source_digest()
    for name, w in synth.WORKLOADS.items():
        if name in d["workloads"]:
            got = bench.measured_traffic(name)
            # at least Q, K, V once; no more than twice the algorithm's bytes
            assert got is not None and bench.algorithmic_bytes(w) // 2 < got < 2 * bench.algorithmic_bytes(w)
    assert len(d["workloads"]) == 4
