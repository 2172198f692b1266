"""The benchmark's HBM traffic field (no GPU): the committed counter summaries belong to the present source of
the grouped FFN's kernels, and stop counting when any file that they are compiled from changes."""
import json
import os
import shutil
import sys

import pytest

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import bench  # noqa: E402

WORKLOADS = ("c2", "c3", "c4", "c5")


@pytest.mark.parametrize("workload", WORKLOADS)
def test_counters_are_those_of_this_source(workload):
    with open(os.path.join(bench.ROOT, "profiles", f"grouped_ffn_{workload}_counters.json")) as f:
        summary = json.load(f)
    got = bench.counter_traffic(workload)
    assert got is not None, "re-take the counters: a source of the grouped FFN's kernels changed"
    assert got == summary["hbm_bytes_per_call"] >= 0.99 * summary["alg_bytes_per_call"]
    # the total is that of the kernels listed (each rounded to whole bytes)
    listed = sum(k["fetch_bytes"] + k["write_bytes"] for k in summary["kernels"])
    assert abs(got - listed) <= 2 * len(summary["kernels"])


def test_key_covers_every_file_of_the_kernels(tmp_path, monkeypatch):
    names = bench.ffn_sources()
    assert {"ffn.hip", "lds_tiles.h", "moe_internal.h"} <= set(names)
    csrc = tmp_path / "csrc"
    shutil.copytree(bench.CSRC, csrc)
    monkeypatch.setattr(bench, "CSRC", str(csrc))
    assert bench.counter_traffic("c4") is not None
    for name in names:
        whole = (csrc / name).read_bytes()
        (csrc / name).write_bytes(whole + b"\n")
        assert bench.counter_traffic("c4") is None, name
        (csrc / name).write_bytes(whole)
    assert bench.counter_traffic("c4") is not None
