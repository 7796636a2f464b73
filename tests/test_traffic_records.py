"""The committed DRAM records belong to the current sources of their kernels
(no GPU needed): bench.py reports a record only then, so a record that was not
taken again after a change to those sources would be lost from its line."""
import importlib.util
import json
import os

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def records():
    with open(os.path.join(ROOT, "profiles", "traffic.json")) as f:
        return json.load(f)


@pytest.mark.parametrize("kernel", sorted(records()))
def test_a_record_is_of_the_current_sources(kernel):
    spec = importlib.util.spec_from_file_location("bench_for_records", os.path.join(ROOT, "bench.py"))
    bench = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(bench)
    rec = records()[kernel]
    assert rec["source_hash"] == bench.source_hash(kernel, rec["bank"])
    per_slice = rec["slice_dram_read_bytes"] + rec["slice_dram_write_bytes"]
    full = per_slice / rec["slice_algorithmic_bytes"] * rec["full_algorithmic_bytes"]
    assert abs(full - rec["dram_bytes_per_launch"]) <= 1
