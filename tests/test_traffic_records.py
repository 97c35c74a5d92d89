"""The DRAM bytes that the bench line reports come from captures that are on record."""
import json
import os

import pytest

from conftest import ROOT

with open(os.path.join(ROOT, "profiles", "traffic.json")) as f:
    RECORDS = json.load(f)


@pytest.mark.parametrize("workload", sorted(RECORDS))
def test_record_and_profile_agree(workload):
    r = RECORDS[workload]
    assert r["dram_bytes_per_launch"] == r["dram_bytes_read"] + r["dram_bytes_write"]
    path = r["source"].split(" ")[0]
    with open(os.path.join(ROOT, path)) as f:
        text = f.read()
    assert r["kernel_source_hash"] in text, f"{path} is of another build than its record"
    unit = next(u for u in (1e6, 1e3) if r["dram_bytes_read"] >= u)
    digits = {f"{r['dram_bytes_read'] / unit:.{n}f}" for n in (1, 2)}
    assert any(f"| dram__bytes_read.sum | {d} {'MB' if unit == 1e6 else 'KB'}" in text for d in digits)
