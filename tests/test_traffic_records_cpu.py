"""The committed records of DRAM traffic belong to the kernels' present sources (another hash, and the bench's
roofline says nothing of traffic)."""
import glob
import hashlib
import json
import os

import pytest

import bench

RECORDS = sorted(glob.glob(os.path.join(bench.ROOT, "profiles", "*traffic*.json")))


def test_there_are_records():
    names = {n for names in bench.TRAFFIC_RECORDS.values() for n in names} | {"mq_traffic.json"}
    assert names == {os.path.basename(p) for p in RECORDS}


@pytest.mark.parametrize("path", RECORDS, ids=os.path.basename)
def test_record_fits_the_sources(path):
    with open(path) as f:
        rec = json.load(f)
    h = hashlib.sha256()
    for name in rec["sources"]:
        with open(os.path.join(bench.ROOT, "paged_kv_gqa_03_gb300", "csrc", name), "rb") as f:
            h.update(f.read())
    assert h.hexdigest() == rec["source_sha256"]
