"""The committed counter records that bench.py reports from are of the kernels
as they are: each was taken on the sources that it names, which hold nothing
of the recurrent layer's operators."""
import json
import os

import pytest

bench = pytest.importorskip("bench")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("name", ["traffic.json", "sq.json"])
def test_records_are_of_the_current_sources(name):
    with open(os.path.join(ROOT, "profiles", name)) as fh:
        records = {k: v for k, v in json.load(fh).items() if not k.startswith("_")}
    assert records
    stale = [k for k in records if bench._profile_record(name, k) is None]
    assert not stale, "taken on other sources: %s" % ", ".join(stale)


def test_traffic_is_reported():
    for key in ("scan", "ssd_chunk_scan", "decode", "conv", "bwd", "bwd_ckpt", "ssd_bwd_dx"):
        assert bench.measured_traffic(key) > 0
