"""The bench's measured HBM traffic: a record in profiles/ counts while the sources of its kernel are those it was taken
on, and only those."""
import json
import os
import re
import shutil

import pytest

import bench

RECORDS = sorted(f for f in os.listdir(os.path.join(bench.ROOT, "profiles")) if re.fullmatch(r"traffic_\w+\.json", f))


def test_there_is_a_record_of_each_workload():
    assert RECORDS == ["traffic_decode.json", "traffic_prefill.json", "traffic_verify.json"]


@pytest.mark.parametrize("record", RECORDS)
def test_records_are_of_the_current_kernels(record):
    """Fails after a change to a kernel's sources until its traffic has been measured again."""
    with open(os.path.join(bench.ROOT, "profiles", record)) as f:
        rec = json.load(f)
    assert bench.recorded_traffic(record[len("traffic_"):-len(".json")]) == rec["hbm_bytes_per_launch"] > 0


def test_hash_covers_a_unit_and_its_headers_only(tmp_path):
    csrc = str(tmp_path / "csrc")
    shutil.copytree(bench.CSRC, csrc)

    def append(name, text):
        with open(os.path.join(csrc, name), "a") as f:
            f.write(text)

    first = bench.kernel_sources_hash("ffn.hip", csrc)
    assert first == bench.kernel_sources_hash("ffn.hip")
    append("norm.hip", "int another_kernel;\n")
    append("ffn.hip", "// a comment\n/* and another */\n")
    assert bench.kernel_sources_hash("ffn.hip", csrc) == first
    append("route_device.hpp", "int more;\n")                          # included by ffn.hip
    second = bench.kernel_sources_hash("ffn.hip", csrc)
    assert second != first
    append("ffn.hip", "int more;\n")
    assert bench.kernel_sources_hash("ffn.hip", csrc) not in (first, second)
