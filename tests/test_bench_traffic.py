"""The DRAM traffic that bench.py reports beside its rate is a profiler's record, which holds for the kernel sources it was
taken of: a change of these takes a new record with it."""
import json
import os

import pytest

import bench
from conftest import ROOT

with open(os.path.join(ROOT, "profiles", "traffic.json")) as f:
    RECORD = json.load(f)


@pytest.mark.parametrize("workload", ["c3", "c5"])
def test_the_record_is_of_the_present_sources(workload):
    assert RECORD["source_sha256"] == bench.kernel_source_sha()
    assert bench.recorded_traffic(workload) == RECORD["verify_bytes_per_call"][workload] > 0


def test_the_caches_sources_are_no_part_of_it():
    """Only the verification kernels' sources count: none of them names the paged cache's kernels."""
    csrc = os.path.join(ROOT, "speculative_sampling_verification_spec_gb300", "csrc")
    counted = [n for n in os.listdir(csrc) if n.endswith((".cu", ".cuh", ".h")) and not n.startswith("spec_kv")]
    assert "spec_kernels.cuh" in counted and "spec_verify.cu" in counted
    for n in counted:
        with open(os.path.join(csrc, n)) as f:
            text = f.read()
        assert "kv_mma" not in text and "spec_kv" not in text, n
