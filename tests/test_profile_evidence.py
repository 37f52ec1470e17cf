"""The committed profiles of the exchange's kernels are of the present sources:
bench.py reports their averages and traffic only while the hashes agree."""
import glob
import json
import os
import shutil

import pytest

import bench

PROFILES = os.path.join(bench.ROOT, "profiles")
COUNTERS = sorted(glob.glob(os.path.join(PROFILES, "counters_*.json")))
TRACES = [p for p in sorted(glob.glob(os.path.join(PROFILES, "*.md")))
          if any(line.startswith("sources_hash: ") for line in open(p))]


def test_counter_summaries_are_current():
    assert len(COUNTERS) >= 60
    for path in COUNTERS:
        d = json.load(open(path))
        assert d["sources_hash"] == bench.kernel_sources_hash(d["kernel"]), path
        assert bench.load_counter_traffic(d["kernel"], d["workload"]) == d["hbm_bytes_per_launch"]


def test_traces_are_current():
    assert len(TRACES) >= 15
    for path in TRACES:
        stamp = [line for line in open(path) if line.startswith("sources_hash: ")]
        assert stamp[0].split()[1] == bench.kernel_sources_hash(), path
    assert bench.load_trace_average("combine_kernel", "large_batch_per_expert_bf16") > 0
    assert bench.load_trace_average("dispatch_bf16_kernel", "large_batch_per_expert_bf16") > 0


def test_the_hashes_cover_the_measured_kernels_sources_only(tmp_path, monkeypatch):
    """A change to a file that holds a measured kernel, or to a shared header, shows; one elsewhere in csrc does not."""
    csrc = tmp_path / "combine_epx_get_amd" / "csrc"
    shutil.copytree(os.path.join(bench.ROOT, "combine_epx_get_amd", "csrc"), csrc)
    monkeypatch.setattr(bench, "ROOT", str(tmp_path))
    every, one = bench.kernel_sources_hash(), bench.kernel_sources_hash("combine_kernel")
    (csrc / "epx_other.hip").write_text("// another operator\n")
    with open(csrc / "epx_api.hip", "a") as f:
        f.write("// an entry point\n")
    assert (every, one) == (bench.kernel_sources_hash(), bench.kernel_sources_hash("combine_kernel"))
    with open(csrc / "epx_layout.hip", "a") as f:
        f.write("// a kernel\n")
    assert bench.kernel_sources_hash() != every and bench.kernel_sources_hash("combine_kernel") == one
    with open(csrc / "epx_device.h", "a") as f:
        f.write("// shared\n")
    assert bench.kernel_sources_hash("combine_kernel") != one


@pytest.mark.parametrize("kernel", sorted(bench.KERNEL_SOURCE))
def test_every_measured_kernel_has_its_source(kernel):
    path = os.path.join(bench.ROOT, "combine_epx_get_amd", "csrc", bench.KERNEL_SOURCE[kernel])
    assert f"{kernel}(" in open(path).read()
