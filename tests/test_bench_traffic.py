"""The bench's measured traffic: its digest covers the sources of the kernels that the bench times, and those alone, so
that a byte-counter summary is dropped when they change and kept when another operator does."""
import os
import re
import shutil

import bench

CSRC = os.path.join(bench.ROOT, "bit_quantized_moe_topk_amd", "csrc")
SOURCES_AT_THE_COUNTERS = "f475385b3a549d32"  # of the sources that the committed summaries were taken on


def others():
    return [f for f in os.listdir(CSRC) if f.startswith(bench.OTHER_SOURCES)]


def test_digest_follows_the_timed_kernels_alone(tmp_path):
    d = str(tmp_path / "csrc")
    shutil.copytree(CSRC, d)
    base = bench.kernel_source_hash(d)
    assert base == bench.kernel_source_hash() and others()
    for f in others():
        with open(os.path.join(d, f), "a") as out:
            out.write("// changed\n")
    (tmp_path / "csrc" / "mx4_more.hip").write_text("// new\n")
    assert bench.kernel_source_hash(d) == base
    for f in ("window.hip", "common.h"):
        with open(os.path.join(d, f), "a") as out:
            out.write("// changed\n")
        assert bench.kernel_source_hash(d) != base
        base = bench.kernel_source_hash(d)


def test_timed_kernels_include_no_other_operator():
    for f in os.listdir(CSRC):
        if f.endswith((".hip", ".h")) and f not in others():
            text = open(os.path.join(CSRC, f)).read()
            names = re.findall(r'#include "([^"]+)"', text)
            assert not [n for n in names if os.path.basename(n).startswith(bench.OTHER_SOURCES)], f


def test_summaries_are_found_on_the_sources_they_were_taken_on():
    if bench.kernel_source_hash() != SOURCES_AT_THE_COUNTERS:
        return  # the timed kernels have changed since: the bench rightly reports none
    for kernel, workload in (("win_layer", "decode"), ("mfma_gateup", "prefill_8k"), ("bat_gateup", "batched_decode")):
        assert bench.measured_traffic(kernel, workload) > 0
