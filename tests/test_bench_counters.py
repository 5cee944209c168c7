"""The bench line's traffic comes from a committed counter summary, which counts
as long as the kernels' own sources and compiler flags are those it was taken on."""
import pytest

import bench
from quantized_decode_mat_amd import build

FILES = ("gemv_q4k.hip", "q4k_row.h", "xq_device.h")


def test_other_files_do_not_void_the_counters(monkeypatch):
    before = bench.sources_sha(FILES)
    monkeypatch.setattr(build, "SOURCES", build.SOURCES + ["another.hip"])
    assert bench.sources_sha(FILES) == before
    monkeypatch.setattr(build, "FLAGS", build.FLAGS + ["-ffast-math"])
    assert bench.sources_sha(FILES) != before
    assert bench.sources_sha(FILES[:1]) != bench.sources_sha(FILES)


@pytest.mark.parametrize("name", list(bench.COUNTED))
def test_committed_counters_are_of_these_sources(name):
    traffic, note = bench.traffic_from_profile(name)
    assert traffic, note
