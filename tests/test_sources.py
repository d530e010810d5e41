"""Every source of the library is one that its build takes (CPU)."""
import os

from muon_newton_schulz_update_amd import build


def test_no_source_is_left_over():
    found = {f for f in os.listdir(build.CSRC) if f.endswith((".hip", ".cpp"))}
    assert found == {*build.DEVICE_SOURCES, *build.HOST_SOURCES, "describe.cpp"}
    for f in os.listdir(build.CSRC):
        assert os.path.getsize(os.path.join(build.CSRC, f)) > 0, f
