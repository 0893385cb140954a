"""The scan's backward kernel reads DPP operands inside inline assembly (fused
row broadcasts, the butterfly's masked additions), where the compiler keeps no
wait states: its assembly is checked like the chunk kernels'
(tests/test_dpp_hazard.py), with the flags the library is built with."""

import os
import shutil
import subprocess

import pytest

from test_dpp_hazard import ROOT, dpp_hazards

SOURCE = os.path.join(ROOT, "gated_delta_rule_101_amd", "csrc", "kda_scan_bwd.hip")


def test_scan_backward_dpp_sources_have_their_wait_states(tmp_path):
    hipcc = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
    if not os.path.exists(hipcc):
        pytest.skip("hipcc not available")
    from gated_delta_rule_101_amd.build_lib import HIPCC_FLAGS, SOURCE_FLAGS
    flags = [f for f in [*HIPCC_FLAGS, *SOURCE_FLAGS.get("kda_scan_bwd.hip", [])] if f != "-fPIC"]
    subprocess.run([hipcc, *flags, "--save-temps", "-c", SOURCE, "-o", str(tmp_path / "k.o")], cwd=tmp_path,
                   check=True, capture_output=True)
    asm = [f for f in os.listdir(tmp_path) if f.endswith(".s") and "gfx950" in f]
    assert asm, os.listdir(tmp_path)
    checked, bad = dpp_hazards(open(tmp_path / asm[0]).read())
    assert checked > 0
    assert not bad, bad[:5]
