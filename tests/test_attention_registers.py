"""The cache attention's kernels keep everything in registers (forms that spilled were found to give wrong rows, for a
cause that was not found), and the exchanges between a wave's lanes stand two wait states behind the vector instruction
that wrote their operands.  Compiled to gfx950 assembly with the build's flags; no GPU needed."""

import os
import re
import shutil
import subprocess
from concurrent.futures import ThreadPoolExecutor

import pytest

from test_dpp_hazard import ROOT, _vregs

SOURCES = ("kda_cache_attend.hip", "kda_cache_attend_rows.hip")


def swap_hazards(text):
    """(swaps of lanes, those whose registers a vector instruction writes within the two instructions in front)."""
    insts = [t.split(";")[0].strip() for t in text.split("\n")]
    insts = [t for t in insts if t and not t.startswith(".") and not t.endswith(":")]
    operands = lambda t: [o.strip() for o in t.split(None, 1)[1].split(",")]      # noqa: E731
    seen, bad = 0, []
    for at, t in enumerate(insts):
        if not re.match(r"v_permlane\d+_swap", t):
            continue
        seen += 1
        mine = _vregs(operands(t)[0]) | _vregs(operands(t)[1])
        waits, j = 0, at - 1
        while j >= 0 and waits < 2:
            if insts[j].startswith("s_nop"):
                waits += int(insts[j].split()[1], 0)
            elif insts[j].startswith("v_"):
                written = _vregs(operands(insts[j])[0])
                if "_swap" in insts[j].split()[0]:
                    written |= _vregs(operands(insts[j])[1])
                if written & mine:
                    bad.append((insts[j], t))
            waits += 1
            j -= 1
    return seen, bad


def test_the_check_sees_a_hazard():
    assert swap_hazards("v_add_f32_e32 v1, v2, v3\nv_permlane32_swap_b32_e32 v1, v4")[1]
    assert swap_hazards("v_add_f32_e32 v1, v2, v3\ns_nop 0\nv_permlane16_swap_b32_e32 v4, v1")[1]
    assert swap_hazards("v_add_f32_e32 v1, v2, v3\ns_nop 1\nv_permlane16_swap_b32_e32 v4, v1") == (1, [])


def test_attention_kernels_do_not_spill(tmp_path):
    hipcc = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
    if not os.path.exists(hipcc):
        pytest.skip("hipcc not available")
    from gated_delta_rule_101_amd.build_lib import CSRC, HIPCC_FLAGS, SOURCE_FLAGS
    assert CSRC.startswith(ROOT)

    def compiled(name):
        out = tmp_path / (name + ".s")
        flags = [f for f in [*HIPCC_FLAGS, *SOURCE_FLAGS.get(name, [])] if f != "-fPIC"]
        r = subprocess.run([hipcc, *flags, "-Rpass-analysis=kernel-resource-usage", "--offload-device-only", "-S",
                            os.path.join(CSRC, name), "-o", str(out)], check=True, capture_output=True, text=True)
        return re.findall(r"Function Name: (\S+)", r.stderr), re.findall(r"ScratchSize \[bytes/lane\]: (\d+)", r.stderr), \
            out.read_text()

    with ThreadPoolExecutor(2) as ex:
        results = list(ex.map(compiled, SOURCES))
    for name, (kernels, scratch, text) in zip(SOURCES, results):
        assert len(kernels) == len(scratch) >= 24, name
        assert not [k for k, s in zip(kernels, scratch) if s != "0"], name
        seen, bad = swap_hazards(text)
        assert seen > 50 and not bad, (name, bad[:3])
